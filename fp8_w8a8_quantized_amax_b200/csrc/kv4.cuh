// kv4.cuh -- the 4-bit KV cache: its format, appending to it, reading it back.
//
// For each (page, head) K and V hold one slab each: page_size rows of D/2 code
// bytes (E2M1, the even element in the low nibble), then page_size rows of
// D/16 scale bytes (E4M3, one per 16 elements).  A slab is one contiguous run
// of 9 D / 16 bytes a token, a multiple of 16 bytes for every page size, so
// that attention can fetch it with bulk copies.  A value is
//   E2M1(code) * E4M3(scale) * g,
// g one static fp32 per tensor.  E2M1 has two significant bits and E4M3 four,
// so code times scale is exact in f16 (and in bf16): what reads the cache
// multiplies exact values and applies g once, in fp32.
#pragma once

#include "ptx.cuh"
#include "rope.cuh"

namespace fp8q {
namespace kv4 {

enum : int {
  kErrBadSlot = 0x201,    // a slot past the cache's last page
  kErrBadPage = 0x202,    // a page table entry outside the cache
  kErrBadLength = 0x203,  // a sequence longer than its page table, or rows past the query tensor
};

struct Cache {
  uint8_t* k;
  uint8_t* v;
  int64_t pages;
  int page_size, page_shift, heads, D;
  float kg, vg;
  __host__ __device__ int64_t slab() const { return static_cast<int64_t>(page_size) * (D * 9 / 16); }
  __host__ __device__ int64_t code_offset(int64_t page, int head, int row) const {
    return (page * heads + head) * slab() + row * (D / 2);
  }
  __host__ __device__ int64_t scale_offset(int64_t page, int head, int row) const {
    return (page * heads + head) * slab() + page_size * (D / 2) + row * (D / 16);
  }
};

// Two fp32 -> two E2M1 codes (lo in bits 0..3), round to nearest even, saturating to +-6.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// One byte of two E2M1 codes -> f16x2, exactly.
__device__ __forceinline__ uint32_t widen_e2m1x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}
// Two E4M3 codes -> f16x2, exactly.
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ float f16lo(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(w));
  return f;
}
__device__ __forceinline__ float f16hi(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(w));
  return f;
}

// The scale code of 16 values with the given amax, and the fp32 step s it
// stands for.  fp32 throughout, each operation rounded once (IEEE), so that
// the codes are defined bit for bit:
//   code = E4M3(amax / (6 g)), round to nearest even, saturating;  s = E4M3(code) g
__device__ __forceinline__ uint32_t scale_code(float amax, float g, float g6, float* s) {
  const uint32_t c = cvt_e4m3x2(__fdiv_rn(amax, g6), 0.0f);
  *s = __fmul_rn(f16lo(widen_e4m3x2(c)), g);
  return c;
}

struct AppendParams {
  Cache c;
  const uint16_t* k;
  const uint16_t* v;
  int64_t kt, kh, vt, vh;   // strides in elements: token, head
  const int64_t* slots;
  const int64_t* pos;       // nullptr: no rotation
  const double* freq;
  int T, R, interleaved;
  float m;
};

// x / s, correctly rounded, for the values of a block with amax |x| (the
// correction step of quant.cuh's Divider; its range, narrowed so that nothing
// overflows here).  Quotients too small for the residual to be exact are far
// below the smallest code; the sign is x's.
struct BlockDivider {
  float s, y;
  bool fast;
};
__device__ __forceinline__ float divide(float x, const BlockDivider& d) {
  if (!d.fast) return __fdiv_rn(x, d.s);
  const float q = x * d.y;
  return copysignf(fmaf(fmaf(-q, d.s, x), d.y, q), x);
}

// Bound by HBM for prompts (2 bytes read an element, 9/16 written), by its
// latency for single tokens.  A CTA takes `tokens` tokens: its threads compute
// the tokens' angles into shared memory, once for all heads (an fp64 sincos
// each), with the first rows' loads on the way.  A warp then takes rows of one
// token's K or V, kBatch at a time; a lane holds four elements of a row (a
// half warp a row at D = 64).  K is rotated in fp64 and rounded once to fp32:
// with fp32 products a value next to a code's border could get another code
// than its definition gives, a whole E2M1 step away.
constexpr int kBatch = 4;

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p, int tokens) {
  constexpr int kLanes = D / 4, kRowsPerWarp = 32 / kLanes, kGroup = kBatch * kRowsPerWarp;
  extern __shared__ double2 angles[];               // [tokens][R / 2] (cos, sin)
  griddep_wait();
  griddep_launch_dependents();
  const int lane = lane_id(), warp = threadIdx.x >> 5;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int t0 = blockIdx.x * tokens, nt = min(tokens, p.T - t0);
  const int groups = (p.c.heads + kGroup - 1) / kGroup, half = p.R / 2;
  const int list = nt * 2 * groups;                 // (token, K or V, group of heads)
  // this lane's place in a rotated row: its angles' index, and (half layout) the lane that holds its partners
  const int d = 4 * l;
  const bool turned = d < p.R, second = !p.interleaved && d >= half;
  const int f = p.interleaved ? d / 2 : (second ? d - half : d);
  const int partner = turned && !p.interleaved ? lane + (second ? -half / 4 : half / 4) : lane;
  bool first = true;
  for (int i = warp; i < list || first; i += 8) {
    const int t = i / (2 * groups), rest = i - t * 2 * groups, is_v = rest >= groups, h0 = (is_v ? rest - groups : rest) * kGroup;
    uint2 raw[kBatch];
    int64_t slot = -1;
    if (i < list) {
      slot = p.slots[t0 + t];
      const uint16_t* x = is_v ? p.v + (t0 + t) * p.vt : p.k + (t0 + t) * p.kt;
      const int64_t xh = is_v ? p.vh : p.kh;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int h = h0 + b * kRowsPerWarp + sub;
        raw[b] = make_uint2(0, 0);
        if (h < p.c.heads) raw[b] = *reinterpret_cast<const uint2*>(x + h * xh + d);
      }
    }
    if (first) {
      first = false;
      if (p.pos != nullptr) {
        for (int j = threadIdx.x; j < nt * half; j += 256) {
          double s, c;
          sincospi(rope::half_turns(p.pos[t0 + j / half], p.freq[j % half]), &s, &c);
          angles[j] = make_double2(c * p.m, s * p.m);
        }
        __syncthreads();
      }
      if (i >= list) return;
    }
    if (slot < 0) continue;
    if (slot >= p.c.pages * p.c.page_size) {
      if (lane == 0) atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadSlot));
      continue;
    }
    const float g = is_v ? p.c.vg : p.c.kg, g6 = __fmul_rn(6.0f, g);
    uint8_t* base = is_v ? p.c.v : p.c.k;
    const int64_t page = slot >> p.c.page_shift;
    const int row = static_cast<int>(slot) & (p.c.page_size - 1);
    double2 cs[4];
    const bool turn = p.pos != nullptr && !is_v;
    if (turn && turned) {
#pragma unroll
      for (int e = 0; e < 4; ++e) cs[e] = angles[t * half + (p.interleaved ? f + e / 2 : f + e)];
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h0 + b * kRowsPerWarp + sub;
      float a[4] = {bf16lo(raw[b].x), bf16hi(raw[b].x), bf16lo(raw[b].y), bf16hi(raw[b].y)};
      if (turn) {
        uint2 other = raw[b];
        if (!p.interleaved) {
          other.x = __shfl_sync(0xFFFFFFFFu, raw[b].x, partner);
          other.y = __shfl_sync(0xFFFFFFFFu, raw[b].y, partner);
        }
        if (turned) {
          float o[4] = {bf16lo(other.x), bf16hi(other.x), bf16lo(other.y), bf16hi(other.y)};
          if (p.interleaved) {
            const float y0 = o[0], y2 = o[2];
            o[0] = o[1]; o[1] = y0; o[2] = o[3]; o[3] = y2;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool back = p.interleaved ? (e & 1) : second;          // the pair's second element
            const double mine = a[e], its = o[e];
            a[e] = __double2float_rn(fma(mine, cs[e].x, back ? its * cs[e].y : -its * cs[e].y));
          }
        }
      }
      float amax = fmaxf(fmaxf(fabsf(a[0]), fabsf(a[1])), fmaxf(fabsf(a[2]), fabsf(a[3])));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      BlockDivider dv;
      const uint32_t sc = scale_code(amax, g, g6, &dv.s);
      dv.y = __frcp_rn(dv.s);
      dv.fast = dv.s >= 0x1p-60f && dv.s <= 0x1p60f && amax <= 0x1p60f;
      uint32_t codes = 0;
      if (dv.s > 0.0f)
        codes = cvt_e2m1x2(divide(a[0], dv), divide(a[1], dv)) | (cvt_e2m1x2(divide(a[2], dv), divide(a[3], dv)) << 8);
      if (h < p.c.heads) {
        *reinterpret_cast<uint16_t*>(base + p.c.code_offset(page, h, row) + d / 2) = static_cast<uint16_t>(codes);
        if ((l & 3) == 0) base[p.c.scale_offset(page, h, row) + l / 4] = static_cast<uint8_t>(sc);
      }
    }
  }
}

struct ReadParams {
  Cache c;
  const int64_t* slots;
  uint16_t* k;
  uint16_t* v;
  int64_t kt, kh, vt, vh;
  int T;
};

// The cached values of the given slots as bf16 (zeros for a negative slot): one
// thread per 8 elements (a 16-byte store), two in flight.
template <int D>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kParts = D / 8, kFlight = 2;
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t heads = static_cast<uint32_t>(p.c.heads), per_token = 2 * heads;
  const uint32_t rows = static_cast<uint32_t>(p.T) * per_token;          // (token, K or V, head)
  const int part = threadIdx.x % kParts;
  const uint32_t step = gridDim.x * (256 / kParts);
  for (uint32_t r = blockIdx.x * (256 / kParts) + threadIdx.x / kParts; r < rows; r += kFlight * step) {
    uint32_t codes[kFlight], scale[kFlight];
    uint16_t* y[kFlight];
    float g[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const uint32_t row = r + i * step;
      y[i] = nullptr;
      if (row >= rows || row < r) continue;          // (past the end, or past 2^32)
      const uint32_t t = row / per_token, rest = row - t * per_token;
      const bool is_v = rest >= heads;
      const uint32_t h = is_v ? rest - heads : rest;
      int64_t slot = p.slots[t];
      if (slot >= p.c.pages * p.c.page_size) {
        atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadSlot));
        slot = -1;
      }
      y[i] = (is_v ? p.v + t * p.vt + h * p.vh : p.k + t * p.kt + h * p.kh) + part * 8;
      g[i] = is_v ? p.c.vg : p.c.kg;
      codes[i] = scale[i] = 0;
      if (slot >= 0) {
        const uint8_t* base = is_v ? p.c.v : p.c.k;
        const int64_t page = slot >> p.c.page_shift;
        const int in_page = static_cast<int>(slot) & (p.c.page_size - 1);
        codes[i] = *reinterpret_cast<const uint32_t*>(base + p.c.code_offset(page, h, in_page) + part * 4);
        scale[i] = base[p.c.scale_offset(page, h, in_page) + part / 2];
      }
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (y[i] == nullptr) continue;
      const float s = f16lo(widen_e4m3x2(scale[i]));
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {                  // code * scale is exact; then one fp32 product, one rounding to bf16
        const uint32_t w = widen_e2m1x2(codes[i] >> (8 * j));
        o[j] = pack_bf16x2(f16lo(w) * s * g[i], f16hi(w) * s * g[i]);
      }
      *reinterpret_cast<uint4*>(y[i]) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace kv4
}  // namespace fp8q
