// kv4.cuh -- the 4-bit KV cache: its format, appending to it, reading it back.
//
// For each (page, head) K and V hold one slab each: page_size rows of D/2 code
// bytes (E2M1, the even element in the low nibble), then page_size rows of
// D/16 scale bytes (E4M3, one per 16 elements).  A slab is one contiguous run
// of 9 D / 16 bytes a token; it, its scales and every 16 rows of either are
// multiples of 16 bytes, so that 16-byte copies and loads stay aligned.  A value is
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

// Two quotients x / s, correctly rounded, from the negated values (the
// correction step of quant.cuh's Divider, on packed fp32; it runs on -x so that
// a zero keeps its sign).  y = RN(1 / s).  Right where s lies in [2^-60, 2^60]
// and |x| <= 2^60: nothing overflows, and quotients too small for the residual
// to be exact are far below the smallest code.
__device__ __forceinline__ uint32_t encode2(float nx0, float nx1, uint64_t ny2, uint64_t s2) {
  const uint64_t nx = f32x2_pack(nx0, nx1), q = mul_f32x2(nx, ny2), r = fma_f32x2(q, s2, nx);
  float q0, q1;
  f32x2_unpack(fma_f32x2(r, ny2, q), q0, q1);
  return cvt_e2m1x2(q0, q1);
}

// Bound by HBM for prompts (2 bytes read an element, 9/16 written) as far as
// the instructions allow, by its latency for single tokens.  A CTA takes
// `tokens` tokens: its threads compute the tokens' angles into shared memory,
// once for all heads (an fp64 sincos each), with the first blocks' loads on the
// way.  A thread keeps its place (head, block of 16 elements) and walks over
// the tokens' K and V: the scale is computed once for 16 values and nothing is
// exchanged between lanes.  K is rotated in fp64 and rounded once to fp32: with
// fp32 products a value next to a code's border could get another code than
// its definition gives, a whole E2M1 step away.  A block's partners (half
// layout) are read from memory as well; they are another thread's elements, so
// they come from L1.  8192 tokens of 8 heads of 128, four tokens a CTA: 21 us,
// 2.0 TB/s (D = 64: 12 us; 4 bytes spill there); 65% of the issue slots are taken
// (quotients, conversions and the fp64 rotation), no unit is at its limit, and
// loads one step further ahead and fewer CTAs changed nothing.  64 tokens: 2.4 us.
// A CTA has 2 tokens heads D / 16 blocks for its 256 threads, whatever the number
// of heads: 8192 tokens of one head take 10 us, of two 11.
template <int D>
__global__ void __launch_bounds__(256, 4) append_kernel(const __grid_constant__ AppendParams p, int tokens) {
  constexpr int kBlocks = D / 16, kCols = D / 32;
  // [tokens][16][kCols] (cos, sin); pair f at (f % 16, f / 16): for one element of their blocks, neighbouring threads
  // read neighbouring entries
  extern __shared__ double2 angles[];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * tokens, nt = min(tokens, p.T - t0);
  const int half = p.R / 2, places = p.c.heads * kBlocks;
  const int groups = max(1, 256 / places), group = threadIdx.x / places;
  const float kg6 = __fmul_rn(6.0f, p.c.kg), vg6 = __fmul_rn(6.0f, p.c.vg);
  bool first = true;
  for (int place = threadIdx.x - group * places; place < places || first; place += 256) {
    const int h = place / kBlocks, d0 = place % kBlocks * 16;
    const bool turns = p.pos != nullptr && d0 < p.R;
    for (int j = group; j < 2 * nt || first; j += groups) {
      const bool there = j < 2 * nt && group < groups && place < places;
      const int t = j >> 1;
      const bool is_v = j & 1;
      const bool turn = turns && !is_v;
      uint32_t raw[8];
      uint2 other[4];
      int64_t slot = -1;
      if (there) {
        slot = p.slots[t0 + t];
        const uint16_t* x = is_v ? p.v + (t0 + t) * p.vt + h * p.vh : p.k + (t0 + t) * p.kt + h * p.kh;
        const uint4 lo = *reinterpret_cast<const uint4*>(x + d0), hi = *reinterpret_cast<const uint4*>(x + d0 + 8);
        raw[0] = lo.x; raw[1] = lo.y; raw[2] = lo.z; raw[3] = lo.w;
        raw[4] = hi.x; raw[5] = hi.y; raw[6] = hi.z; raw[7] = hi.w;
        if (turn && !p.interleaved) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {              // R is a multiple of 8: four elements change sides together
            const int d = d0 + 4 * q;
            if (d < p.R) other[q] = *reinterpret_cast<const uint2*>(x + (d < half ? d + half : d - half));
          }
        }
      }
      if (first) {
        first = false;
        if (p.pos != nullptr) {
          for (int i = threadIdx.x; i < nt * half; i += 256) {
            const int u = i / half, f = i - u * half;
            angles[(u * 16 + (f & 15)) * kCols + (f >> 4)] = rope::cos_sin_f64(p.pos[t0 + u], p.freq[f], p.m);
          }
          __syncthreads();
        }
        if (!there) return;
      }
      if (slot < 0) continue;
      if (slot >= p.c.pages * p.c.page_size) {
        atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadSlot));
        continue;
      }
      float a[16];                                   // the negated values
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t n = raw[e] ^ 0x80008000u;
        a[2 * e] = bf16lo(n);
        a[2 * e + 1] = bf16hi(n);
      }
      if (turn) {
        const double2* table = angles + t * 16 * kCols;
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            if (d0 + e < p.R) {
              const int f = (d0 + e) / 2;
              const double2 cs = table[(f & 15) * kCols + (f >> 4)];
              const double x0 = a[e], x1 = a[e + 1];
              a[e] = __double2float_rn(fma(x0, cs.x, -x1 * cs.y));
              a[e + 1] = __double2float_rn(fma(x1, cs.x, x0 * cs.y));
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int d = d0 + 4 * q;
            if (d < p.R) {
              const bool second = d >= half;
              const int f = second ? d - half : d;   // a multiple of 4: its four pairs lie kCols apart
              const double2* cs = table + (f & 15) * kCols + (f >> 4);
              const uint32_t sign = second ? 0x80008000u : 0u;             // -its x1's sign in y0, +its x0's in y1, negated
              const uint32_t o0 = other[q].x ^ sign, o1 = other[q].y ^ sign;
              const float o[4] = {bf16lo(o0), bf16hi(o0), bf16lo(o1), bf16hi(o1)};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const double2 c = cs[e * kCols];
                a[4 * q + e] = __double2float_rn(fma(static_cast<double>(a[4 * q + e]), c.x, static_cast<double>(o[e]) * c.y));
              }
            }
          }
        }
      }
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) amax = fmaxf(fmaxf(fabsf(a[e]), fabsf(a[e + 1])), amax);
      float s;
      const uint32_t sc = scale_code(amax, is_v ? p.c.vg : p.c.kg, is_v ? vg6 : kg6, &s);
      uint32_t codes[2] = {0, 0};
      if (s >= 0x1p-60f && s <= 0x1p60f && amax <= 0x1p60f) {
        const float y = -__frcp_rn(s);
        const uint64_t ny2 = f32x2_pack(y, y), s2 = f32x2_pack(s, s);
#pragma unroll
        for (int e = 0; e < 16; e += 2) codes[e / 8] |= encode2(a[e], a[e + 1], ny2, s2) << (4 * (e % 8));
      } else if (s > 0.0f) {
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          codes[e / 8] |= cvt_e2m1x2(__fdiv_rn(-a[e], s), __fdiv_rn(-a[e + 1], s)) << (4 * (e % 8));
      }
      uint8_t* base = is_v ? p.c.v : p.c.k;
      const int64_t page = slot >> p.c.page_shift;
      const int row = static_cast<int>(slot) & (p.c.page_size - 1);
      *reinterpret_cast<uint2*>(base + p.c.code_offset(page, h, row) + d0 / 2) = make_uint2(codes[0], codes[1]);
      base[p.c.scale_offset(page, h, row) + d0 / 16] = static_cast<uint8_t>(sc);
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
// thread per 16 elements of one row, as many threads as there are such blocks
// (two or four a thread, loads first: 10.1 and 12.9 us where this takes 8.8, for
// 8192 tokens of 8 heads of 128: 4.9 TB/s, partly of L2).
template <int D>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kBlocks = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t heads = static_cast<uint32_t>(p.c.heads), per_token = 2 * heads;
  const uint32_t row = blockIdx.x * (256 / kBlocks) + threadIdx.x / kBlocks;   // (token, K or V, head)
  if (row >= static_cast<uint32_t>(p.T) * per_token) return;
  const int block = threadIdx.x % kBlocks;
  const uint32_t t = row / per_token, rest = row - t * per_token;
  const bool is_v = rest >= heads;
  const uint32_t h = is_v ? rest - heads : rest;
  int64_t slot = p.slots[t];
  if (slot >= p.c.pages * p.c.page_size) {
    atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadSlot));
    slot = -1;
  }
  uint2 codes = make_uint2(0, 0);
  uint32_t scale = 0;
  if (slot >= 0) {
    const uint8_t* base = is_v ? p.c.v : p.c.k;
    const int64_t page = slot >> p.c.page_shift;
    const int in_page = static_cast<int>(slot) & (p.c.page_size - 1);
    codes = *reinterpret_cast<const uint2*>(base + p.c.code_offset(page, h, in_page) + block * 8);
    scale = base[p.c.scale_offset(page, h, in_page) + block];
  }
  const float s = f16lo(widen_e4m3x2(scale)), g = is_v ? p.c.vg : p.c.kg;
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {                      // code * scale is exact; then one fp32 product, one rounding to bf16
    const uint32_t w = widen_e2m1x2((j < 4 ? codes.x : codes.y) >> (8 * (j & 3)));
    o[j] = pack_bf16x2(f16lo(w) * s * g, f16hi(w) * s * g);
  }
  uint4* y = reinterpret_cast<uint4*>((is_v ? p.v + t * p.vt + h * p.vh : p.k + t * p.kt + h * p.kh) + block * 16);
  y[0] = make_uint4(o[0], o[1], o[2], o[3]);
  y[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace kv4
}  // namespace fp8q
