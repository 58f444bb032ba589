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
__device__ __forceinline__ uint32_t scale_code(float amax, float g, float* s) {
  const uint32_t c = cvt_e4m3x2(__fdiv_rn(amax, __fmul_rn(6.0f, g)), 0.0f);
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

// One warp per (token, head) row of K or V; lane l holds elements
// [l D/32, (l + 1) D/32).  K is rotated in fp64 and rounded once to fp32:
// with fp32 products a value next to a code's border could get another code
// than its definition gives, a whole E2M1 step away.
template <int D>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p) {
  constexpr int E = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = lane_id();
  const int64_t unit = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  if (unit >= 2ll * p.T * p.c.heads) return;
  const bool is_v = unit & 1;
  const int h = static_cast<int>((unit >> 1) % p.c.heads);
  const int64_t t = (unit >> 1) / p.c.heads;
  const int64_t slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= p.c.pages * p.c.page_size) {
    if (lane == 0) atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadSlot));
    return;
  }
  const uint16_t* x = is_v ? p.v + t * p.vt + h * p.vh : p.k + t * p.kt + h * p.kh;
  float a[E];
#pragma unroll
  for (int i = 0; i < E; ++i) a[i] = bf16lo(x[lane * E + i]);
  if (!is_v && p.pos != nullptr) {
    const int half = p.R / 2;
    float y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int d = lane * E + i;
      y[i] = a[i];
      if (d < p.R) {
        const bool second = p.interleaved ? (d & 1) : d >= half;
        const int f = p.interleaved ? d / 2 : (second ? d - half : d);
        const int other = p.interleaved ? d ^ 1 : (second ? d - half : d + half);
        double s, c;
        sincospi(rope::half_turns(p.pos[t], p.freq[f]), &s, &c);
        const double m = p.m, mine = a[i], its = bf16lo(x[other]);
        y[i] = __double2float_rn(second ? fma(mine, c * m, its * (s * m)) : fma(mine, c * m, -its * (s * m)));
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) a[i] = y[i];
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(a[i]));
#pragma unroll
  for (int o = 1; o < 16 / E; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  float s;
  const uint32_t sc = scale_code(amax, is_v ? p.c.vg : p.c.kg, &s);
  uint8_t* base = is_v ? p.c.v : p.c.k;
  const int64_t page = slot / p.c.page_size;
  const int row = static_cast<int>(slot % p.c.page_size);
  uint8_t* codes = base + p.c.code_offset(page, h, row);
#pragma unroll
  for (int i = 0; i < E; i += 2)
    codes[(lane * E + i) / 2] =
        static_cast<uint8_t>(s > 0.0f ? cvt_e2m1x2(__fdiv_rn(a[i], s), __fdiv_rn(a[i + 1], s)) : 0u);
  if (lane % (16 / E) == 0) base[p.c.scale_offset(page, h, row) + lane / (16 / E)] = static_cast<uint8_t>(sc);
}

struct ReadParams {
  Cache c;
  const int64_t* slots;
  uint16_t* k;
  uint16_t* v;
  int64_t kt, kh, vt, vh;
  int T;
};

// The cached values of the given slots as bf16 (zeros for a negative slot):
// one thread per 16 elements.
__global__ void __launch_bounds__(256) read_kernel(ReadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int blocks = p.c.D / 16;
  const int64_t total = 2ll * p.T * p.c.heads * blocks;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int b = static_cast<int>(i % blocks);
    const int64_t r = i / blocks;
    const int h = static_cast<int>(r % p.c.heads);
    const int64_t t2 = r / p.c.heads;
    const bool is_v = t2 >= p.T;
    const int64_t t = is_v ? t2 - p.T : t2;
    uint16_t* y = (is_v ? p.v + t * p.vt + h * p.vh : p.k + t * p.kt + h * p.kh) + b * 16;
    int64_t slot = p.slots[t];
    if (slot >= p.c.pages * p.c.page_size) {
      atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadSlot));
      slot = -1;
    }
    uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0) {
      const uint8_t* base = is_v ? p.c.v : p.c.k;
      const int64_t page = slot / p.c.page_size;
      const int row = static_cast<int>(slot % p.c.page_size);
      const uint2 q = *reinterpret_cast<const uint2*>(base + p.c.code_offset(page, h, row) + b * 8);
      const float s = f16lo(widen_e4m3x2(base[p.c.scale_offset(page, h, row) + b])) * (is_v ? p.c.vg : p.c.kg);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = widen_e2m1x2((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
        o[j] = pack_bf16x2(f16lo(w) * s, f16hi(w) * s);
      }
    }
    reinterpret_cast<uint4*>(y)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(y)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace kv4
}  // namespace fp8q
