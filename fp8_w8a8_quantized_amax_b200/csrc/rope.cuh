// rope.cuh -- rotary positions: the angles, and the rotation of bf16 heads.
//
// A pair (x0, x1) of a head at position p is turned by the angle a = p f_i:
//   y0 = x0 c - x1 s,  y1 = x1 c + x0 s,  c = m cos a, s = m sin a
// (s changes sign for the inverse rotation, which is also the gradient of the
// forward one).  The half layout pairs dimension i with i + R/2, the
// interleaved one 2i with 2i + 1 (i < R/2); dimensions from R on are copied.
#pragma once

#include "ptx.cuh"

namespace fp8q {
namespace rope {

// cos and sin of p * f.  The angle is taken in turns in fp64 (p f / 2 pi, off
// by at most 2^-52 of itself: 4e-11 turns at a million positions) and reduced
// by a whole number of turns, exactly; fp32 would lose the angle of far
// positions (at p = 131072 and f = 1, a step of fp32 is 0.008 radians).
constexpr double kTurnsPerRadian = 0.15915494309189533577;

// The fraction of a turn, in [-1/2, 1/2].
__device__ __forceinline__ double turn(int64_t p, double f) {
  const double t = static_cast<double>(p) * (f * kTurnsPerRadian);
  return t - rint(t);
}

__device__ __forceinline__ float2 cos_sin(int64_t p, double f, float m, bool inverse) {
  float s, c;
  sincospif(static_cast<float>(2.0 * turn(p, f)), &s, &c);   // |half turns| <= 1: fp32 is off by 2^-25 of a turn
  return make_float2(c * m, inverse ? -s * m : s * m);
}

// The same in fp64, by the Taylor series on an eighth of a turn to either side
// of the nearest quarter: with |x| <= pi / 4 the first terms left out are
// x^17 / 17! < 5e-17 and x^18 / 18! < 3e-18.  (The library's sincospi took a
// third of the append kernel's instructions.)
__device__ __forceinline__ double2 cos_sin_f64(int64_t p, double f, double m) {
  const double r = turn(p, f), quarter = rint(4.0 * r);
  const double x = 6.283185307179586477 * fma(quarter, -0.25, r), z = x * x;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;
  s = fma(s, z, 1.0 / 6227020800.0);
  c = fma(c, z, -1.0 / 87178291200.0);
  s = fma(s, z, -1.0 / 39916800.0);
  c = fma(c, z, 1.0 / 479001600.0);
  s = fma(s, z, 1.0 / 362880.0);
  c = fma(c, z, -1.0 / 3628800.0);
  s = fma(s, z, -1.0 / 5040.0);
  c = fma(c, z, 1.0 / 40320.0);
  s = fma(s, z, 1.0 / 120.0);
  c = fma(c, z, -1.0 / 720.0);
  s = fma(s, z, -1.0 / 6.0);
  c = fma(c, z, 1.0 / 24.0);
  s = fma(s * z, x, x);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  const int q = static_cast<int>(quarter) & 3;     // cos and sin of q quarters and x
  const double a = (q & 1) ? s : c, b = (q & 1) ? c : s;
  return make_double2((q == 1 || q == 2) ? -a * m : a * m, (q & 2) ? -b * m : b * m);
}

struct Params {
  const uint16_t* x;
  uint16_t* y;
  const int64_t* pos;
  const double* freq;
  int64_t xt, xh, yt, yh;   // strides in elements: token, head
  int T, H, D, R;
  float m;
  int interleaved, inverse;
};

// Any strides and alignment, any even R: one thread per pair of a (token, head);
// the dimensions behind the rotated part are copied by the same threads.  An
// angle in fp64 for each pair and 2-byte accesses bound it: 8192 tokens of 40
// heads of 128 take 57 us with R = 24 (2.9 TB/s), 73 with R = 40, 147 with R = 128
// and unaligned rows, where the kernel below takes 28 to 35.
__global__ void __launch_bounds__(256) rope_any_kernel(const __grid_constant__ Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int half = p.R / 2;
  const int64_t total = static_cast<int64_t>(p.T) * p.H * half;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int k = static_cast<int>(i % half);
    const int64_t row = i / half;
    const int h = static_cast<int>(row % p.H);
    const int64_t t = row / p.H;
    const uint16_t* x = p.x + t * p.xt + h * p.xh;
    uint16_t* y = p.y + t * p.yt + h * p.yh;
    const float2 cs = cos_sin(p.pos[t], p.freq[k], p.m, p.inverse != 0);
    const int d0 = p.interleaved ? 2 * k : k, d1 = p.interleaved ? 2 * k + 1 : k + half;
    const float x0 = bf16lo(x[d0]), x1 = bf16lo(x[d1]);
    const uint32_t o = pack_bf16x2(x0 * cs.x - x1 * cs.y, x1 * cs.x + x0 * cs.y);
    y[d0] = static_cast<uint16_t>(o);
    y[d1] = static_cast<uint16_t>(o >> 16);
    if (p.x != p.y)
      for (int d = p.R + k; d < p.D; d += half) y[d] = x[d];
  }
}

// 16-byte rows and R a multiple of 16: bound by HBM (2 bytes read, 2 written an
// element).  A CTA takes `tokens` tokens; its threads first compute the
// tokens' angles into shared memory, once for all heads (an fp64 product, a
// reduction and an fp32 sincos each: per element they would cost more than the
// bytes), with their first loads already on the way.  A unit is eight pairs:
// two 16-byte vectors, R / 2 apart (half layout) or side by side (interleaved).
// A thread walks the units u, u + 256, ... of the CTA's (token, head, unit)
// list, one at a time: the loads in flight come from eight CTAs an SM (32
// registers; the interleaved layout needs a few more, so six: 3.5 against 3.8
// us for 777 tokens of 13 heads of 64), which beat two units a thread with four
// CTAs and loads one step ahead (8 and 24 bytes spill).  8192 tokens of 8 + 32 heads
// of 128 take 28.5 us, 5.9 TB/s (four tokens a CTA; 33.8 us with eight); interleaved
// 32.8, and 34.6 with R = 64.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(256, INTERLEAVED ? 6 : 8) rope_vec_kernel(const __grid_constant__ Params p, int tokens) {
  // [tokens][4][U][2] (cos, sin): pairs 2j and 2j + 1 of neighbouring units side by side, so that lanes read other banks
  extern __shared__ float2 table[];
  griddep_wait();
  griddep_launch_dependents();
  const int half = p.R / 2, U = p.R / 16;
  const int t0 = blockIdx.x * tokens, nt = min(tokens, p.T - t0);
  // heads [h0, h1) of the tokens, where one token's heads are shared out over gridDim.y CTAs
  const int hper = (p.H + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * hper, h1 = min(p.H, h0 + hper);
  if (h0 >= h1) return;
  const int list = nt * (h1 - h0) * U;
  struct Where {
    int t, h, u;
  };
  const int su = 256 % U, sh = 256 / U % (h1 - h0), st = 256 / U / (h1 - h0);
  Where w;
  w.u = threadIdx.x % U;
  w.h = threadIdx.x / U % (h1 - h0);
  w.t = threadIdx.x / U / (h1 - h0);
  auto offset = [&](const Where& a) { return INTERLEAVED ? 16 * a.u : 8 * a.u; };
  const int next = INTERLEAVED ? 8 : half;          // elements from a unit's first vector to its second
  bool first = true;
  for (int i = threadIdx.x; i < list || first; i += 256) {
    uint4 v0, v1;
    if (i < list) {
      const uint16_t* x = p.x + (t0 + w.t) * p.xt + (h0 + w.h) * p.xh + offset(w);
      v0 = *reinterpret_cast<const uint4*>(x);
      v1 = *reinterpret_cast<const uint4*>(x + next);
    }
    if (first) {                                    // the angles, while the first loads are on their way
      first = false;
      for (int j = threadIdx.x; j < nt * half; j += 256) {
        const int t = j / half, f = j - t * half;
        table[t * half + (f / 2 % 4 * U + f / 8) * 2 + f % 2] = cos_sin(p.pos[t0 + t], p.freq[f], p.m, p.inverse != 0);
      }
      __syncthreads();
    }
    if (i >= list) break;
    const float4* cs = reinterpret_cast<const float4*>(table + w.t * half) + w.u;
    const uint32_t a[4] = {v0.x, v0.y, v0.z, v0.w}, b[4] = {v1.x, v1.y, v1.z, v1.w};
    uint32_t ya[4], yb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 c = cs[j * U];                   // pairs 2j and 2j + 1: (cos, sin) each
      if constexpr (INTERLEAVED) {
        const uint32_t q0 = j < 2 ? a[2 * j] : b[2 * j - 4], q1 = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
        const float x0 = bf16lo(q0), x1 = bf16hi(q0), x2 = bf16lo(q1), x3 = bf16hi(q1);
        const uint32_t r0 = pack_bf16x2(x0 * c.x - x1 * c.y, x1 * c.x + x0 * c.y);
        const uint32_t r1 = pack_bf16x2(x2 * c.z - x3 * c.w, x3 * c.z + x2 * c.w);
        if (j < 2) { ya[2 * j] = r0; ya[2 * j + 1] = r1; }
        else { yb[2 * j - 4] = r0; yb[2 * j - 3] = r1; }
      } else {
        const float x0 = bf16lo(a[j]), x2 = bf16hi(a[j]), x1 = bf16lo(b[j]), x3 = bf16hi(b[j]);
        ya[j] = pack_bf16x2(x0 * c.x - x1 * c.y, x2 * c.z - x3 * c.w);
        yb[j] = pack_bf16x2(x1 * c.x + x0 * c.y, x3 * c.z + x2 * c.w);
      }
    }
    uint16_t* y = p.y + (t0 + w.t) * p.yt + (h0 + w.h) * p.yh + offset(w);
    *reinterpret_cast<uint4*>(y) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
    *reinterpret_cast<uint4*>(y + next) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
    w.u += su;
    w.h += sh;
    w.t += st;
    if (w.u >= U) { w.u -= U; ++w.h; }
    if (w.h >= h1 - h0) { w.h -= h1 - h0; ++w.t; }
  }
  if (p.D > p.R && p.x != p.y) {                    // the rest of the heads: copied
    const int C = (p.D - p.R) / 8;
    for (int i = threadIdx.x; i < nt * (h1 - h0) * C; i += 256) {
      const int c = i % C, h = i / C % (h1 - h0), t = i / C / (h1 - h0);
      *reinterpret_cast<uint4*>(p.y + (t0 + t) * p.yt + (h0 + h) * p.yh + p.R + 8 * c) =
          *reinterpret_cast<const uint4*>(p.x + (t0 + t) * p.xt + (h0 + h) * p.xh + p.R + 8 * c);
    }
  }
}

}  // namespace rope
}  // namespace fp8q
