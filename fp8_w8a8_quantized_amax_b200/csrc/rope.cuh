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

__device__ __forceinline__ double half_turns(int64_t p, double f) {
  const double t = static_cast<double>(p) * (f * kTurnsPerRadian);
  return 2.0 * (t - rint(t));
}

__device__ __forceinline__ float2 cos_sin(int64_t p, double f, float m, bool inverse) {
  float s, c;
  sincospif(static_cast<float>(half_turns(p, f)), &s, &c);   // |half turns| <= 1: fp32 is off by 2^-25 of a turn
  return make_float2(c * m, inverse ? -s * m : s * m);
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

// One thread per pair of a (token, head), any strides; the dimensions behind
// the rotated part are copied by the same threads.
__global__ void __launch_bounds__(256) rope_kernel(Params p) {
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

}  // namespace rope
}  // namespace fp8q
