// kv4_attention.cuh -- attention over the paged 4-bit KV cache.
//
// For query row i of sequence b (n_b rows, the last n_b of its kv_len tokens):
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(sm_scale q.k_j - m),
// over the visible keys j: j < kv_len; causal: j <= pos, pos = kv_len - n_b + i;
// a window W: j > pos - W.  One pass: running maximum m and sum, rescaled when m grows.
#pragma once

#include "kv4.cuh"

namespace fp8q {
namespace kv4 {

struct AttnParams {
  Cache c;
  const uint16_t* q;
  uint16_t* o;
  float* lse;               // nullptr: not written
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* q_start;   // nullptr: one row per sequence
  int64_t qt, qh, ot, oh, table_stride;
  int T, B, Hq, group, max_pages, max_q;
  float scale;              // sm_scale * g_k
  int causal;
  int64_t window;           // 0: none
};

// The rows [r0, r0 + n) and cached tokens of sequence b, bounded to what the
// tensors hold (a length that has to be cut sets the error word).
struct Seq {
  int r0, n, kv;
};

__device__ __forceinline__ Seq sequence(const AttnParams& p, int b) {
  const int64_t r0 = p.q_start ? p.q_start[b] : b;
  const int64_t n = p.q_start ? p.q_start[b + 1] - r0 : 1;
  const int64_t kv = p.kv_len[b], most = static_cast<int64_t>(p.max_pages) * p.c.page_size;
  const int64_t r = min(max(r0, static_cast<int64_t>(0)), static_cast<int64_t>(p.T));
  Seq s;
  s.r0 = static_cast<int>(r);
  s.n = static_cast<int>(min(max(n, static_cast<int64_t>(0)), min(p.T - r, static_cast<int64_t>(p.max_q))));
  s.kv = static_cast<int>(min(max(kv, static_cast<int64_t>(0)), most));
  if (s.r0 != r0 || s.n != n || s.kv != kv) atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadLength));
  return s;
}

// Visible keys [first, last) of the row at position pos.
__device__ __forceinline__ void visible(const AttnParams& p, const Seq& s, int pos, int* first, int* last) {
  *last = p.causal ? min(s.kv, pos + 1) : s.kv;
  const int64_t f = p.window > 0 ? static_cast<int64_t>(pos) - p.window + 1 : 0;
  *first = f > 0 ? static_cast<int>(min(f, static_cast<int64_t>(0x7FFFFFFF))) : 0;
}

// One CTA per (row, query head), its four warps taking every fourth key; a
// lane holds D/32 dimensions.
template <int D>
__global__ void __launch_bounds__(128) attention_kernel(AttnParams p) {
  constexpr int E = D / 32;
  __shared__ float red_m[4], red_l[4], red_o[4][D];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = lane_id(), warp = threadIdx.x >> 5;
  const int h = blockIdx.x % p.Hq, kvh = h / p.group;
  const int row = blockIdx.x / p.Hq;
  // the sequence that holds this row
  int b = -1;
  Seq s = {0, 0, 0};
  for (int i = 0; i < p.B; ++i) {
    const Seq c = sequence(p, i);
    if (row >= c.r0 && row < c.r0 + c.n) {
      b = i;
      s = c;
    }
  }
  if (b < 0) return;                       // a row behind the last sequence
  int first, last;
  visible(p, s, s.kv - s.n + row - s.r0, &first, &last);
  float q[E], acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = bf16lo(p.q[row * p.qt + h * p.qh + lane * E + i]) * p.scale;
    acc[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = first + warp; j < last; j += 4) {
    const int page = p.table[b * p.table_stride + j / p.c.page_size];
    if (page < 0 || page >= p.c.pages) {
      atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadPage));
      continue;
    }
    const int r = j % p.c.page_size;
    float k[E], v[E];
    const int64_t at = p.c.code_offset(page, kvh, r) + lane * E / 2, sat = p.c.scale_offset(page, kvh, r) + lane * E / 16;
    const float ks = f16lo(widen_e4m3x2(p.c.k[sat])), vs = f16lo(widen_e4m3x2(p.c.v[sat]));
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const uint32_t kw = widen_e2m1x2(p.c.k[at + i / 2]), vw = widen_e2m1x2(p.c.v[at + i / 2]);
      k[i] = f16lo(kw) * ks;
      k[i + 1] = f16hi(kw) * ks;
      v[i] = f16lo(vw) * vs;
      v[i + 1] = f16hi(vw) * vs;
    }
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) x = fmaf(q[i], k[i], x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    const float mn = fmaxf(m, x), w = expf(x - mn), f = expf(m - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(w, v[i], acc[i] * f);
  }
  if (lane == 0) {
    red_m[warp] = m;
    red_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) red_o[warp][lane * E + i] = acc[i];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, red_m[w]);
  for (int w = 0; w < 4; ++w)
    if (red_l[w] > 0.0f) sum += red_l[w] * expf(red_m[w] - top);
  for (int d = threadIdx.x; d < D; d += 128) {
    float o = 0.0f;
    for (int w = 0; w < 4; ++w)
      if (red_l[w] > 0.0f) o += red_o[w][d] * expf(red_m[w] - top);
    p.o[row * p.ot + h * p.oh + d] = static_cast<uint16_t>(pack_bf16x2(sum > 0.0f ? o / sum * p.c.vg : 0.0f, 0.0f));
  }
  if (p.lse && threadIdx.x == 0) p.lse[static_cast<int64_t>(row) * p.Hq + h] = top + logf(sum);
}

}  // namespace kv4
}  // namespace fp8q
