// kv4_prefill.cuh -- attention of many new tokens over the paged 4-bit KV
// cache (prompts, parts of prompts): tcgen05 tensor cores.
//
// The formulas are those of kv4_attention.cuh.  Here one key meets hundreds of
// query rows (a group's heads times the new tokens), so the work is the two
// products, 4 D operations per row and key.
//   S [128 rows, 128 keys] = Q [128, D] . K^T     (both operands in shared memory)
//   O [128 rows, D]       += P [128, 128] . V     (P in tensor memory)
// A CTA works on 256 rows as two tiles, whose softmaxes take turns with the
// products: while the tensor cores work for one tile, its own threads (one per
// row, no exchange between lanes) turn the other's S into P.  The cache is read
// once per 256 rows and widened to f16 (exactly; E2M1 times E4M3) by four warps
// that write the 128-byte-swizzled operand tiles: K as a K-major operand, V,
// whose rows run along D, as an MN-major one, so both are written alike.
//
// Roles: warps 0-3 and 4-7 softmax of tile 0 and 1, warps 8-11 widening, warp 12
// issues the products.  Tensor memory (512 columns): S0, S1 (P over the first
// half of S), O0, O1.  The list of (256 rows, key head) items, each with its own
// run of 128-key steps, is cut evenly over the CTAs as in the kernel for few
// rows; parts of a cut item are joined by the last of its CTAs, in CTA order.
#pragma once

#include "kv4_attention.cuh"

namespace fp8q {
namespace kv4 {
namespace many {

constexpr int kRows = 256, kKeys = 128;
constexpr int kThreads = 13 * 32;
constexpr int kJobs = 32;

template <int D>
struct Layout {
  static constexpr int kTile = 128 * D * 2;                       // 128 rows of f16
  static constexpr int kV = 0, kK = 2 * kTile, kQ = 4 * kTile;    // two stages of V and K, Q of two tiles
  static constexpr int kJobOff = 6 * kTile;
  static constexpr int kBar = kJobOff + kJobs * 64;
  // at least half of an SM's shared memory, so that one CTA at a time holds its tensor memory
  static constexpr int kNeed = kBar + 512 + 1024;
  static constexpr int kBytes = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
  static constexpr int kPart = kRows * (D + 2);                   // floats of a partial result
  static_assert(kBytes <= 232448, "shared memory per CTA");
};

// 256 rows of a sequence, and the keys [first, hi) that some of them sees.
struct Unit {
  Seq s;
  int row0, rows, first, lo, hi, steps;
};

__device__ __forceinline__ Unit unit_of(const AttnParams& p, int u) {
  Unit x;
  const int b = u / p.row_tiles;
  x.row0 = (u - b * p.row_tiles) * kRows;
  x.s = sequence(p, b);
  x.rows = min(kRows, x.s.n * p.group - x.row0);
  x.first = x.lo = x.hi = 0;
  x.steps = 1;
  if (x.rows <= 0) {
    x.rows = x.steps = 0;
    return x;
  }
  const int base = x.s.kv - x.s.n;
  x.hi = visible_last(p, x.s, base + (x.row0 + x.rows - 1) / p.group);
  x.first = visible_first(p, base + x.row0 / p.group);
  x.lo = x.first & ~(kKeys - 1);
  x.steps = max(1, (x.hi - x.lo + kKeys - 1) / kKeys);
  return x;
}

struct Job {
  Unit x;
  int u, head, step, steps;
  int64_t s;
};
static_assert(sizeof(Job) <= 64, "the layout's job list");

// Column c of the softmax's view: keys outside [first, last) of the row count as minus infinity.
template <bool MASK>
__device__ __forceinline__ float masked(uint32_t v, int c, int first, int last) {
  const float f = __uint_as_float(v);
  return !MASK || (c >= first && c < last) ? f : -INFINITY;
}

template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t taddr, int first, int last) {
  float top = -INFINITY;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + 32 * c, r);
    tmem_ld_wait_regs(r);
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      top = fmaxf(top, fmaxf(masked<MASK>(r[i], 32 * c + i, first, last), masked<MASK>(r[i + 1], 32 * c + i + 1, first, last)));
  }
  return top;
}

template <bool MASK>
__device__ __forceinline__ float row_exp(uint32_t taddr, int first, int last, float qscale, float nbase) {
  const uint64_t scale2 = f32x2_pack(qscale, qscale), base2 = f32x2_pack(nbase, nbase);
  uint64_t sum2 = f32x2_pack(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32], w[16];
    tmem_ld_32x32b_x32(taddr + 32 * c, r);
    tmem_ld_wait_regs(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = masked<MASK>(r[2 * i], 32 * c + 2 * i, first, last);
      float y = masked<MASK>(r[2 * i + 1], 32 * c + 2 * i + 1, first, last);
      f32x2_unpack(fma_f32x2(f32x2_pack(x, y), scale2, base2), x, y);
      x = ex2(x);
      y = ex2(y);
      sum2 = add_f32x2(sum2, f32x2_pack(x, y));
      w[i] = pack_f16x2(x, y);
    }
    tmem_st_32x32b_x16(taddr + 16 * c, w);          // over columns that have been read
  }
  float a, b;
  f32x2_unpack(sum2, a, b);
  return a + b;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<D>;
  constexpr int kHalf = 128 * 128;                  // bytes of a tile's 64-element half
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Job* jobs = reinterpret_cast<Job*>(smem + L::kJobOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t *q_full = bars, *s_full = bars + 2, *p_full = bars + 4, *o_full = bars + 6;
  uint64_t *k_full = bars + 8, *k_empty = bars + 10, *v_full = bars + 12, *v_empty = bars + 14, *drain = bars + 16, *join = bars + 17;
  int64_t* misc = reinterpret_cast<int64_t*>(smem + L::kBar + 160);     // 13 warps' sums, the first job's unit and place
  int* flags = reinterpret_cast<int*>(smem + L::kBar + 160 + 16 * 8);
  volatile int* abort = flags;
  int* njobs = flags + 1;
  int* last_one = flags + 2;                        // two
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(flags + 4);
  const int warp = threadIdx.x >> 5, lane = lane_id();

  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
      mbar_init(&join[i], 128);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's range of the list: a scan over the (sequence, row tile) units ----
  const int units = p.B * p.row_tiles;
  int64_t total = 0, before = 0, mine = 0;
  auto scan = [&](int base) {
    const int u = base + static_cast<int>(threadIdx.x);
    mine = u < units ? static_cast<int64_t>(unit_of(p, u).steps) * p.c.heads : 0;
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t w = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += w;
    }
    __syncthreads();
    if (lane == 31) misc[warp] = v;
    __syncthreads();
    int64_t ahead = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) ahead += misc[w];
      all += misc[w];
    }
    before = ahead + v - mine;
    return all;
  };
  for (int base = 0; base < units; base += kThreads) total += scan(base);
  Range range;
  range.q = total / gridDim.x;
  range.r = total - range.q * gridDim.x;
  const int64_t begin = range.begin(blockIdx.x), end = range.begin(blockIdx.x + 1);
  if (begin == end) return;
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  {
    int64_t ahead = 0;
    for (int base = 0; base < units; base += kThreads) {
      const int64_t all = units <= kThreads ? total : scan(base);
      if (begin >= ahead && begin < ahead + all) {
        const int64_t at = begin - ahead - before;
        if (at >= 0 && at < mine) {
          misc[14] = base + static_cast<int>(threadIdx.x);
          misc[15] = at;
        }
        break;
      }
      ahead += all;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // counts of what a role has waited for, over all jobs
  int tiles = 0;                 // key tiles (widening warps, product warp)
  int turns = 0, done = 0;       // softmax: S tiles, items; product warp: the first tile's
  int meets = 0;                 // softmax: meetings of a tile's threads
  int turns1 = 0, done1 = 0;     // product warp: the second tile's
  int64_t next_s = begin;
  for (;;) {
    // ---- the next jobs of this CTA ----
    if (threadIdx.x == 0) {
      int n = 0;
      int u, head, step;
      if (next_s == begin) {
        u = static_cast<int>(misc[14]);
        const int steps = unit_of(p, u).steps;
        head = static_cast<int>(misc[15] / steps);
        step = static_cast<int>(misc[15] - static_cast<int64_t>(head) * steps);
      } else {
        u = jobs[kJobs - 1].u;
        head = jobs[kJobs - 1].head + 1;             // a job that is not the last one ends its item
        step = 0;
      }
      Unit x = unit_of(p, u);
      int64_t s = next_s;
      while (n < kJobs && s < end) {
        while ((head >= p.c.heads || x.rows == 0) && u + 1 < units) {
          head = 0;
          x = unit_of(p, ++u);
        }
        Job& j = jobs[n++];
        j.x = x;
        j.u = u;
        j.head = head++;
        j.step = step;
        j.steps = static_cast<int>(min(static_cast<int64_t>(x.steps - step), end - s));
        j.s = s;
        s += j.steps;
        step = 0;
      }
      *njobs = n;
    }
    __syncthreads();
    const int n = *njobs;

    if (warp == 12) {
      // ---------------------------------------------------------- products ---
      constexpr uint32_t kIdescS = idesc_f16_f32(128, kKeys, false), kIdescO = idesc_f16_f32(128, D, true);
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int steps = jobs[i].steps, two = jobs[i].x.rows > 128 ? 2 : 1;
        auto score = [&](int w, int tile) {          // S_w = Q_w . K_tile^T
          const uint32_t a = smem_u32(smem + L::kQ + w * L::kTile), b = smem_u32(smem + L::kK + (tile & 1) * L::kTile);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_f16_ss(tmem + w * 128, umma_desc_sw128(a + k / 4 * kHalf + k % 4 * 32),
                       umma_desc_sw128(b + k / 4 * kHalf + k % 4 * 32), kIdescS, k > 0);
            mma_commit(&s_full[w]);
            if (w == two - 1) mma_commit(&k_empty[tile & 1]);
          }
          __syncwarp();
        };
        for (int w = 0; w < two && ok; ++w) {
          ok = mbar_wait(&q_full[w], (w ? done1 : done) & 1, abort, kErrWaitFull);
          if (ok && w == 0) ok = mbar_wait(&k_full[tiles & 1], (tiles >> 1) & 1, abort, kErrWaitFull);
          if (!ok) break;
          tc_fence_after();
          score(w, tiles);
        }
        for (int j = 0; j < steps && ok; ++j) {
          const int tile = tiles + j;
          ok = mbar_wait(&v_full[tile & 1], (tile >> 1) & 1, abort, kErrWaitFull);
          for (int w = 0; w < two && ok; ++w) {
            ok = mbar_wait(&p_full[w], (w ? turns1 : turns) & 1, abort, kErrWaitTmemFull);
            if (!ok) break;
            if (w) ++turns1; else ++turns;
            tc_fence_after();
            const uint32_t v = smem_u32(smem + L::kV + (tile & 1) * L::kTile);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                mma_f16_ts(tmem + 256 + w * 128, tmem + w * 128 + k * 8, umma_desc_mn_sw128(v + k * 2048, kHalf), kIdescO,
                           j > 0 || k > 0);
              if (j + 1 == steps) mma_commit(&o_full[w]);
              if (w == two - 1) mma_commit(&v_empty[tile & 1]);
            }
            __syncwarp();
            if (j + 1 < steps) {
              if (w == 0) {
                ok = mbar_wait(&k_full[(tile + 1) & 1], ((tile + 1) >> 1) & 1, abort, kErrWaitFull);
                if (!ok) break;
                tc_fence_after();
              }
              score(w, tile + 1);
            }
          }
        }
        tiles += steps;
        ++done;
        if (two == 2) ++done1;
      }
    } else if (warp >= 8) {
      // ---------------------------------------------------------- widening ---
      // One thread per key; the next tile's bytes are on their way while this one's are widened.
      const int r = threadIdx.x - 256;
      uint4 raw[2][D / 32];
      uint2 sc[2];
      auto fetch = [&](const Job& j, int step, int which) {
        const int key = j.x.lo + (j.step + step) * kKeys + r;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[which][i] = make_uint4(0, 0, 0, 0);
        sc[which] = make_uint2(0, 0);
        if (key < j.x.hi && key >= j.x.first) {
          const int page = p.table[j.u / p.row_tiles * p.table_stride + (key >> p.c.page_shift)];
          if (page < 0 || page >= p.c.pages) {
            atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadPage));
            return;
          }
          const uint8_t* base = which ? p.c.v : p.c.k;
          const int row = key & (p.c.page_size - 1);
          const uint4* src = reinterpret_cast<const uint4*>(base + p.c.code_offset(page, j.head, row));
#pragma unroll
          for (int i = 0; i < D / 32; ++i) raw[which][i] = src[i];
          const uint8_t* ss = base + p.c.scale_offset(page, j.head, row);
          if constexpr (D == 128) sc[which] = *reinterpret_cast<const uint2*>(ss);
          else sc[which].x = *reinterpret_cast<const uint32_t*>(ss);
        }
      };
      auto widen = [&](int which, uint8_t* dst) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {           // 32 elements: two scales, four 16-byte chunks
          const uint32_t two = widen_e4m3x2((i < 2 ? sc[which].x : sc[which].y) >> (i % 2 * 16));
          const uint32_t s0 = __byte_perm(two, two, 0x1010), s1 = __byte_perm(two, two, 0x3232);
          const uint32_t w[4] = {raw[which][i].x, raw[which][i].y, raw[which][i].z, raw[which][i].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t e[4];
            widen4(w[c], e);
            const uint32_t s = c < 2 ? s0 : s1;
            const int chunk = 4 * (i % 2) + c;
            *reinterpret_cast<uint4*>(dst + i / 2 * kHalf + r * 128 + ((chunk ^ (r & 7)) << 4)) =
                make_uint4(mul_f16x2(e[0], s), mul_f16x2(e[1], s), mul_f16x2(e[2], s), mul_f16x2(e[3], s));
          }
        }
        fence_proxy_async_smem();
      };
      bool ok = true;
      if (n > 0) {
        fetch(jobs[0], 0, 0);
        fetch(jobs[0], 0, 1);
      }
      for (int i = 0; i < n && ok; ++i) {
        const int steps = jobs[i].steps;
        for (int j = 0; j < steps && ok; ++j, ++tiles) {
          const bool more = j + 1 < steps || i + 1 < n;
          const Job& nj = jobs[j + 1 < steps ? i : i + 1];
          const int ns = j + 1 < steps ? j + 1 : 0;
          const int st = tiles & 1, ph = ((tiles >> 1) & 1) ^ 1;
          ok = mbar_wait(&k_empty[st], ph, abort, kErrWaitEmpty);
          if (!ok) break;
          widen(0, smem + L::kK + st * L::kTile);
          mbar_arrive(&k_full[st]);
          if (more) fetch(nj, ns, 0);
          ok = mbar_wait(&v_empty[st], ph, abort, kErrWaitEmpty);
          if (!ok) break;
          widen(1, smem + L::kV + st * L::kTile);
          mbar_arrive(&v_full[st]);
          if (more) fetch(nj, ns, 1);
        }
      }
    } else {
      // ----------------------------------------------------------- softmax ---
      const int w = warp >> 2, r = threadIdx.x & 127;
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // 32 lanes a warp
      const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + 256 + w * 128;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const Job& job = jobs[i];
        const Unit x = job.x;
        if (w * 128 >= x.rows) continue;
        const int row = x.row0 + w * 128 + r;
        const bool real = w * 128 + r < x.rows;
        const int token = min(row, x.row0 + x.rows - 1) / p.group, pos = x.s.kv - x.s.n + token;
        const int h = job.head * p.group + row - row / p.group * p.group;
        // ---- the query row: scaled to f16, into the swizzled operand tile ----
        float qscale;
        {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (x.s.r0 + static_cast<int64_t>(token)) * p.qt + h * p.qh);
          uint8_t* dst = smem + L::kQ + w * L::kTile + r * 128;
          float amax = 0.0f;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = real ? src[c] : make_uint4(0, 0, 0, 0);
            amax = fmaxf(amax, fmaxf(fmaxf(fmaxf(fabsf(bf16lo(v.x)), fabsf(bf16hi(v.x))), fmaxf(fabsf(bf16lo(v.y)), fabsf(bf16hi(v.y)))),
                                     fmaxf(fmaxf(fabsf(bf16lo(v.z)), fabsf(bf16hi(v.z))), fmaxf(fabsf(bf16lo(v.w)), fabsf(bf16hi(v.w))))));
          }
          const int k = row_exponent(amax);
          const float up = pow2(k);
          qscale = fmaxf(pow2(-k) * p.scale, kLeastScale);
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) {
            const uint4 v = real ? src[c] : make_uint4(0, 0, 0, 0);
            const uint4 f = make_uint4(pack_f16x2(bf16lo(v.x) * up, bf16hi(v.x) * up), pack_f16x2(bf16lo(v.y) * up, bf16hi(v.y) * up),
                                       pack_f16x2(bf16lo(v.z) * up, bf16hi(v.z) * up), pack_f16x2(bf16lo(v.w) * up, bf16hi(v.w) * up));
            *reinterpret_cast<uint4*>(dst + c / 8 * kHalf + (((c & 7) ^ (r & 7)) << 4)) = f;
          }
          fence_proxy_async_smem();
          mbar_arrive(&q_full[w]);
        }
        const int vfirst = visible_first(p, pos), vlast = visible_last(p, x.s, pos);
        float nbase = 0.0f, limit = -INFINITY, sum = 0.0f;
        int key = x.lo + job.step * kKeys;
        for (int j = 0; j < job.steps; ++j, key += kKeys, ++turns) {
          ok = mbar_wait(&s_full[w], turns & 1, abort, kErrWaitTmemFull);
          if (!ok) break;
          tc_fence_after();
          const int first = vfirst - key, last = vlast - key;
          const bool whole = __all_sync(0xFFFFFFFFu, first <= 0 && last >= kKeys);
          const float top = whole ? row_max<false>(ts, 0, 0) : row_max<true>(ts, first, last);
          if (__any_sync(0xFFFFFFFFu, top > limit)) {
            const float was = limit == -INFINITY ? -INFINITY : -nbase, now = fmaxf(was, top * qscale);
            float f = 1.0f;
            if (now > was) {
              f = ex2(was - now);                    // 0 from -infinity
              nbase = -now;
              limit = (now + kSlack) / qscale;
              sum *= f;
            }
            if (j > 0) {                             // S of this step was issued after O's last product: O is at rest
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(to + 32 * c, o);
                tmem_ld_wait_regs(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st_32x32b_x32(to + 32 * c, o);
              }
            }
          }
          sum += whole ? row_exp<false>(ts, 0, 0, qscale, nbase) : row_exp<true>(ts, first, last, qscale, nbase);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[w]);
        }
        if (!ok) break;
        ok = mbar_wait(&o_full[w], done & 1, abort, kErrWaitTmemFull);
        if (!ok) break;
        ++done;
        tc_fence_after();
        // ---- the item's end ----
        const int64_t i0 = job.s - job.step, i1 = i0 + x.steps;
        const float top = limit == -INFINITY ? -INFINITY : -nbase;
        const int64_t out_token = x.s.r0 + static_cast<int64_t>(token);
        uint16_t* out = p.o + out_token * p.ot + h * p.oh;
        if (i0 >= begin && i1 <= end) {
          const float f = sum > 0.0f ? p.c.vg / sum : 0.0f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_ld_wait_regs(o);
            if (real) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 v;
                v.x = pack_bf16x2(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f);
                v.y = pack_bf16x2(__uint_as_float(o[e + 2]) * f, __uint_as_float(o[e + 3]) * f);
                v.z = pack_bf16x2(__uint_as_float(o[e + 4]) * f, __uint_as_float(o[e + 5]) * f);
                v.w = pack_bf16x2(__uint_as_float(o[e + 6]) * f, __uint_as_float(o[e + 7]) * f);
                *reinterpret_cast<uint4*>(out + 32 * c + e) = v;
              }
            }
          }
          if (p.lse && real) p.lse[out_token * p.Hq + h] = sum > 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
          tc_fence_before();
        } else {
          // a part: [D / 4][256] float4 (coalesced over the rows), the bases, the sums
          const int row_in = w * 128 + r;
          float* slot = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (job.s == begin ? 0 : 1)) * L::kPart;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_ld_wait_regs(o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              __stcg(reinterpret_cast<float4*>(slot) + (8 * c + e) * kRows + row_in,
                     make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                 __uint_as_float(o[4 * e + 3])));
          }
          tc_fence_before();
          __stcg(slot + kRows * D + row_in, top);
          __stcg(slot + kRows * (D + 1) + row_in, sum);
          const int c0 = range.owner(i0), parts = range.owner(i1 - 1) - c0 + 1;
          // a tile's 128 threads meet at an mbarrier: its wait is bounded, so that none waits for one that gave up
          auto meet = [&]() {
            mbar_arrive(&join[w]);
            return mbar_wait(&join[w], meets++ & 1, abort, kErrWaitEmpty);
          };
          __threadfence();
          if (!(ok = meet())) break;
          if (r == 0) last_one[w] = atom_add_acq_rel_gpu(p.count + 2 * c0 + w, 1u) == static_cast<unsigned>(parts - 1);
          if (!(ok = meet())) break;
          if (last_one[w]) {
            __threadfence();
            const float* at0 = p.part + (2 * static_cast<int64_t>(c0) + (range.begin(c0) != i0 ? 1 : 0)) * L::kPart;
            const float* at1 = p.part + 2 * (static_cast<int64_t>(c0) + 1) * L::kPart;     // the others', 2 kPart apart
            auto part = [&](int c) { return c == 0 ? at0 : at1 + 2 * static_cast<int64_t>(c - 1) * L::kPart; };
            float m = -INFINITY, l = 0.0f;
            for (int c = 0; c < parts; ++c) m = fmaxf(m, __ldcg(part(c) + kRows * D + row_in));
            for (int c = 0; c < parts; ++c) {
              const float mc = __ldcg(part(c) + kRows * D + row_in);
              if (mc != -INFINITY) l += __ldcg(part(c) + kRows * (D + 1) + row_in) * ex2(mc - m);
            }
            const float f = l > 0.0f ? p.c.vg / l : 0.0f;
            for (int e = 0; e < D / 8; ++e) {
              float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
              for (int c = 0; c < parts; ++c) {
                const float mc = __ldcg(part(c) + kRows * D + row_in), g = mc == -INFINITY ? 0.0f : ex2(mc - m);
                const float4 u = __ldcg(reinterpret_cast<const float4*>(part(c)) + 2 * e * kRows + row_in);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(part(c)) + (2 * e + 1) * kRows + row_in);
                a.x += u.x * g; a.y += u.y * g; a.z += u.z * g; a.w += u.w * g;
                b.x += v.x * g; b.y += v.y * g; b.z += v.z * g; b.w += v.w * g;
              }
              if (real)
                *reinterpret_cast<uint4*>(out + 8 * e) = make_uint4(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f),
                                                                    pack_bf16x2(b.x * f, b.y * f), pack_bf16x2(b.z * f, b.w * f));
            }
            if (p.lse && real) p.lse[out_token * p.Hq + h] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
            if (r == 0) p.count[2 * c0 + w] = 0;
          }
          if (!(ok = meet())) break;                 // last_one is free again
        }
      }
    }
    __syncwarp();
    next_s = jobs[n - 1].s + jobs[n - 1].steps;
    __syncthreads();
    if (next_s >= end || *abort) break;
  }
  // After a wait that ran out, what the tensor cores still work on ends before their memory is given back.
  if (*abort && warp == 12) {
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mbar_wait_drain(drain, 0, kErrWaitDrain);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace many
}  // namespace kv4
}  // namespace fp8q
