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
// issues the products.  A softmax warp brings its 32 rows' queries of the next
// item as soon as the last S of the item before is done, ahead of that item's
// end.  Tensor memory (512 columns): S0, S1 (P over the first half of S), O0,
// O1.  The list of (256 rows, key head) items, each with its own run of 128-key
// steps, is cut over the CTAs as in the kernel for few rows, or each item by
// itself; its parts are joined by the last of its CTAs, in CTA order.
//
// Measured: 2048 new tokens of 32 heads behind 6144 cached ones (8 key heads, D =
// 128): 262 to 267 us a call on new inputs, 0.92 PFLOP/s of the visible products
// (0.56 of what a library product reaches); 245 us for launches back to back.  A
// step of 256 rows takes 3.9 K cycles where its products take 2.05 K: a tile's
// chain S, maximum, exponentials, P . V is longer than the other tile's share of
// the tensor cores, and a row's two passes over tensor memory by one thread are
// its longest link.  13 warps compiled together leave 128 registers a thread: at D
// = 128 the roles spill (128 bytes stored, 496 loaded), at D = 64 hardly (8, 40).
// Sixteen softmax warps (one pass, S held in registers) spilled and were slower;
// eight with registers moved to them have not been tried.
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
  static constexpr int kScaleOff = kJobOff + kJobs * 64;          // fp32 [256]: the rows' score factors
  static constexpr int kBar = kScaleOff + kRows * 4;
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

// The lists of steps count kOver steps more in front of every item, as in the
// kernel for few rows: here an item's pipeline fills and its sums are written.
constexpr int kOver = 2;

// A part joined costs about 3 us (the parts of an item are read by its last CTA alone), a step 2 us once the pipeline
// is full: where there are few steps a CTA takes at least kLeast of them (256 rows of 8 heads over 2000 keys: 54 -> 35
// us; with 2 or 6, 40).  And where there are no more items than CTAs, each is cut by itself, into equal parts, unless
// that takes kJoinCost steps longer than an even share of the list, which gives most CTAs the ends of two items (256
// rows over 500 keys: 27 -> 22 us, over 8000: 88 -> 63; 2000 rows over 2000: 53 -> 42; at 0 the list again).
constexpr int kLeast = 4, kJoinCost = 6;

struct Job {
  Unit x;
  int u, head, step, steps;
  int64_t s;
};
static_assert(sizeof(Job) <= 64, "the layout's job list");

__device__ __forceinline__ void make_job(const Unit& x, int u, int head, int step, int64_t s, int64_t end, Job* j) {
  j->x = x;
  j->u = u;
  j->head = head;
  j->step = step;
  j->steps = static_cast<int>(min(static_cast<int64_t>(x.steps - step), end - s));
  j->s = s;
}

// Keys outside [first, last) of a row of S become minus infinity (the first and last tiles of an item only, so apart:
// the two passes below are then compiled once).
__device__ __forceinline__ void row_mask(uint32_t ts, int first, int last) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(ts + 32 * c, r);
    tmem_ld_wait_regs(r);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (32 * c + i < first || 32 * c + i >= last) r[i] = 0xFF800000u;
    tmem_st_32x32b_x32(ts + 32 * c, r);
  }
  tmem_st_wait();
}

// Both passes over a row of S work on 32 columns while the next 32 are on their way from tensor memory.
__device__ __forceinline__ float row_max(uint32_t ts) {
  float top[2] = {-INFINITY, -INFINITY};
  uint32_t r[2][32];
  tmem_ld_32x32b_x32(ts, r[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld_wait_regs(r[c & 1]);
    if (c < 3) tmem_ld_32x32b_x32(ts + 32 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      top[i / 2 & 1] = fmaxf(top[i / 2 & 1], fmaxf(__uint_as_float(r[c & 1][i]), __uint_as_float(r[c & 1][i + 1])));
  }
  return fmaxf(top[0], top[1]);
}

// 2^z for two values on the FMA pipes: z = n + r, |r| <= 1/2, a polynomial of degree 5 in r (least maximal relative error,
// 2^-22; fitted on a grid by repeated weighted least squares), and n added to the exponent.  z is held at -126 from
// below, so minus infinity becomes 2^-126, an f16 zero.
__device__ __forceinline__ void exp2_poly(uint64_t z2, float& x, float& y) {
  f32x2_unpack(z2, x, y);
  const uint64_t z = f32x2_pack(fmaxf(x, -126.0f), fmaxf(y, -126.0f));
  const uint64_t magic = f32x2_pack(12582912.0f, 12582912.0f), minus = f32x2_pack(-12582912.0f, -12582912.0f);
  const uint64_t t = add_f32x2(z, magic);            // 1.5 2^23 + n: n in the low bits
  const uint64_t n = add_f32x2(t, minus);
  const uint64_t r = fma_f32x2(n, f32x2_pack(-1.0f, -1.0f), z);
  uint64_t q = f32x2_pack(0.001327647129073739f, 0.001327647129073739f);
  q = fma_f32x2(q, r, f32x2_pack(0.009675540961325169f, 0.009675540961325169f));
  q = fma_f32x2(q, r, f32x2_pack(0.05550713092088699f, 0.05550713092088699f));
  q = fma_f32x2(q, r, f32x2_pack(0.24022120237350464f, 0.24022120237350464f));
  q = fma_f32x2(q, r, f32x2_pack(0.6931469440460205f, 0.6931469440460205f));
  q = fma_f32x2(q, r, f32x2_pack(1.0000001192092896f, 1.0000001192092896f));
  float qx, qy, tx, ty;
  f32x2_unpack(q, qx, qy);
  f32x2_unpack(t, tx, ty);
  x = __uint_as_float(__float_as_uint(tx) * 8388608u + __float_as_uint(qx));
  y = __uint_as_float(__float_as_uint(ty) * 8388608u + __float_as_uint(qy));
}

// One pair in kPoly is raised on the FMA pipes, the others by the function unit, which by itself would take half the
// softmax's time.
constexpr int kPoly = 6;

// P = 2^(S qscale + nbase) in f16 over S; returns the sum.
__device__ __forceinline__ float row_exp(uint32_t ts, float qscale, float nbase) {
  const uint64_t scale2 = f32x2_pack(qscale, qscale), base2 = f32x2_pack(nbase, nbase);
  uint64_t sum2[2] = {f32x2_pack(0.0f, 0.0f), f32x2_pack(0.0f, 0.0f)};
  uint32_t r[2][32];
  tmem_ld_32x32b_x32(ts, r[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld_wait_regs(r[c & 1]);
    if (c < 3) tmem_ld_32x32b_x32(ts + 32 * (c + 1), r[(c + 1) & 1]);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = __uint_as_float(r[c & 1][2 * i]), y = __uint_as_float(r[c & 1][2 * i + 1]);
      const uint64_t z = fma_f32x2(f32x2_pack(x, y), scale2, base2);
      if (i % kPoly == kPoly - 1) {
        exp2_poly(z, x, y);
      } else {
        f32x2_unpack(z, x, y);
        x = ex2(x);
        y = ex2(y);
      }
      sum2[i & 1] = add_f32x2(sum2[i & 1], f32x2_pack(x, y));
      w[i] = pack_f16x2(x, y);
    }
    tmem_st_32x32b_x16(ts + 16 * c, w);             // over columns that have been read
  }
  float a, b;
  f32x2_unpack(add_f32x2(sum2[0], sum2[1]), a, b);
  return a + b;
}

// A warp's arrival: one for all its lanes (128 arrivals on one barrier are taken one by one).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
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
  uint64_t *k_full = bars + 8, *k_empty = bars + 10, *v_full = bars + 12, *v_empty = bars + 14, *drain = bars + 16;
  int64_t* misc = reinterpret_cast<int64_t*>(smem + L::kBar + 176);     // the warps' sums
  int* flags = reinterpret_cast<int*>(smem + L::kBar + 176 + 19 * 8);
  volatile int* abort = flags;
  int* njobs = flags + 1;
  int* longest_of = flags + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(flags + 4);
  float* qscales = reinterpret_cast<float*>(smem + L::kScaleOff);
  const int warp = threadIdx.x >> 5, lane = lane_id();

  if (threadIdx.x == 0) {
    *abort = 0;
    *longest_of = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's range of the list: a scan over the (sequence, row tile) units ----
  const int units = p.B * p.row_tiles;
  // (steps in the low 40 bits, items above: both are bounded by the host)
  int64_t total = 0, before = 0, mine = 0;
  int longest = 0;
  auto scan = [&](int base) {
    const int u = base + static_cast<int>(threadIdx.x);
    mine = 0;
    if (u < units) {
      const int steps = unit_of(p, u).steps;
      if (steps > 0) mine = (steps + kOver + kOneItem) * p.c.heads;
      longest = max(longest, steps);
    }
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
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  if (lane == 0) atomicMax(longest_of, longest);
  __syncthreads();
  longest = *longest_of;
  const int items = static_cast<int>(total >> 40);
  const int64_t everything = total;
  total &= kOneItem - 1;
  const int ctas = static_cast<int>(max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), total / kLeast)));
  Range range;
  range.q = quotient(total, ctas);
  range.r = total - range.q * ctas;
  // Where there are no more items than CTAs each may be left to `each` CTAs of its own, in parts of equal steps.
  const int each = items > 0 ? max(1, min(static_cast<int>(gridDim.x) / items, longest / kLeast)) : 1;
  const bool apart = items <= static_cast<int>(gridDim.x) && (longest + each - 1) / each + kOver <= range.q + kJoinCost;
  if (static_cast<int>(blockIdx.x) >= (apart ? items * each : ctas)) return;
  const int64_t begin = apart ? static_cast<int64_t>(blockIdx.x) / each : range.begin(blockIdx.x);
  const int64_t end = apart ? begin + 1 : range.begin(blockIdx.x + 1);
  if (begin == end) return;
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  {
    int64_t ahead = 0;
    for (int base = 0; base < units; base += kThreads) {
      const int64_t all = units <= kThreads ? everything : scan(base), all_w = apart ? all >> 40 : all & (kOneItem - 1);
      if (begin >= ahead && begin < ahead + all_w) {
        const int64_t at = begin - ahead - (apart ? before >> 40 : before & (kOneItem - 1));
        if (at >= 0 && at < (apart ? mine >> 40 : mine & (kOneItem - 1))) {      // the first job is this thread's
          const int u = base + static_cast<int>(threadIdx.x);
          const Unit x = unit_of(p, u);
          if (apart) {
            const int parts = min(each, x.steps), k = min(static_cast<int>(blockIdx.x) % each, parts);
            const int s0 = static_cast<int>(static_cast<int64_t>(x.steps) * k / parts);
            const int s1 = static_cast<int>(static_cast<int64_t>(x.steps) * min(k + 1, parts) / parts);
            make_job(x, u, static_cast<int>(at), s0, s0, s1, jobs);
            misc[18] = s1;
          } else {
            const int steps = x.steps + kOver, head = static_cast<int>(quotient(at, steps));
            const int off = static_cast<int>(at - static_cast<int64_t>(head) * steps);
            make_job(x, u, head, max(0, off - kOver), begin + max(0, kOver - off), end, jobs);
            misc[18] = end;
          }
        }
        break;
      }
      ahead += all_w;
    }
  }
  if (threadIdx.x == 0) {
    misc[16] = apart ? -1 : range.q;
    misc[17] = apart ? each : range.r;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool none = jobs[0].steps <= 0;              // the range lies ahead of an item's first step
  // What a role needs between items only is read back from shared memory there, not held in registers.
  const volatile int64_t* kept = misc;               // range.q and range.r (or -1 and `each`), this CTA's end
  auto range_end = [&]() { return kept[18]; };

  // counts of what a role has waited for, over all jobs
  int tiles = 0;                 // key tiles (widening warps, product warp)
  int turns = 0, done = 0;       // softmax: S tiles, items; product warp: the first tile's
  int turns1 = 0, done1 = 0;     // product warp: the second tile's
  // The jobs of a CTA are listed kJobs at a time.  The first of a list stands before the roles begin with it; the
  // others are listed meanwhile by the product warp.  Every role walks through the list by itself.
  auto meet_all = []() {
    __syncwarp();
    asm volatile("bar.sync 0;" ::: "memory");
  };
  // the job after `j`, if the range reaches it (j then ends its item)
  auto job_after = [&](const Job& j, Job* to) {
    Unit x = j.x;
    int u = j.u, head = j.head + 1;
    const int64_t s = j.s + j.steps + kOver, end = range_end();
    if (s >= end) return false;
    while ((head >= p.c.heads || x.rows == 0) && u + 1 < units) {
      head = 0;
      x = unit_of(p, ++u);
    }
    make_job(x, u, head, 0, s, end, to);
    return true;
  };
  auto list_jobs = [&]() {                           // one thread, after jobs[0]
    int n = 1;
    while (n < kJobs && job_after(jobs[n - 1], &jobs[n])) ++n;
    *njobs = n;
  };
  auto list_done = [&](int n) {                     // every role is through the list: whether there is no other
    meet_all();
    const Job last = jobs[n - 1];
    const bool over = last.s + last.steps + kOver >= range_end() || *abort;
    if (over) return true;
    meet_all();
    if (threadIdx.x == 12 * 32) job_after(last, &jobs[0]);
    meet_all();
    return false;
  };
  if (none) {
  } else if (warp < 8) {
    for (;;) {
      // ----------------------------------------------------------- softmax ---
      const int w = warp >> 2, r = threadIdx.x & 127;
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;       // 32 lanes a warp
      const uint32_t ts = tmem + lanes + w * 128, to = tmem + lanes + 256 + w * 128;
      // This warp's 32 rows of an item's queries: a row by D / 8 lanes, 16 bytes each, all on their way at once; scaled
      // to f16, into the swizzled operand tile.
      auto bring_queries = [&](const Job& job) {
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const int c = lane % kLanes, first = (warp & 3) * 32 + lane / kLanes;
        uint4 v[kLanes];
        const int row = job.x.row0 + w * 128 + first, dt = kAtOnce / p.group, dh = kAtOnce - dt * p.group;
        int t = row / p.group, h = row - t * p.group;
        const uint16_t* src = p.q + static_cast<int64_t>(job.x.s.r0) * p.qt + static_cast<int64_t>(job.head) * p.group * p.qh + 8 * c;
#pragma unroll
        for (int u = 0; u < kLanes; ++u) {
          v[u] = make_uint4(0, 0, 0, 0);
          if (w * 128 + first + u * kAtOnce < job.x.rows) v[u] = *reinterpret_cast<const uint4*>(src + t * p.qt + h * p.qh);
          t += dt;
          h += dh;
          if (h >= p.group) {
            h -= p.group;
            ++t;
          }
        }
#pragma unroll
        for (int u = 0; u < kLanes; ++u) {
          const int r = first + u * kAtOnce;
          const uint32_t a[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          float amax = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16lo(a[e])), fabsf(bf16hi(a[e]))));
#pragma unroll
          for (int o = 1; o < kLanes; o *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          const int k = row_exponent(amax);
          const float up = pow2(k);
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = pack_f16x2(bf16lo(a[e]) * up, bf16hi(a[e]) * up);
          *reinterpret_cast<uint4*>(smem + L::kQ + w * L::kTile + c / 8 * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
          if (c == 0) qscales[w * 128 + r] = fmaxf(pow2(-k) * p.scale, kLeastScale);
        }
        fence_proxy_async_smem();
        warp_arrive(&q_full[w]);
      };
      const bool first_mine = w * 128 < jobs[0].x.rows;
      if (first_mine) bring_queries(jobs[0]);
      meet_all();
      const int n = *njobs;
      auto next_job = [&](int i) {                 // the next item with rows of this tile
        while (i < n && w * 128 >= jobs[i].x.rows) ++i;
        return i;
      };
      bool ok = true;
      int i = next_job(0);
      if (!first_mine && i < n) bring_queries(jobs[i]);
      for (int following; i < n && ok; i = following) {
        const volatile Job& job = jobs[i];
        following = next_job(i + 1);
        const float qscale = qscales[w * 128 + r];   // (written by this warp)
        const bool idle = w * 128 + (r & ~31) >= job.x.rows;
        int vfirst, vlast;
        {
          const Seq seq = {job.x.s.r0, job.x.s.n, job.x.s.kv};
          const int pos = seq.kv - seq.n + (job.x.row0 + min(w * 128 + r, job.x.rows - 1)) / p.group;
          vfirst = visible_first(p, pos);
          vlast = visible_last(p, seq, pos);
        }
        float nbase = 0.0f, limit = -INFINITY, sum = 0.0f;
        int key = job.x.lo + job.step * kKeys;
        const int steps = job.steps;
        for (int j = 0; j < steps; ++j, key += kKeys, ++turns) {
          ok = mbar_spin(&s_full[w], turns & 1, abort, kErrWaitTmemFull);
          if (!ok) break;
          tc_fence_after();
          if (idle) {                                // none of this warp's rows is one: what they hold is never read
            tc_fence_before();
            warp_arrive(&p_full[w]);
            continue;
          }
          const int first = vfirst - key, last = vlast - key;
          if (!__all_sync(0xFFFFFFFFu, first <= 0 && last >= kKeys)) row_mask(ts, first, last);
          const float top = row_max(ts);
          if (__any_sync(0xFFFFFFFFu, top > limit)) {
            const float was = limit == -INFINITY ? INFINITY : nbase, now = base_above(top, qscale);
            float f = 1.0f;
            if (now < was) {
              f = ex2(now - was);                    // 0 from infinity
              nbase = now;
              limit = base_limit(top, qscale);
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
          sum += row_exp(ts, qscale, nbase);
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&p_full[w]);
        }
        if (!ok) break;
        __syncwarp();
        if (following < n) bring_queries(jobs[following]);
        ok = mbar_wait(&o_full[w], done & 1, abort, kErrWaitTmemFull);
        if (!ok) break;
        ++done;
        tc_fence_after();
        // ---- the item's end ----
        const float top = limit == -INFINITY ? -INFINITY : -nbase;
        if (limit == -INFINITY) sum = 0.0f;        // no visible key (the polynomial's least value is not zero)
        const bool real = w * 128 + r < job.x.rows;
        const int row = job.x.row0 + w * 128 + r, token = row / p.group, h = job.head * p.group + row - token * p.group;
        const int64_t out_token = job.x.s.r0 + static_cast<int64_t>(token);
        uint16_t* out = p.o + out_token * p.ot + h * p.oh;
        if (job.steps == job.x.steps) {
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
        } else if (!idle) {
          // A part: [D / 4][256] float4 (coalesced over the rows), the bases, the sums.  Every warp joins its own 32
          // rows: the last CTA's warp to get here, in CTA order.
          const int64_t i0 = job.s - job.step, i1 = i0 + job.x.steps;  // the item's steps in the list
          Range range;
          range.q = kept[16];
          range.r = kept[17];
          const int row_in = w * 128 + r;
          float* slot = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (job.step > 0 ? 0 : 1)) * L::kPart;
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
          int c0, parts;
          if (range.q < 0) {                         // CTAs of its own
            c0 = static_cast<int>(blockIdx.x) / static_cast<int>(range.r) * static_cast<int>(range.r);
            parts = min(static_cast<int>(range.r), job.x.steps);
          } else {
            c0 = range.owner(i0);
            parts = range.owner(i1 - 1) - c0 + 1;
          }
          unsigned* count = p.count + c0 * 8 + warp;
          __threadfence();
          __syncwarp();
          unsigned arrived = 0;
          if (lane == 0) arrived = atom_add_acq_rel_gpu(count, 1u);
          arrived = __shfl_sync(0xFFFFFFFFu, arrived, 0);
          if (arrived == static_cast<unsigned>(parts - 1)) {
            __threadfence();
            if (lane == 0) *count = 0;
            const float* at0 = p.part + (2 * static_cast<int64_t>(c0) + 1) * L::kPart;
            const float* at1 = p.part + 2 * (static_cast<int64_t>(c0) + 1) * L::kPart;     // the others', 2 kPart apart
            auto part = [&](int c) { return c == 0 ? at0 : at1 + 2 * static_cast<int64_t>(c - 1) * L::kPart; };
            float m = -INFINITY, l = 0.0f;
#pragma unroll 4
            for (int c = 0; c < parts; ++c) m = fmaxf(m, __ldcg(part(c) + kRows * D + row_in));
            auto share = [&](int c) {              // a part's factor
              const float mc = __ldcg(part(c) + kRows * D + row_in);
              return mc == -INFINITY ? 0.0f : ex2(mc - m);
            };
#pragma unroll 4
            for (int c = 0; c < parts; ++c) l += __ldcg(part(c) + kRows * (D + 1) + row_in) * share(c);
            const float f = l > 0.0f ? p.c.vg / l : 0.0f;
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {     // 32 columns: eight loads on their way
              float4 a[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) a[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
              for (int c = 0; c < parts; ++c) {
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(part(c)) + (8 * e + k) * kRows + row_in);
                const float g = share(c);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  a[k].x += v[k].x * g; a[k].y += v[k].y * g; a[k].z += v[k].z * g; a[k].w += v[k].w * g;
                }
              }
              if (real) {
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                  *reinterpret_cast<uint4*>(out + 32 * e + 4 * k) =
                      make_uint4(pack_bf16x2(a[k].x * f, a[k].y * f), pack_bf16x2(a[k].z * f, a[k].w * f),
                                 pack_bf16x2(a[k + 1].x * f, a[k + 1].y * f), pack_bf16x2(a[k + 1].z * f, a[k + 1].w * f));
              }
            }
            if (p.lse && real) p.lse[out_token * p.Hq + h] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
          }
        }
      }
      if (list_done(n)) break;
    }
  } else if (warp < 12) {
    for (;;) {
      // ---------------------------------------------------------- widening ---
      // One thread per key; the next tile's bytes are on their way while this one's are widened.
      const int r = threadIdx.x - 256;
      uint4 raw[2][D / 32];
      uint2 sc[2];
      // a key's page (-1: no such key), looked up one tile ahead of its bytes
      auto page_of = [&](const Job& j, int step) {
        const int key = j.x.lo + (j.step + step) * kKeys + r;
        return key < j.x.hi && key >= j.x.first ? p.table[j.u / p.row_tiles * p.table_stride + (key >> p.c.page_shift)] : -1;
      };
      auto fetch = [&](const Job& j, int step, int page, int which) {
        const int key = j.x.lo + (j.step + step) * kKeys + r;
        const bool there = key < j.x.hi && key >= j.x.first;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[which][i] = make_uint4(0, 0, 0, 0);
        sc[which] = make_uint2(0, 0);
        if (there && (page < 0 || page >= p.c.pages)) atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadPage));
        if (there && page >= 0 && page < p.c.pages) {
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
      // tiles in turn: at (i, j) the one widened, then the one whose bytes are fetched, then the one whose page is
      int fi = 0, fj = 0;
      auto step_on = [&](int& i, int& j) {
        if (++j == jobs[i].steps) {
          j = 0;
          ++i;
        }
      };
      int page = page_of(jobs[0], 0);
      fetch(jobs[0], 0, page, 0);
      fetch(jobs[0], 0, page, 1);
      meet_all();
      const int n = *njobs;
      step_on(fi, fj);
      page = fi < n ? page_of(jobs[fi], fj) : -1;
      for (int i = 0; i < n && ok; ++i) {
        const int steps = jobs[i].steps;
        for (int j = 0; j < steps && ok; ++j, ++tiles) {
          const int st = tiles & 1, ph = ((tiles >> 1) & 1) ^ 1;
          ok = mbar_wait(&k_empty[st], ph, abort, kErrWaitEmpty);
          if (!ok) break;
          widen(0, smem + L::kK + st * L::kTile);
          warp_arrive(&k_full[st]);
          if (fi < n) fetch(jobs[fi], fj, page, 0);
          ok = mbar_wait(&v_empty[st], ph, abort, kErrWaitEmpty);
          if (!ok) break;
          widen(1, smem + L::kV + st * L::kTile);
          warp_arrive(&v_full[st]);
          if (fi < n) {
            fetch(jobs[fi], fj, page, 1);
            step_on(fi, fj);
            page = fi < n ? page_of(jobs[fi], fj) : -1;
          }
        }
      }
      if (list_done(n)) break;
    }
  } else {
    for (;;) {
      if (lane == 0) list_jobs();
      meet_all();
      const int n = *njobs;
      // ---------------------------------------------------------- products ---
      constexpr uint32_t kIdescS = idesc_f16_f32(128, kKeys, false), kIdescO = idesc_f16_f32(128, D, true);
      // descriptors of the tiles' starts: an offset is added to the address field (shared memory ends below its range)
      const uint64_t q_desc = umma_desc_sw128(smem_u32(smem + L::kQ)), k_desc = umma_desc_sw128(smem_u32(smem + L::kK));
      const uint64_t v_desc = umma_desc_mn_sw128(smem_u32(smem + L::kV), kHalf);
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int steps = jobs[i].steps, two = jobs[i].x.rows > 128 ? 2 : 1;
        auto score = [&](int w, int tile) {          // S_w = Q_w . K_tile^T
          const uint64_t a = q_desc + (w * L::kTile >> 4), b = k_desc + ((tile & 1) * L::kTile >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_f16_ss(tmem + w * 128, a + ((k / 4 * kHalf + k % 4 * 32) >> 4), b + ((k / 4 * kHalf + k % 4 * 32) >> 4),
                         kIdescS, k > 0);
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
            ok = mbar_spin(&p_full[w], (w ? turns1 : turns) & 1, abort, kErrWaitTmemFull);
            if (!ok) break;
            if (w) ++turns1; else ++turns;
            tc_fence_after();
            const uint64_t v = v_desc + ((tile & 1) * L::kTile >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                mma_f16_ts(tmem + 256 + w * 128, tmem + w * 128 + k * 8, v + (k * 2048 >> 4), kIdescO,
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
      if (list_done(n)) break;
    }
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
