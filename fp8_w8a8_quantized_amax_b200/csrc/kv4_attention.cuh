// kv4_attention.cuh -- attention over the paged 4-bit KV cache.
//
// For query row i of sequence b (n_b rows, the last n_b of its kv_len tokens):
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(sm_scale q.k_j - m),
// over the visible keys j: j < kv_len; causal: j <= pos, pos = kv_len - n_b + i;
// a window W: j > pos - W.  One pass over the cache: running maximum m and sum
// in fp32, the sums rescaled when m grows.
#pragma once

#include "kv4.cuh"
#include "kv4_list.cuh"

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
  unsigned* count;          // workspace: arrivals at the item that is cut at a CTA's end
  float* part;              // workspace: two partial results per CTA
  int64_t qt, qh, ot, oh, table_stride;
  int T, B, Hq, group, max_pages, max_q, row_tiles;
  float scale;              // sm_scale * g_k * log2(e)
  int causal;
  int64_t window;           // 0: none
};

constexpr float kLn2 = 0.693147180559945309f;

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
__device__ __forceinline__ int visible_first(const AttnParams& p, int pos) {
  if (p.window <= 0) return 0;
  const int64_t f = static_cast<int64_t>(pos) - p.window + 1;
  return f > 0 ? static_cast<int>(f) : 0;
}
__device__ __forceinline__ int visible_last(const AttnParams& p, const Seq& s, int pos) {
  return p.causal ? max(0, min(s.kv, pos + 1)) : s.kv;
}

// A sum over the list holds its steps in the low 40 bits and its items above (the host bounds both).
constexpr int64_t kOneItem = static_cast<int64_t>(1) << 40;

// The softmax base.  It is raised only when a score passes the one before by 2^kSlack, and lies 2^kLift below the score
// that raised it: the largest P of a row lies between 2^kLift and 2^(kLift + kSlack) = 2^15, the last power of two that
// f16 has.  P is rounded to f16, the sum of the weights takes it unrounded; with kLift = 0 keys 16.5 nats below a
// dominant one were off by 13%, and from 17.4 on nothing was left of them.  Now a weight keeps f16's 11 bits down to
// 2^-21 of the row's largest, and n keys lose at most n 2^-32 of it below that.  Both are rounded so that P never passes
// 2^15, whatever the size of the scores.
constexpr float kSlack = 8.0f, kLift = 7.0f;
__device__ __forceinline__ float rcp_approx(float x) {    // off by 2^-23 of itself at most
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The negated base that a largest score asks for; infinity where it is minus infinity (no visible key).
__device__ __forceinline__ float base_above(float top, float qscale) { return __fmaf_rd(-top, qscale, kLift); }
// The score up to which it is kept, 2^kSlack above that one in the exponent: an approximate quotient will do, as it is taken
// a little too small.
__device__ __forceinline__ float base_limit(float top, float qscale) {
  return __fadd_rd(top, (kSlack - 0.001f) * rcp_approx(qscale));
}

__device__ __forceinline__ void widen4(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// One half of an f16x2 in both halves (the multiplication takes either half of a register by itself).
__device__ __forceinline__ uint32_t dup_lo(uint32_t a) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t dup_hi(uint32_t a) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: no accumulator to read.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The scores' factor stays a normal number: minus infinity times it has to be minus infinity.
constexpr float kLeastScale = 1.17549435e-38f;

// A power of two that brings a value of magnitude amax to [2^14, 2^15) (as far
// as fp32 has it), by its exponent k.
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);
  return amax > 0.0f ? min(126, 141 - e) : 0;
}
__device__ __forceinline__ float pow2(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// ------------------------------------------------------------ few rows ---
//
// Up to 8 NT query rows per key head (the group's heads times the new tokens)
// meet every cached key, so the work is the stream of the cache: 9 D / 8 bytes
// per key and head.  Matrix instructions keep the products off the CUDA cores;
// with at most 8 NT columns they are mma.sync m16n8k16 with the keys (then the
// dimensions) as rows: the dequantized operand goes straight from registers
// into the instruction, where tcgen05 would want it written back to shared
// memory first.
//   S^T [16 keys, 8 rows]  = K [16 keys, D] . Q^T       (A = K, dequantized)
//   O^T [16 dims, 8 rows] += V^T [16 dims, 16 keys] . P^T  (A = V^T)
// Both contractions may go over their index in any order as long as both
// operands agree, so each lane takes a contiguous run of a cache row: of K's
// rows 32 elements (one 16-byte load, two scales), of V's rows 16 (one scale).
// V^T's operand pairs two keys in a register: the two keys' nibbles are merged
// into bytes (two logic operations for four values) before they are widened.
// E2M1 times E4M3 is exact in f16.  Q is scaled by a power of two per row so
// that its bf16 values are f16 values (exactly down to 2^-31 of the row's
// largest; smaller ones are rounded to multiples of at most 2^-38 of it); P is
// rounded to f16, its base chosen for that (above).
//
// The keys of a (sequence, key head) are cut into steps of WARPS * 32; the
// list of all steps is cut evenly over the CTAs (stream-K, as in the linear's
// decode kernel), whatever the lengths.  A warp takes 32 keys of each step
// through its own two-stage ring of asynchronous copies and keeps its own running
// maximum, sum and O^T; the warps' results are joined where an item ends.  An
// item cut between CTAs is joined by the last of them to finish, in CTA order.
//
// Measured, launches back to back: 64 sequences of 410 .. 8192 keys, 32 + 8 heads
// of 128, one token each: 76 us, 4.3 TB/s of cache (0.67 of a copy).  HBM does not
// bound it there, nor does any unit: the issue slots are 62% and the ALUs 50%
// busy with a key's conversions, products with the scales and matrix
// instructions, whose latencies 16 warps an SM do not hide.  One token behind
// 131072 keys (three heads to a key head): 42 us, of which the joins take about
// 8.  One sequence of 500 keys: 8.6 us, the latency of a prologue, four steps and
// a join.  16 sequences of four drafted tokens, 32 rows and 4096 keys: 48 us; two
// tiles of 16 rows widen every key twice, with 12 warps an SM.
namespace few {

constexpr int kTile = 32;     // keys of a warp per step
constexpr int kStages = 2;
constexpr int kJoinCost = 4;  // steps that joining an item's parts takes (2: 500 keys 8.8 -> 10.1 us; 8: as 4)

template <int D, int NT, int WARPS>
struct Layout {
  static constexpr int kThreads = 32 * WARPS;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStep = WARPS * kTile;
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);       // K codes, K scales, V codes, V scales
  static constexpr int kRedStride = D + 4;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  // [8][kRedStride] fp32 a warp, over the warp's free stage: the partial results meet eight rows at a time
  static_assert(8 * kRedStride * 4 <= kStageBytes, "eight rows in a stage");
  // and the bases and sums of as many parts as are joined at a time (kJoin, or the groups of kJoin that there can be)
  static_assert(kMaxCtas / kJoin >= kJoin && kMaxCtas / kJoin / WARPS * kRows * 8 <= kStageBytes, "over the free stages");
  static constexpr int kMl = WARPS * kWarpBytes;                   // [WARPS][kRows] m, then l
  static constexpr int kQ = kMl + 2 * WARPS * kRows * 4;           // Q fragments
  static constexpr int kRaw = kQ + NT * (D / 16) * 32 * 8;         // the current and the next job's query rows, as they are
  static constexpr int kRawBytes = kRows * D * 2;
  static constexpr int kMisc = kRaw + 2 * kRawBytes;
  static constexpr int kJobs = kMisc + 128;                        // two jobs of at most 64 bytes
  static constexpr int kBytes = kJobs + 128;
  static constexpr int kPart = kRows * (D + 2);                    // floats of a partial result
};

// A sequence's keys [first, hi) that some row sees, lo (first rounded down to a
// tile), the steps they make and the number of items (row tiles times key heads).
struct Span {
  Seq s;
  int first, lo, hi, steps, items;
};

template <int ROWS, int STEP>
__device__ __forceinline__ Span span(const AttnParams& p, int b) {
  Span x;
  x.s = sequence(p, b);
  x.hi = x.s.kv;
  x.first = visible_first(p, x.s.kv - x.s.n);
  x.lo = x.first & ~(kTile - 1);
  x.steps = max(1, (x.hi - x.lo + STEP - 1) / STEP);
  x.items = x.s.n > 0 ? (x.s.n * p.group + ROWS - 1) / ROWS * p.c.heads : 0;
  return x;
}

// A CTA's part of one item: `steps` steps from step `step`, key `key` on, its
// place in the list, and what the item is.
struct Job {
  Span x;
  int b, item, step, steps, key;
  int64_t s;                 // the part's first step in the list
};
static_assert(sizeof(Job) <= 64, "two of them in the layout");

// The list of steps counts kOver steps more in front of every item: what an
// item costs beside its keys (its queries, its join), so that the CTAs that get
// many short items are not the last ones.  A cut that falls into them is a cut
// ahead of the item's first step.
//
// The job of sequence b, item `item` (may be one past the last), step `step`,
// the item's extra steps starting at s - step - kOver in the list; the CTA's
// range ends at `end` (steps <= 0: ahead of the job).
template <int ROWS, int STEP>
__device__ __forceinline__ void make_job(const AttnParams& p, int b, int item, int step, int64_t s, int64_t end, Job* j) {
  Span x = span<ROWS, STEP>(p, b);
  while (item >= x.items && b + 1 < p.B) {     // the first sequence from here on that has rows: one exists, as s < end
    item = 0;
    x = span<ROWS, STEP>(p, ++b);
  }
  j->x = x;
  j->b = b;
  j->item = item;
  j->step = step;
  j->steps = static_cast<int>(min(static_cast<int64_t>(x.steps - step), end - s));
  j->key = x.lo + step * STEP;
  j->s = s;
}

template <int D, int NT, int WARPS, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) attention_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<D, NT, WARPS>;
  constexpr int kRows = L::kRows, kStep = L::kStep, kSteps = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = lane_id(), warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  // warp w's partial O^T at the end of a job; `stage` is then the stage of the next tile, in flight, and the other free
  auto red_of = [&](int w, int stage) {
    return reinterpret_cast<float*>(smem + w * L::kWarpBytes + (stage ^ 1) * L::kStageBytes);
  };
  float* ml = reinterpret_cast<float*>(smem + L::kMl);
  uint2* qs = reinterpret_cast<uint2*>(smem + L::kQ);
  Job* jobs = reinterpret_cast<Job*>(smem + L::kJobs);             // two: the current one and its successor
  int64_t* misc = reinterpret_cast<int64_t*>(smem + L::kMisc);
  int* red_max = reinterpret_cast<int*>(misc + 13);
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's range of the list: a scan over the sequences' steps ----
  // (steps in the low 40 bits, items above: B items and steps are bounded by the host)
  int64_t total = 0, before = 0;     // before: what lies ahead of this thread's sequence, in the last chunk scanned
  int64_t mine = 0;
  int longest = 0;
  auto scan = [&](int base) {
    const int b = base + static_cast<int>(threadIdx.x);
    mine = 0;
    if (b < p.B) {
      const Span x = span<kRows, kStep>(p, b);
      mine = static_cast<int64_t>(x.items) * (x.steps + kOver + kOneItem);
      if (x.items > 0) longest = max(longest, x.steps);
    }
    int64_t v = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) misc[warp] = v;
    __syncthreads();
    int64_t ahead = 0, all = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) ahead += misc[w];
      all += misc[w];
    }
    before = ahead + v - mine;
    return all;
  };
  for (int base = 0; base < p.B; base += L::kThreads) total += scan(base);
  Range range;
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  if (lane == 0) red_max[warp] = longest;
  const int items = static_cast<int>(total >> 40);
  const int64_t steps_all = total & (kOneItem - 1);
  range.q = quotient(steps_all, gridDim.x);
  range.r = steps_all - range.q * gridDim.x;
  __syncthreads();
  for (int w = 0; w < WARPS; ++w) longest = max(longest, red_max[w]);
  // As many CTAs as items, or more: each item is left to one of them where its steps take no longer than an even share
  // and the join (64 sequences of 1000 keys and 8 heads: 28 -> 22 us).
  const bool by_item = items <= static_cast<int>(gridDim.x) &&
                       longest + kOver <= max(range.q, static_cast<int64_t>(kOver + 1)) + kJoinCost;
  {
    const int64_t begin = by_item ? static_cast<int64_t>(blockIdx.x) : range.begin(blockIdx.x);
    const int64_t end = by_item ? (begin < items ? kOneItem : begin) : range.begin(blockIdx.x + 1);
    if (begin == end) return;
    // What is needed between jobs only is read back from shared memory there, not held in registers through the loop
    // over the keys (spills inside that loop cost 10%).
    if (threadIdx.x == 0) {
      misc[11] = by_item ? -1 : range.q;
      misc[12] = range.r;
    }
    int64_t ahead = 0;
    for (int base = 0; base < p.B; base += L::kThreads) {
      const int64_t all = p.B <= L::kThreads ? total : scan(base);
      const int64_t all_w = by_item ? all >> 40 : all & (kOneItem - 1);
      if (begin >= ahead && begin < ahead + all_w) {
        const int64_t at = begin - ahead - (by_item ? before >> 40 : before & (kOneItem - 1));
        if (at >= 0 && at < (by_item ? mine >> 40 : mine & (kOneItem - 1))) {
          const int b = base + static_cast<int>(threadIdx.x);
          const int steps = span<kRows, kStep>(p, b).steps + kOver;
          const int item = static_cast<int>(by_item ? at : quotient(at, steps));
          const int off = by_item ? 0 : static_cast<int>(at - static_cast<int64_t>(item) * steps);
          make_job<kRows, kStep>(p, b, item, max(0, off - kOver), begin + max(0, kOver - off), end, jobs);
        }
        break;
      }
      ahead += all_w;
    }
  }
  __syncthreads();
  if (jobs[0].steps <= 0) return;

  // ---- loads: the warp's tile of a step, from one page (two where pages hold 16 keys) ----
  // Nine 16-byte copies a lane at D = 128: four of K's codes, four of V's, one of the scales (lanes 0 .. 15 K's, the
  // others V's).  Bulk copies would need one instruction per run, issued lane by lane: with four runs a tile they
  // took as many issue slots as the products (95 us against 89 us then, on 64 ragged sequences of up to 8192 keys).
  uint8_t* stages = smem + warp * kStages * L::kStageBytes;
  const uint32_t slab = static_cast<uint32_t>(p.c.slab()), page_bytes = slab * p.c.heads;
  constexpr int kLoads = L::kCodes / 512;           // 16-byte copies a lane for one tensor's codes
  constexpr int kScaleLanes = L::kScales / 16;      // lanes that copy one tensor's scales
  const int scale_key = lane % kScaleLanes * (256 / D);                 // first key of this lane's 16 bytes of scales
  const int64_t v_from_k = p.c.v - p.c.k;
  // what this lane's copies start from: K's codes (and the scales, of K or V) of an item's head
  auto codes_of = [&](int head) { return p.c.k + static_cast<int64_t>(head) * slab + lane * 16; };
  auto scales_of = [&](int head) {
    return (lane < kScaleLanes ? p.c.k : p.c.v) + static_cast<int64_t>(head) * slab + p.c.page_size * (D / 2);
  };
  // Pages of a tile's two halves (one page, where pages hold 32 keys or more).  A half that no key needs is stood in
  // for by the nearest that one does: what is read there is masked.
  auto pages_of = [&](const int32_t* row, int key, int lo, int hi) {
    int2 v;
    v.x = row[min(max(key, lo), hi - 1) >> p.c.page_shift];
    v.y = row[min(max(key + kTile / 2, lo), hi - 1) >> p.c.page_shift];
    return v;
  };
  auto issue = [&](const uint8_t* codes, const uint8_t* scales, int2 page, int key, int stage) {
    if (static_cast<unsigned>(max(page.x, page.y)) >= static_cast<unsigned>(p.c.pages) || min(page.x, page.y) < 0) {
      atomicCAS(&g_device_error, 0, static_cast<int>(kErrBadPage));
      page = make_int2(0, 0);
    }
    uint8_t* dst = stages + stage * L::kStageBytes + lane * 16;
    const int in_page = p.c.page_size - 1;
    const uint8_t* src[2];
    src[0] = codes + static_cast<uint64_t>(static_cast<uint32_t>(page.x)) * page_bytes + (key & in_page) * (D / 2);
    src[1] = codes + static_cast<uint64_t>(static_cast<uint32_t>(page.y)) * page_bytes + ((key + kTile / 2) & in_page) * (D / 2);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint8_t* from = src[i / (kLoads / 2)] + i % (kLoads / 2) * 512;
      cp_async_16(dst + i * 512, from);
      cp_async_16(dst + L::kCodes + L::kScales + i * 512, from + v_from_k);
    }
    if (lane < 2 * kScaleLanes)
      cp_async_16(dst + L::kCodes + (lane < kScaleLanes ? 0 : L::kCodes),
                  scales + static_cast<uint64_t>(static_cast<uint32_t>(scale_key < kTile / 2 ? page.x : page.y)) * page_bytes +
                      ((key + scale_key) & in_page) * (D / 16));
  };

  // per row: the scores' factor, the base (negated; 0 before the first key), the score at which it is raised, the sum
  float qscale[NT][2], nbase[NT][2], limit[NT][2], l[NT][2];
  float o[kSteps][NT][4];
  auto stored_range = [&]() {
    const volatile int64_t* m = misc;
    Range r;
    r.q = m[11];
    r.r = m[12];
    return r;
  };
  auto first_pages = [&](int slot) {                // of a job's first tile
    const Job& j = jobs[slot];
    const int k = j.key + warp * kTile;
    return k < j.x.hi ? pages_of(p.table + j.b * p.table_stride, k, j.x.first, j.x.hi) : make_int2(0, 0);
  };
  // A job's query rows, on their way while the job before it is worked on (one group of copies).
  auto fetch_rows = [&](int slot) {
    const Job& j = jobs[slot];
    const int row0 = j.item / p.c.heads * kRows, rows = min(kRows, j.x.s.n * p.group - row0), head = j.item % p.c.heads;
    for (int i = threadIdx.x; i < rows * (D / 8); i += L::kThreads) {
      const int r = i / (D / 8), row = row0 + r;
      cp_async_16(smem + L::kRaw + slot * L::kRawBytes + i * 16,
                  p.q + (j.x.s.r0 + row / p.group) * p.qt + (head * p.group + row % p.group) * p.qh + i % (D / 8) * 8);
    }
    cp_async_commit();
  };
  int stage = 0, which = 0;
  fetch_rows(0);
  {
    const Job& j = jobs[0];
    const int key = j.key + warp * kTile, head = j.item % p.c.heads;
    if (key < j.x.hi)
      issue(codes_of(head), scales_of(head), first_pages(0), key, 0);
    cp_async_commit();
  }
  cp_async_wait<1>();
  __syncthreads();

  for (;; which ^= 1) {
    // ---- an item (or this CTA's part of it): its query rows, and the next job ----
    const volatile Job& job = jobs[which];
    bool more;
    {
      const Range range = stored_range();
      const int64_t end = range.begin(blockIdx.x + 1);
      more = range.q >= 0 && job.s + job.steps + kOver < end;      // (q < 0: one item a CTA)
      if (more && threadIdx.x == 0)                    // (then this job ends its item)
        make_job<kRows, kStep>(p, job.b, job.item + 1, 0, job.s + job.steps + kOver, end, &jobs[which ^ 1]);
    }
    const int hi = job.x.hi, lo = job.x.first, steps = job.steps, head = job.item % p.c.heads;
    int all_first, all_last;                        // keys that every row of the item sees
    {
      const Seq seq = {job.x.s.r0, job.x.s.n, job.x.s.kv};
      const int row0 = job.item / p.c.heads * kRows, rows = min(kRows, seq.n * p.group - row0);
      all_last = visible_last(p, seq, seq.kv - seq.n + row0 / p.group);
      all_first = visible_first(p, seq.kv - seq.n + (row0 + rows - 1) / p.group);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // lane (g, t) holds row 8 nt + g, elements [t D/4, (t + 1) D/4)
        const int r = nt * 8 + g;
        uint32_t w[D / 8];
        if (r < rows) {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(smem + L::kRaw + which * L::kRawBytes) + r * D + t * (D / 4);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) w[i] = 0;
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const int k = row_exponent(amax);
        const float up = pow2(k), down = fmaxf(pow2(-k) * p.scale, kLeastScale);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t b0 = pack_f16x2(bf16lo(w[2 * i]) * up, bf16hi(w[2 * i]) * up);
          const uint32_t b1 = pack_f16x2(bf16lo(w[2 * i + 1]) * up, bf16hi(w[2 * i + 1]) * up);
          if (warp == nt % WARPS) qs[(nt * kSteps + i) * 32 + lane] = make_uint2(b0, b1);
        }
        qscale[nt][0] = __shfl_sync(0xFFFFFFFFu, down, 8 * t);
        qscale[nt][1] = __shfl_sync(0xFFFFFFFFu, down, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          nbase[nt][i] = 0.0f;
          limit[nt][i] = -INFINITY;
          l[nt][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
      }
    }
    const int32_t* table = p.table + job.b * p.table_stride;
    int key = job.key + warp * kTile;
    const uint8_t* codes = codes_of(head);
    const uint8_t* scales = scales_of(head);
    int2 page = make_int2(0, 0);                    // of the tile to fetch next
    if (key + kStep < hi) page = pages_of(table, key + kStep, lo, hi);
    __syncthreads();                                // jobs[which ^ 1] and the fragments are written
    if (more) {
      fetch_rows(which ^ 1);
      if (steps == 1) page = first_pages(which ^ 1);
    }

    for (int i = 0; i < steps; ++i, key += kStep, stage ^= 1) {
      // ---- the next step's tile goes on its way ----
      if (i + 1 < steps) {
        if (key + kStep < hi) issue(codes, scales, page, key + kStep, stage ^ 1);
        if (i + 2 < steps) {
          if (key + 2 * kStep < hi) page = pages_of(table, key + 2 * kStep, lo, hi);
        } else if (more) {
          page = first_pages(which ^ 1);
        }
      } else if (more) {
        const Job& j = jobs[which ^ 1];
        const int k = j.key + warp * kTile, h = j.item % p.c.heads;
        if (k < j.x.hi) issue(codes_of(h), scales_of(h), page, k, stage ^ 1);
      }
      cp_async_commit();                            // one group a step, empty or not
      cp_async_wait<1>();                           // all but the next step's
      if (key >= hi) continue;
      __syncwarp();                                 // the other lanes' copies too
      const uint8_t* kc = stages + stage * L::kStageBytes;
      const uint8_t* ks = kc + L::kCodes;
      const uint8_t* vc = ks + L::kScales;
      const uint8_t* vs = vc + L::kCodes;
      const bool whole = key >= all_first && key + kTile <= all_last;
      // Row r of a 16-key tile is key r ^ (r / 4 & 1): K's rows of neighbouring lane groups and V's rows 2t (and
      // 2t + 1) of the four t then lie in different banks (V: at most two lanes to a bank).
      const int kg = g ^ ((g >> 2) & 1);
      float sc[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int r0 = mt * 16 + kg, r1 = r0 + 8;
        uint32_t w0[D / 32], w1[D / 32], s0[2], s1[2];
        if constexpr (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(kc + r0 * 64 + t * 16);
          const uint4 b = *reinterpret_cast<const uint4*>(kc + r1 * 64 + t * 16);
          w0[0] = a.x; w0[1] = a.y; w0[2] = a.z; w0[3] = a.w;
          w1[0] = b.x; w1[1] = b.y; w1[2] = b.z; w1[3] = b.w;
          const uint32_t x = widen_e4m3x2(*reinterpret_cast<const uint16_t*>(ks + r0 * 8 + t * 2));
          const uint32_t y = widen_e4m3x2(*reinterpret_cast<const uint16_t*>(ks + r1 * 8 + t * 2));
          s0[0] = dup_lo(x); s0[1] = dup_hi(x);
          s1[0] = dup_lo(y); s1[1] = dup_hi(y);
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(kc + r0 * 32 + t * 8);
          const uint2 b = *reinterpret_cast<const uint2*>(kc + r1 * 32 + t * 8);
          w0[0] = a.x; w0[1] = a.y;
          w1[0] = b.x; w1[1] = b.y;
          const uint32_t x = widen_e4m3x2(ks[r0 * 4 + t] | (static_cast<uint32_t>(ks[r1 * 4 + t]) << 8));
          s0[0] = s0[1] = dup_lo(x);
          s1[0] = s1[1] = dup_hi(x);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t a[4], b[4];
          widen4(w0[w], a);
          widen4(w1[w], b);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[j] = mul_f16x2(a[j], s0[w / 2]);
            b[j] = mul_f16x2(b[j], s1[w / 2]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q = qs[(nt * kSteps + 2 * w + h) * 32 + lane];
              if (w == 0 && h == 0) mma16816_first(sc[mt][nt], a[0], b[0], a[1], b[1], q.x, q.y);
              else mma16816(sc[mt][nt], a[2 * h], b[2 * h], a[2 * h + 1], b[2 * h + 1], q.x, q.y);
            }
        }
      }
      // Softmax over the tile: element i of sc is key (g, g + 8)[i / 2], row 2t + i % 2.
      if (__builtin_expect(!whole, 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const Seq seq = {job.x.s.r0, job.x.s.n, job.x.s.kv};
            const int row0 = job.item / p.c.heads * kRows, end_row = seq.n * p.group - 1;
            const int pos = seq.kv - seq.n + min(row0 + nt * 8 + 2 * t + q, end_row) / p.group;
            const int first = visible_first(p, pos), last = visible_last(p, seq, pos);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int k = key + mt * 16 + kg + h * 8;
                if (k < first || k >= last) sc[mt][nt][2 * h + q] = -INFINITY;
              }
          }
      }
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(fmaxf(sc[0][nt][i], sc[0][nt][i + 2]), fmaxf(sc[1][nt][i], sc[1][nt][i + 2]));
        }
        if (__any_sync(0xFFFFFFFFu, top[0] > limit[nt][0] || top[1] > limit[nt][1])) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d *= 2) top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], d));
            // (a row without a visible key so far stays at a base of 0, and its limit at -infinity)
            const float was = limit[nt][i] == -INFINITY ? INFINITY : nbase[nt][i];
            const float now = base_above(top[i], qscale[nt][i]);
            if (now < was) {
              const float f = ex2(now - was);       // 0 from infinity
              nbase[nt][i] = now;
              limit[nt][i] = base_limit(top[i], qscale[nt][i]);
              l[nt][i] *= f;
#pragma unroll
              for (int d = 0; d < kSteps; ++d) {
                o[d][nt][i] *= f;
                o[d][nt][i + 2] *= f;
              }
            }
          }
        }
        const uint64_t scale2 = f32x2_pack(qscale[nt][0], qscale[nt][1]), base2 = f32x2_pack(nbase[nt][0], nbase[nt][1]);
        uint64_t l2 = f32x2_pack(l[nt][0], l[nt][1]);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x, y;
            f32x2_unpack(fma_f32x2(f32x2_pack(sc[mt][nt][2 * h], sc[mt][nt][2 * h + 1]), scale2, base2), x, y);
            x = ex2(x);
            y = ex2(y);
            l2 = add_f32x2(l2, f32x2_pack(x, y));
            pf[mt][nt][h] = transpose8x8(pack_f16x2(x, y));
          }
        f32x2_unpack(l2, l[nt][0], l[nt][1]);
      }
      // V^T: row g (and g + 8) of m-tile i is element g D/8 + 2i (and + 1); columns 2t, 2t + 1 (and + 8) are keys
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int ka = mt * 16 + (2 * t ^ (t >> 1)), kb = mt * 16 + ((2 * t + 1) ^ (t >> 1));
        const int keys[4] = {ka, kb, ka + 8, kb + 8};
        uint32_t vw[4][D / 64], sv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint2 a = *reinterpret_cast<const uint2*>(vc + keys[i] * 64 + g * 8);
            vw[i][0] = a.x;
            vw[i][1] = a.y;
            sv[i] = vs[keys[i] * 8 + g];
          } else {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(vc + keys[i] * 32 + g * 4);
            sv[i] = vs[keys[i] * 4 + (g >> 1)];
          }
        }
        // what lies outside the keys, or was not loaded, need not be a number that times zero is zero
        if (__builtin_expect(!whole, 0)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key + keys[i] >= hi || key + keys[i] < lo) sv[i] = 0;
        }
        const uint32_t s01 = widen_e4m3x2(sv[0] | (sv[1] << 8)), s23 = widen_e4m3x2(sv[2] | (sv[3] << 8));
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t e0[4], e1[4], e2[4], e3[4];
          widen4((vw[0][w] & 0x0F0F0F0Fu) | ((vw[1][w] << 4) & 0xF0F0F0F0u), e0);
          widen4(((vw[0][w] >> 4) & 0x0F0F0F0Fu) | (vw[1][w] & 0xF0F0F0F0u), e1);
          widen4((vw[2][w] & 0x0F0F0F0Fu) | ((vw[3][w] << 4) & 0xF0F0F0F0u), e2);
          widen4(((vw[2][w] >> 4) & 0x0F0F0F0Fu) | (vw[3][w] & 0xF0F0F0F0u), e3);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e0[j] = mul_f16x2(e0[j], s01);
            e1[j] = mul_f16x2(e1[j], s01);
            e2[j] = mul_f16x2(e2[j], s23);
            e3[j] = mul_f16x2(e3[j], s23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816(o[4 * w + j][nt], e0[j], e1[j], e2[j], e3[j], pf[mt][nt][0], pf[mt][nt][1]);
          }
        }
      }
      __syncwarp();                                 // every lane has read the stage before it is filled again
    }

    // ---- the end of the job: the warps' results joined ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][i], d);
        if (g == 0) {
          const int r = nt * 8 + 2 * t + i;
          ml[warp * kRows + r] = limit[nt][i] == -INFINITY ? -INFINITY : -nbase[nt][i];
          ml[(WARPS + warp) * kRows + r] = l[nt][i];
        }
      }
    const Seq seq = {job.x.s.r0, job.x.s.n, job.x.s.kv};
    const int row0 = job.item / p.c.heads * kRows, rows = min(kRows, seq.n * p.group - row0);
    const Range range = stored_range();
    const int64_t i0 = job.s - job.step, i1 = i0 + job.x.steps;      // the item's steps in the list
    const bool split = job.steps < job.x.steps;
    auto finish = [&](int r, int d, float4 v, float top, float sum) {
      const int row = row0 + r;
      const int64_t token = seq.r0 + row / p.group;
      const int h = head * p.group + row % p.group;
      const float f = sum > 0.0f ? p.c.vg / sum : 0.0f;
      uint2 w;
      w.x = pack_bf16x2(v.x * f, v.y * f);
      w.y = pack_bf16x2(v.z * f, v.w * f);
      *reinterpret_cast<uint2*>(p.o + token * p.ot + h * p.oh + d) = w;
      if (p.lse && d == 0) p.lse[token * p.Hq + h] = sum > 0.0f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    };
    float* slot = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (job.step > 0 ? 0 : 1)) * L::kPart;   // a CTA's first job, its last
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      __syncthreads();                              // ml is written; the eight rows before these are read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = nt * 8 + 2 * t + i;
        float top = -INFINITY;
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w * kRows + r]);
        const float f = limit[nt][i] == -INFINITY ? 0.0f : ex2(-nbase[nt][i] - top);
        float* dst = red_of(warp, stage) + (2 * t + i) * L::kRedStride + g * (D / 8);
#pragma unroll
        for (int d = 0; d < kSteps; d += 2)
          *reinterpret_cast<float4*>(dst + 2 * d) = make_float4(o[d][nt][i] * f, o[d][nt][i + 2] * f,
                                                                o[d + 1][nt][i] * f, o[d + 1][nt][i + 2] * f);
      }
      __syncthreads();
      for (int i = threadIdx.x; i < min(8, rows - 8 * nt) * (D / 4); i += L::kThreads) {
        const int r = nt * 8 + i / (D / 4), d = i % (D / 4) * 4;
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w * kRows + r]);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < WARPS; ++w) {
          const float mw = ml[w * kRows + r];
          if (mw != -INFINITY) sum += ml[(WARPS + w) * kRows + r] * ex2(mw - top);
          const float4 x = *reinterpret_cast<const float4*>(red_of(w, stage) + (r - nt * 8) * L::kRedStride + d);
          v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
        }
        if (!split) {
          finish(r, d, v, top, sum);
        } else {
          __stcg(reinterpret_cast<float4*>(slot + r * D + d), v);
          if (d == 0) {
            __stcg(slot + kRows * D + r, top);
            __stcg(slot + kRows * (D + 1) + r, sum);
          }
        }
      }
    }
    if (split) {
      // The last of the item's CTAs to get here joins their parts, in CTA order, and leaves the counters zero.  Many
      // parts (a long context of few heads) are joined in two levels: groups of consecutive CTAs first, each by its
      // last, into its first part's place, then the groups (92 parts of 4 KB by one CTA took 10 us, bound by what one SM
      // reads from L2).
      const int c0 = range.owner(i0);
      const Joins joins = {c0, range.owner(i1 - 1) - c0 + 1};
      float* at0 = p.part + (2 * static_cast<int64_t>(c0) + 1) * L::kPart;
      float* at1 = p.part + 2 * (static_cast<int64_t>(c0) + 1) * L::kPart;     // the others', 2 kPart apart
      auto part_at = [&](int c) { return c == 0 ? at0 : at1 + 2 * static_cast<int64_t>(c - 1) * L::kPart; };
      Meeting meet = joins.first(static_cast<int>(blockIdx.x));
      for (;;) {
        const int from = meet.from, n = meet.n, stride = meet.stride;
        unsigned* count = p.count + meet.counter;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) misc[10] = atom_add_acq_rel_gpu(count, 1u);
        __syncthreads();
        if (static_cast<int>(misc[10]) != n - 1) break;
        __threadfence();
        if (threadIdx.x == 0) *count = 0;
        // the parts' bases and sums, over the warps' free stages
        auto mls = [&](int c) { return red_of(c % WARPS, stage) + c / WARPS * 2 * kRows; };
        for (int i = threadIdx.x; i < n * kRows; i += L::kThreads) {
          const int c = i / kRows, r = i % kRows;
          const float* src = part_at(from + c * stride) + kRows * D + r;
          *reinterpret_cast<float2*>(mls(c) + 2 * r) = make_float2(__ldcg(src), __ldcg(src + kRows));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * (D / 4); i += L::kThreads) {
          const int r = i / (D / 4), d = i % (D / 4) * 4;
          float top = -INFINITY, sum = 0.0f;
          for (int c = 0; c < n; ++c) top = fmaxf(top, mls(c)[2 * r]);
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
          for (int c = 0; c < n; ++c) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part_at(from + c * stride)) + i);
            const float2 ml2 = *reinterpret_cast<const float2*>(mls(c) + 2 * r);
            const float f = ml2.x == -INFINITY ? 0.0f : ex2(ml2.x - top);
            sum += ml2.y * f;
            v.x += x.x * f; v.y += x.y * f; v.z += x.z * f; v.w += x.w * f;
          }
          if (meet.final) {
            finish(r, d, v, top, sum);
          } else {
            float* dst = part_at(from);
            __stcg(reinterpret_cast<float4*>(dst) + i, v);
            if (d == 0) {
              __stcg(dst + kRows * D + r, top);
              __stcg(dst + kRows * (D + 1) + r, sum);
            }
          }
        }
        if (meet.final) break;
        meet = joins.second();
        __syncthreads();                            // misc and mls are free again
      }
    }
    if (!more) break;
    __syncthreads();                                // red, ml, misc and jobs[which] are free again
  }
}

}  // namespace few

}  // namespace kv4
}  // namespace fp8q
