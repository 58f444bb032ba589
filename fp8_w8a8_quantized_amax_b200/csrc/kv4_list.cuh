// kv4_list.cuh -- how attention over the 4-bit KV cache cuts the list of all its
// steps over the CTAs, and where the parts of a cut item meet.  Plain arithmetic
// that compiles for the host too: the tests walk through many lists with it.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FP8Q_KV4_HD __host__ __device__ __forceinline__
#else
#define FP8Q_KV4_HD inline
#endif

namespace fp8q {
namespace kv4 {

constexpr int kMaxCtas = 1024;  // counters of each level in the workspace's header

// The list of all steps of a call, cut evenly over the CTAs.
FP8Q_KV4_HD int64_t quotient(int64_t a, int64_t b) {     // a >= 0, b > 0; mostly 32-bit values
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

struct Range {
  int64_t q, r;   // CTA c takes q + 1 steps when c < r, else q
  FP8Q_KV4_HD int64_t begin(int64_t c) const { return c * q + (c < r ? c : r); }
  FP8Q_KV4_HD int owner(int64_t s) const {
    const int64_t big = r * (q + 1);
    return static_cast<int>(s < big ? quotient(s, q + 1) : r + quotient(s - big, q));
  }
};

namespace few {

constexpr int kJoin = 16;     // parts of an item joined at a time
constexpr int kOver = 3;      // steps that an item costs beside its keys, counted in front of it in the list

// A meeting: n results, those of the parts from, from + stride, ..., counted at
// one of the header's counters; the last to arrive joins them.
struct Meeting {
  int from, n, stride, counter;
  bool final;                 // they make up the item
};

// The meetings of an item that is cut into `parts` >= 2 parts, those of the CTAs
// c0, c0 + 1, ...: groups of kJoin consecutive parts, then the groups.
//
// No two meetings of a call have one counter.  An item's groups count at their
// first CTA's counter of the first level.  Where a group has two parts or more
// that CTA comes before the item's last one, and the next item begins in the last
// one or behind it.  A group of one part alone (17, 33, ... parts) is the item's
// last CTA, in which the next item may begin, with a group that counts there: the
// part alone, which has nothing to be joined with, goes on to the second level at
// once.  That counts at c0's counter of its own level: one item goes on past the
// end of a CTA.
struct Joins {
  int c0, parts;
  FP8Q_KV4_HD int groups() const { return parts <= kJoin ? 1 : (parts + kJoin - 1) / kJoin; }
  FP8Q_KV4_HD Meeting second() const { return {0, groups(), kJoin, kMaxCtas + c0, true}; }
  // where CTA cta's part goes first
  FP8Q_KV4_HD Meeting first(int cta) const {
    const int from = (cta - c0) / kJoin * kJoin, n = parts - from < kJoin ? parts - from : kJoin;
    return n == 1 ? second() : Meeting{from, n, 1, c0 + from, parts <= kJoin};
  }
};

}  // namespace few
}  // namespace kv4
}  // namespace fp8q
