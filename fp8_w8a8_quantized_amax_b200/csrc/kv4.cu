// kv4.cu -- C ABI of rotary positions and the 4-bit KV cache: argument checks
// and dispatch.  Arguments are checked before anything touches CUDA.
#include <cmath>

#include "host.cuh"
#include "kv4.cuh"
#include "kv4_attention.cuh"
#include "kv4_prefill.cuh"
#include "rope.cuh"

// The device error word of this file's kernels (fp8q_device_error reads it).
int fp8q_kv4_error_word(int clear, int* word) {
  if (cudaMemcpyFromSymbol(word, fp8q::g_device_error, sizeof(int)) != cudaSuccess) return -1;
  const int zero = 0;
  if (clear && cudaMemcpyToSymbol(fp8q::g_device_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  return 0;
}

namespace {

constexpr int64_t kStrideMax = static_cast<int64_t>(1) << 40;
constexpr int64_t kExtentMax = static_cast<int64_t>(1) << 48;   // elements; more than a device's memory has addresses for

bool finite_positive(float v) { return v > 0.0f && v < 3.0e38f; }   // also rejects NaN

// Strides of a [T, H, D] tensor with contiguous heads, in elements (those of a dimension of size 1 do not matter): no
// offset passes kExtentMax, so what is computed of them stays inside 63 bits.
bool bad_strides(int64_t T, int64_t H, int64_t t, int64_t h) {
  return t < 0 || h < 0 || (T > 1 && t > kExtentMax / (T - 1)) || (H > 1 && h > kExtentMax / (H - 1));
}

// Whether the (token, head) rows of a tensor that is written overlap.
bool rows_overlap(int64_t T, int64_t H, int64_t D, int64_t t, int64_t h) {
  const bool tokens_outside = (H == 1 || h >= D) && (T == 1 || t >= (H - 1) * h + D);
  const bool heads_outside = (T == 1 || t >= D) && (H == 1 || h >= (T - 1) * t + D);
  return !tokens_outside && !heads_outside;
}

fp8q_status check_rope(const int64_t* positions, const double* freq, int64_t rot_dim, int64_t D, int flags, float m) {
  if (rot_dim <= 0 || rot_dim > D || rot_dim % 2 != 0) return FP8Q_ERR_INVALID_ARG;
  if (flags & ~(FP8Q_ROPE_INTERLEAVED | FP8Q_ROPE_INVERSE)) return FP8Q_ERR_INVALID_ARG;
  if (!finite_positive(m) || !positions || !freq) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(freq, 8)) return FP8Q_ERR_MISALIGNED;
  return FP8Q_OK;
}

fp8q_status check_cache(const fp8q_kv4_cache* c) {
  if (!c || !c->k_pages || !c->v_pages) return FP8Q_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->kv_heads <= 0) return FP8Q_ERR_INVALID_ARG;
  if (!finite_positive(c->k_scale) || !finite_positive(c->v_scale)) return FP8Q_ERR_INVALID_ARG;
  if (c->page_size <= 0 || (c->page_size & (c->page_size - 1)) != 0) return FP8Q_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return FP8Q_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || c->kv_heads > 4096 || c->num_pages > kInt32Max)
    return FP8Q_ERR_UNSUPPORTED;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return FP8Q_ERR_MISALIGNED;
  return FP8Q_OK;
}

fp8q::kv4::Cache device_cache(const fp8q_kv4_cache* c) {
  fp8q::kv4::Cache d;
  d.k = static_cast<uint8_t*>(c->k_pages);
  d.v = static_cast<uint8_t*>(c->v_pages);
  d.pages = c->num_pages;
  d.page_size = c->page_size;
  d.page_shift = 31 - __builtin_clz(static_cast<unsigned>(c->page_size));
  d.heads = c->kv_heads;
  d.D = c->head_dim;
  d.kg = c->k_scale;
  d.vg = c->v_scale;
  return d;
}

// A bf16 [T, heads, D] operand of the cache's entry points.
fp8q_status check_rows(const void* p, int64_t T, int64_t H, int64_t t, int64_t h) {
  if (!p || bad_strides(T, H, t, h)) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(p, 16) || t % 8 != 0 || h % 8 != 0) return FP8Q_ERR_MISALIGNED;
  return FP8Q_OK;
}

// What a call of these sizes launches: the kernel for few rows with 8 nt rows a
// tile, or (nt = 0) the one for many; `ctas` CTAs; and the workspace: a header
// of arrival counters, then two partial results per CTA.  One kernel takes the
// whole call, by the longest sequence's rows (lengths stay on the device): 2048
// rows and 63 single tokens of 410 .. 8192 keys take 560 us in one call, 244 + 74
// in two.
constexpr size_t kWorkspaceHeader = 2 * fp8q::kv4::kMaxCtas * sizeof(unsigned);
static_assert(kWorkspaceHeader == FP8Q_KV4_WORKSPACE_HEADER, "as declared");

struct AttentionPlan {
  int nt, ctas, row_tiles;
  size_t part;
  size_t bytes() const { return kWorkspaceHeader + static_cast<size_t>(2 * ctas) * part; }
};

AttentionPlan attention_plan(const fp8q_kv4_cache* c, int64_t T, int64_t Hq, int64_t max_q_len, int sms) {
  const int64_t rows = (max_q_len < T ? max_q_len : T) * (Hq / c->kv_heads);
  AttentionPlan a;
  // Rows of a key head (the group's heads times the new tokens), D = 128.  Tiles of 8 have four CTAs an SM and little
  // to join, tiles of 16 dequantize a key for twice the rows.  24 rows: three tiles of 8 against two of 16 take 37
  // against 38 us for 16 sequences of 4096 keys, 17 against 20 for ones of 700, 78 against 75 for 32 of 8000; 32 rows:
  // 47 against 47, 19 against 22, 104 against 95.  Half a tensor-memory tile pays from six tiles of 16 on: 80 rows 84
  // against 88, 31 against 44, 200 against 194 us; 96 rows: 96 against 88, 34 against 44, 239 against 193.
  a.nt = rows <= 24 ? 1 : (rows <= 80 ? 2 : 0);
  a.ctas = sms * (a.nt == 1 ? (c->head_dim == 64 ? 5 : 4) : (a.nt == 2 ? 3 : 1));
  const int most = fp8q::kv4::kMaxCtas / (a.nt ? 1 : 4);       // a CTA has two of the header's counters, or eight
  if (a.ctas > most) a.ctas = most;
  const int64_t tile = a.nt ? 8 * a.nt : fp8q::kv4::many::kRows;
  a.row_tiles = static_cast<int>((rows + tile - 1) / tile);
  a.part = static_cast<size_t>(tile) * (c->head_dim + 2) * sizeof(float);
  return a;
}

template <int D>
fp8q_status launch_many(const fp8q::kv4::AttnParams& p, int ctas, int dev, void* stream) {
  using L = fp8q::kv4::many::Layout<D>;
  auto k = fp8q::kv4::many::attention_kernel<D>;
  fp8q_status st = ensure_smem(k, L::kBytes, dev);
  if (st != FP8Q_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(ctas)), dim3(fp8q::kv4::many::kThreads), L::kBytes, stream, p);
}

template <int D, int NT, int CTAS>
fp8q_status launch_few(const fp8q::kv4::AttnParams& p, int ctas, int dev, void* stream) {
  constexpr int kWarps = 4;
  using L = fp8q::kv4::few::Layout<D, NT, kWarps>;
  auto k = fp8q::kv4::few::attention_kernel<D, NT, kWarps, CTAS>;
  fp8q_status st = ensure_smem(k, L::kBytes, dev);
  if (st != FP8Q_OK) return st;
  return launch(k, dim3(static_cast<unsigned>(ctas)), dim3(L::kThreads), L::kBytes, stream, p);
}

unsigned blocks_for(int64_t items, int64_t per_block, int64_t most) {
  const int64_t n = (items + per_block - 1) / per_block;
  return static_cast<unsigned>(n < most ? n : most);
}

}  // namespace

extern "C" {

fp8q_status fp8q_rope_frequencies(double* freq, int64_t rot_dim, double theta, const fp8q_rope_scaling* scaling) {
  if (!freq || rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > 65536) return FP8Q_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !(theta < 1e300)) return FP8Q_ERR_INVALID_ARG;   // also rejects NaN
  const int type = scaling ? scaling->type : FP8Q_ROPE_UNSCALED;
  const double pi2 = 2.0 * 3.14159265358979323846;
  double factor = 1.0, low = 0.0, high = 0.0;
  if (type != FP8Q_ROPE_UNSCALED) {
    factor = scaling->factor;
    if (!(factor >= 1.0) || !(factor < 1e300)) return FP8Q_ERR_INVALID_ARG;
  }
  if (type == FP8Q_ROPE_LLAMA3 || type == FP8Q_ROPE_YARN) {
    if (!(scaling->original_max_position >= 1.0) || !(scaling->original_max_position < 1e300))
      return FP8Q_ERR_INVALID_ARG;
    if (!(scaling->low > 0.0) || !(scaling->high > scaling->low) || !(scaling->high < 1e300))
      return FP8Q_ERR_INVALID_ARG;
  }
  switch (type) {
    case FP8Q_ROPE_UNSCALED:
    case FP8Q_ROPE_LINEAR:
    case FP8Q_ROPE_LLAMA3: break;
    case FP8Q_ROPE_YARN: {
      // the (fractional) pair index whose frequency makes n turns over the original context
      auto index = [&](double n) {
        return rot_dim * std::log(scaling->original_max_position / (n * pi2)) / (2.0 * std::log(theta));
      };
      low = std::floor(index(scaling->high));
      high = std::ceil(index(scaling->low));
      if (low < 0.0) low = 0.0;
      if (high > rot_dim - 1.0) high = rot_dim - 1.0;
      if (!(high > low)) high = low + 0.001;
      break;
    }
    default: return FP8Q_ERR_INVALID_ARG;
  }
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(theta, -2.0 * static_cast<double>(i) / static_cast<double>(rot_dim));
    double keep = 1.0;                                     // share of f that is not stretched
    if (type == FP8Q_ROPE_LINEAR) keep = 0.0;
    if (type == FP8Q_ROPE_LLAMA3) {
      const double turns = scaling->original_max_position * f / pi2;
      keep = (turns - scaling->low) / (scaling->high - scaling->low);
    }
    if (type == FP8Q_ROPE_YARN) keep = 1.0 - (static_cast<double>(i) - low) / (high - low);
    keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
    freq[i] = keep * f + (1.0 - keep) * (f / factor);
  }
  return FP8Q_OK;
}

fp8q_status fp8q_rope(const void* X_bf16, int64_t T, int64_t H, int64_t D, int64_t x_token_stride,
                      int64_t x_head_stride, const int64_t* positions, const double* freq, int64_t rot_dim, int flags,
                      float mscale, void* Y_bf16, int64_t y_token_stride, int64_t y_head_stride, void* stream) {
  if (T < 0 || H <= 0 || D <= 0) return FP8Q_ERR_INVALID_ARG;
  if (rot_dim <= 0 || rot_dim > D || rot_dim % 2 != 0) return FP8Q_ERR_INVALID_ARG;
  if (T == 0) return FP8Q_OK;
  fp8q_status st = check_rope(positions, freq, rot_dim, D, flags, mscale);
  if (st != FP8Q_OK) return st;
  if (!X_bf16 || !Y_bf16) return FP8Q_ERR_INVALID_ARG;
  if (bad_strides(T, H, x_token_stride, x_head_stride) || bad_strides(T, H, y_token_stride, y_head_stride))
    return FP8Q_ERR_INVALID_ARG;
  if (T > kInt32Max || H > 65536 || D > 65536 || T * H > kInt32Max) return FP8Q_ERR_UNSUPPORTED;
  if (rows_overlap(T, H, D, y_token_stride, y_head_stride)) return FP8Q_ERR_INVALID_ARG;
  if (X_bf16 == Y_bf16 && ((T > 1 && x_token_stride != y_token_stride) || (H > 1 && x_head_stride != y_head_stride)))
    return FP8Q_ERR_INVALID_ARG;
  if (!aligned(X_bf16, 2) || !aligned(Y_bf16, 2)) return FP8Q_ERR_MISALIGNED;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != FP8Q_OK) return st;
  fp8q::rope::Params p;
  p.x = static_cast<const uint16_t*>(X_bf16);
  p.y = static_cast<uint16_t*>(Y_bf16);
  p.pos = positions;
  p.freq = freq;
  p.xt = x_token_stride;
  p.xh = x_head_stride;
  p.yt = y_token_stride;
  p.yh = y_head_stride;
  p.T = static_cast<int>(T);
  p.H = static_cast<int>(H);
  p.D = static_cast<int>(D);
  p.R = static_cast<int>(rot_dim);
  p.m = mscale;
  p.interleaved = (flags & FP8Q_ROPE_INTERLEAVED) != 0;
  p.inverse = (flags & FP8Q_ROPE_INVERSE) != 0;
  // 16-byte rows take the vector kernel; anything else, one pair a thread
  const bool vec = rot_dim % 16 == 0 && D % 8 == 0 && rot_dim <= 1024 && aligned(X_bf16, 16) && aligned(Y_bf16, 16) &&
                   (T == 1 || (x_token_stride % 8 == 0 && y_token_stride % 8 == 0)) &&
                   (H == 1 || (x_head_stride % 8 == 0 && y_head_stride % 8 == 0));
  if (!vec)
    return launch(fp8q::rope::rope_any_kernel, dim3(blocks_for(T * H * (rot_dim / 2), 256, 8ll * sms)), dim3(256), 0,
                  stream, p);
  // Four tokens a CTA share the launch and the angles where that still gives every SM several CTAs; a few tokens are
  // spread over the SMs by heads instead.
  const int tokens = T >= 16ll * sms ? 4 : 1;
  const int64_t units = H * (rot_dim / 16);
  int64_t split = T < sms ? (units + 255) / 256 : 1;
  if (split > H) split = H;
  const dim3 grid(static_cast<unsigned>((T + tokens - 1) / tokens), static_cast<unsigned>(split));
  const size_t bytes = static_cast<size_t>(tokens) * (rot_dim / 2) * sizeof(float2);
  auto k = p.interleaved ? fp8q::rope::rope_vec_kernel<true> : fp8q::rope::rope_vec_kernel<false>;
  return launch(k, grid, dim3(256), bytes, stream, p, tokens);
}

size_t fp8q_kv4_page_bytes(int64_t page_size, int64_t kv_heads, int64_t head_dim) {
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return 0;
  if (kv_heads <= 0 || kv_heads > 4096 || (head_dim != 64 && head_dim != 128)) return 0;
  return static_cast<size_t>(page_size * kv_heads * (head_dim * 9 / 16));
}

fp8q_status fp8q_kv4_append(const fp8q_kv4_cache* cache, const void* K_bf16, int64_t k_token_stride,
                            int64_t k_head_stride, const void* V_bf16, int64_t v_token_stride, int64_t v_head_stride,
                            const int64_t* slots, int64_t T, const int64_t* positions, const double* freq,
                            int64_t rot_dim, int flags, float mscale, void* stream) {
  fp8q_status st = check_cache(cache);
  if (st != FP8Q_OK) return st;
  if (T < 0) return FP8Q_ERR_INVALID_ARG;
  if (T == 0) return FP8Q_OK;
  if ((st = check_rows(K_bf16, T, cache->kv_heads, k_token_stride, k_head_stride)) != FP8Q_OK) return st;
  if ((st = check_rows(V_bf16, T, cache->kv_heads, v_token_stride, v_head_stride)) != FP8Q_OK) return st;
  if (!slots) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return FP8Q_ERR_MISALIGNED;
  if (positions || freq) {
    if (flags & FP8Q_ROPE_INVERSE) return FP8Q_ERR_INVALID_ARG;
    if ((st = check_rope(positions, freq, rot_dim, cache->head_dim, flags, mscale)) != FP8Q_OK) return st;
    if (rot_dim % 8 != 0) return FP8Q_ERR_UNSUPPORTED;
  }
  if (T > kInt32Max / (2 * cache->kv_heads)) return FP8Q_ERR_UNSUPPORTED;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != FP8Q_OK) return st;
  fp8q::kv4::AppendParams p;
  p.c = device_cache(cache);
  p.k = static_cast<const uint16_t*>(K_bf16);
  p.v = static_cast<const uint16_t*>(V_bf16);
  p.kt = k_token_stride;
  p.kh = k_head_stride;
  p.vt = v_token_stride;
  p.vh = v_head_stride;
  p.slots = slots;
  p.pos = positions;
  p.freq = freq;
  p.T = static_cast<int>(T);
  p.R = positions ? static_cast<int>(rot_dim) : 0;
  p.interleaved = (flags & FP8Q_ROPE_INTERLEAVED) != 0;
  p.m = mscale;
  auto k = cache->head_dim == 64 ? fp8q::kv4::append_kernel<64> : fp8q::kv4::append_kernel<128>;
  const int tokens = T >= 16ll * sms ? 4 : 1;      // as in fp8q_rope
  return launch(k, dim3(blocks_for(T, tokens, kInt32Max)), dim3(256),
                static_cast<size_t>(tokens) * (cache->head_dim / 2) * sizeof(double2), stream, p, tokens);
}

fp8q_status fp8q_kv4_read(const fp8q_kv4_cache* cache, const int64_t* slots, int64_t T, void* K_bf16,
                          int64_t k_token_stride, int64_t k_head_stride, void* V_bf16, int64_t v_token_stride,
                          int64_t v_head_stride, void* stream) {
  fp8q_status st = check_cache(cache);
  if (st != FP8Q_OK) return st;
  if (T < 0) return FP8Q_ERR_INVALID_ARG;
  if (T == 0) return FP8Q_OK;
  if ((st = check_rows(K_bf16, T, cache->kv_heads, k_token_stride, k_head_stride)) != FP8Q_OK) return st;
  if ((st = check_rows(V_bf16, T, cache->kv_heads, v_token_stride, v_head_stride)) != FP8Q_OK) return st;
  if (rows_overlap(T, cache->kv_heads, cache->head_dim, k_token_stride, k_head_stride) ||
      rows_overlap(T, cache->kv_heads, cache->head_dim, v_token_stride, v_head_stride))
    return FP8Q_ERR_INVALID_ARG;
  if (!slots) return FP8Q_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return FP8Q_ERR_MISALIGNED;
  if (T > kInt32Max / (2 * cache->kv_heads)) return FP8Q_ERR_UNSUPPORTED;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != FP8Q_OK) return st;
  fp8q::kv4::ReadParams p;
  p.c = device_cache(cache);
  p.slots = slots;
  p.k = static_cast<uint16_t*>(K_bf16);
  p.v = static_cast<uint16_t*>(V_bf16);
  p.kt = k_token_stride;
  p.kh = k_head_stride;
  p.vt = v_token_stride;
  p.vh = v_head_stride;
  p.T = static_cast<int>(T);
  const int64_t items = 2 * T * cache->kv_heads * (cache->head_dim / 16);
  auto k = cache->head_dim == 64 ? fp8q::kv4::read_kernel<64> : fp8q::kv4::read_kernel<128>;
  return launch(k, dim3(blocks_for(items, 256, kInt32Max)), dim3(256), 0, stream, p);
}

size_t fp8q_kv4_attention_workspace_size(const fp8q_kv4_cache* cache, int64_t B, int64_t T, int64_t Hq,
                                         int64_t max_q_len) {
  if (check_cache(cache) != FP8Q_OK || B <= 0 || T <= 0 || Hq <= 0 || max_q_len <= 0) return 0;
  if (Hq % cache->kv_heads != 0 || T > kInt32Max || Hq > 65536 || T * Hq > kInt32Max || B > 65536) return 0;
  int dev, sms;
  if (current_device(&dev, &sms) != FP8Q_OK) return 0;
  return attention_plan(cache, T, Hq, max_q_len, sms).bytes();
}

fp8q_status fp8q_kv4_attention(const fp8q_kv4_cache* cache, const void* Q_bf16, int64_t q_token_stride,
                               int64_t q_head_stride, int64_t T, int64_t Hq, const int32_t* page_table,
                               int64_t table_stride, int64_t max_pages, const int32_t* kv_len, const int32_t* q_start,
                               int64_t B, int64_t max_q_len, float sm_scale, int causal, int64_t window,
                               void* O_bf16, int64_t o_token_stride, int64_t o_head_stride, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  fp8q_status st = check_cache(cache);
  if (st != FP8Q_OK) return st;
  if (T < 0 || B < 0 || Hq <= 0 || max_q_len <= 0 || max_pages < 0 || window < 0) return FP8Q_ERR_INVALID_ARG;
  if (Hq % cache->kv_heads != 0 || (causal != 0 && causal != 1)) return FP8Q_ERR_INVALID_ARG;
  if (!finite_positive(sm_scale) || !(sm_scale * cache->k_scale < 1.0e38f)) return FP8Q_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return FP8Q_OK;
  if (!q_start && (T < B || max_q_len != 1)) return FP8Q_ERR_INVALID_ARG;
  if ((st = check_rows(Q_bf16, T, Hq, q_token_stride, q_head_stride)) != FP8Q_OK) return st;
  if ((st = check_rows(O_bf16, T, Hq, o_token_stride, o_head_stride)) != FP8Q_OK) return st;
  if (rows_overlap(T, Hq, cache->head_dim, o_token_stride, o_head_stride)) return FP8Q_ERR_INVALID_ARG;
  // (a table without a page needs no memory: every sequence is empty)
  if ((!page_table && max_pages > 0) || !kv_len || (B > 1 && table_stride < max_pages)) return FP8Q_ERR_INVALID_ARG;
  if (!workspace) return FP8Q_ERR_INVALID_ARG;   // its size needs the device; presence and alignment do not
  if (!aligned(page_table, 4) || !aligned(kv_len, 4) || !aligned(q_start, 4) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return FP8Q_ERR_MISALIGNED;
  if (T > kInt32Max || Hq > 65536 || T * Hq > kInt32Max || B > 65536 || table_stride > kStrideMax ||
      max_pages > kInt32Max || max_pages * cache->page_size > kInt32Max - 65536)   // (keys past a length are ints too)
    return FP8Q_ERR_UNSUPPORTED;
  // the kernels count items in 23 bits and steps in 40
  const int64_t items = B * cache->kv_heads * attention_plan(cache, T, Hq, max_q_len, 1).row_tiles;
  if (items >= (1 << 22) || items * (max_pages * cache->page_size / 128 + 8) >= (static_cast<int64_t>(1) << 39))
    return FP8Q_ERR_UNSUPPORTED;
  int dev, sms;
  if ((st = current_device(&dev, &sms)) != FP8Q_OK) return st;
  fp8q::kv4::AttnParams p;
  p.c = device_cache(cache);
  p.q = static_cast<const uint16_t*>(Q_bf16);
  p.o = static_cast<uint16_t*>(O_bf16);
  p.lse = lse;
  p.table = page_table;
  p.kv_len = kv_len;
  p.q_start = q_start;
  p.qt = q_token_stride;
  p.qh = q_head_stride;
  p.ot = o_token_stride;
  p.oh = o_head_stride;
  p.table_stride = table_stride;
  p.T = static_cast<int>(T);
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.group = static_cast<int>(Hq / cache->kv_heads);
  p.max_pages = static_cast<int>(max_pages);
  p.max_q = static_cast<int>(max_q_len < T ? max_q_len : T);
  p.scale = sm_scale * cache->k_scale * 1.44269504088896340736f;
  p.causal = causal;
  p.window = window;
  const AttentionPlan plan = attention_plan(cache, T, Hq, max_q_len, sms);
  if (workspace_bytes < plan.bytes()) return FP8Q_ERR_INVALID_ARG;
  p.count = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWorkspaceHeader);
  p.row_tiles = plan.row_tiles;
  // No more CTAs than there can be steps of 128 keys: CTAs without work are not free, and where they fill the SMs the
  // few that have some come to share an SM (64 rows of 8 heads over 500 keys: 16 -> 12 us).
  int64_t keys = max_pages * cache->page_size;
  if (window > 0 && window < keys - p.max_q - 128) keys = window + p.max_q + 128;
  const int64_t steps = items * ((keys + 127) / 128 + 1);
  const int ctas = static_cast<int>(plan.ctas < steps ? plan.ctas : steps);
  if (cache->head_dim == 128) {
    if (plan.nt == 1) return launch_few<128, 1, 4>(p, ctas, dev, stream);
    if (plan.nt == 2) return launch_few<128, 2, 3>(p, ctas, dev, stream);
    return launch_many<128>(p, ctas, dev, stream);
  }
  if (plan.nt == 1) return launch_few<64, 1, 5>(p, ctas, dev, stream);
  if (plan.nt == 2) return launch_few<64, 2, 3>(p, ctas, dev, stream);
  return launch_many<64>(p, ctas, dev, stream);
}

}  // extern "C"
