// The serving operators' entry points with their arguments in one array of
// 64-bit words: a call through a foreign-function interface that converts every
// argument on its own costs less with one (ctypes: 0.1 us an argument).
#include <cstdint>
#include <cstring>

#include "tq_internal.h"

namespace {

// The words of a call, taken one after the other.
struct Words {
  const unsigned char *at;
  bool fits = true;  // every integer so far fits its argument
  explicit Words(const void *words) : at(static_cast<const unsigned char *>(words)) {}
  template <typename W>
  W next() {
    W w;
    std::memcpy(&w, at, sizeof w);
    at += sizeof w;
    return w;
  }
  // a pointer, a 32-bit integer, a 64-bit one, a size, a floating-point number
  template <typename T>
  T *ptr() {
    return reinterpret_cast<T *>((uintptr_t)next<uint64_t>());
  }
  int32_t i32() {
    const int64_t w = next<int64_t>();
    fits = fits && w >= INT32_MIN && w <= INT32_MAX;
    return (int32_t)w;
  }
  int64_t i64() { return next<int64_t>(); }
  size_t size() { return (size_t)next<uint64_t>(); }
  float f32() { return (float)next<double>(); }
};

tq_status too_large(const char *call) {
  return tq::report_error(TQ_ERR_INVALID, "%s: an integer does not fit 32 bits", call);
}

}  // namespace

extern "C" {

tq_status tq_decode_attention_shared_words(const void *words) {
  if (!words) return tq::report_error(TQ_ERR_INVALID, "words is NULL");
  Words w(words);
  tq_ctx *ctx = w.ptr<tq_ctx>();
  const tq_cache *cache = w.ptr<const tq_cache>();
  const void *q = w.ptr<const void>();
  const int32_t q_dtype = w.i32(), n_q_heads = w.i32();
  const int32_t *seq_lens = w.ptr<const int32_t>(), *cu_group = w.ptr<const int32_t>();
  const int32_t *prefix_lens = w.ptr<const int32_t>();
  const int32_t n_groups = w.i32(), max_group = w.i32(), max_prefix = w.i32(), max_suffix = w.i32();
  const float scale = w.f32();
  void *out = w.ptr<void>();
  const int32_t out_dtype = w.i32();
  float *lse = w.ptr<float>();
  void *workspace = w.ptr<void>();
  const size_t workspace_bytes = w.size();
  void *stream = w.ptr<void>();
  if (!w.fits) return too_large("tq_decode_attention_shared");
  return tq_decode_attention_shared(ctx, cache, q, q_dtype, n_q_heads, seq_lens, cu_group, prefix_lens, n_groups,
                                    max_group, max_prefix, max_suffix, scale, out, out_dtype, lse, workspace,
                                    workspace_bytes, stream);
}

tq_status tq_prompt_attention_words(const void *words) {
  if (!words) return tq::report_error(TQ_ERR_INVALID, "words is NULL");
  Words w(words);
  tq_ctx *ctx = w.ptr<tq_ctx>();
  const void *q = w.ptr<const void>(), *k = w.ptr<const void>(), *v = w.ptr<const void>();
  const int64_t q_stride = w.i64(), k_stride = w.i64(), v_stride = w.i64();
  const int32_t n_tok = w.i32(), n_q_heads = w.i32(), n_kv_heads = w.i32();
  const int32_t *cu_seqlens = w.ptr<const int32_t>();
  const int32_t n_seqs = w.i32(), max_len = w.i32();
  const float scale = w.f32();
  void *out = w.ptr<void>();
  const int32_t out_dtype = w.i32();
  float *lse = w.ptr<float>();
  void *stream = w.ptr<void>();
  if (!w.fits) return too_large("tq_prompt_attention");
  return tq_prompt_attention(ctx, q, k, v, q_stride, k_stride, v_stride, n_tok, n_q_heads, n_kv_heads, cu_seqlens, n_seqs,
                             max_len, scale, out, out_dtype, lse, stream);
}

tq_status tq_build_tables_words(const void *words) {
  if (!words) return tq::report_error(TQ_ERR_INVALID, "words is NULL");
  Words w(words);
  tq_ctx *ctx = w.ptr<tq_ctx>();
  const tq_cache *cache = w.ptr<const tq_cache>();
  int32_t *block_table = w.ptr<int32_t>();
  const int32_t *cached_lens = w.ptr<const int32_t>(), *new_lens = w.ptr<const int32_t>();
  const int32_t *free_list = w.ptr<const int32_t>();
  const int32_t n_free = w.i32();
  const int32_t *free_start = w.ptr<const int32_t>();
  int32_t *free_end = w.ptr<int32_t>();
  const int32_t *cu_group = w.ptr<const int32_t>(), *prefix_lens = w.ptr<const int32_t>();
  const int32_t n_groups = w.i32(), n_tok = w.i32();
  int32_t *seq_idx = w.ptr<int32_t>(), *pos = w.ptr<int32_t>();
  int64_t *slots = w.ptr<int64_t>();
  int32_t *cu_new = w.ptr<int32_t>(), *seq_lens = w.ptr<int32_t>();
  void *stream = w.ptr<void>();
  if (!w.fits) return too_large("tq_build_tables");
  return tq_build_tables(ctx, cache, block_table, cached_lens, new_lens, free_list, n_free, free_start, free_end,
                         cu_group, prefix_lens, n_groups, n_tok, seq_idx, pos, slots, cu_new, seq_lens, stream);
}

}  // extern "C"
