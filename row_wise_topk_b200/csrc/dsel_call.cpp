// dsel_call: the serving operators with their arguments in an array of 8-byte words.
#include <cstdint>
#include <cstring>

#include "../../include/dsel.h"

namespace {

// Reads the words in order; an int32 argument's word must fit it.
struct Words {
  const unsigned char* at;
  bool fits = true;
  int64_t wide() {
    int64_t w;
    std::memcpy(&w, at, 8);
    at += 8;
    return w;
  }
  int32_t narrow() {
    const int64_t w = wide();
    if (w < INT32_MIN || w > INT32_MAX) fits = false;
    return static_cast<int32_t>(w);
  }
  float real() {
    double d;
    std::memcpy(&d, at, 8);
    at += 8;
    return static_cast<float>(d);
  }
  template <typename T>
  T* pointer() {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(wide()));
  }
};

int logits(Words w) {
  auto* x = w.pointer<const void>();
  const int dtype = w.narrow();
  const int64_t rows = w.wide();
  const int32_t vocab = w.narrow();
  const int64_t x_stride = w.wide();
  auto* tokens = w.pointer<const void>();
  const int token_dtype = w.narrow();
  const int32_t width = w.narrow();
  const int64_t tokens_stride = w.wide();
  auto* prompt_len = w.pointer<const int32_t>();
  auto* total_len = w.pointer<const int32_t>();
  auto* repetition = w.pointer<const float>();
  auto* frequency = w.pointer<const float>();
  auto* presence = w.pointer<const float>();
  auto* bias_offsets = w.pointer<const int32_t>();
  auto* bias_ids = w.pointer<const int32_t>();
  auto* bias_values = w.pointer<const float>();
  const int64_t bias_count = w.wide();
  auto* mask = w.pointer<const void>();
  const int64_t mask_stride = w.wide();
  const int64_t mask_count = w.wide();
  auto* mask_rows = w.pointer<const int32_t>();
  auto* out = w.pointer<float>();
  const int64_t out_stride = w.wide();
  auto* stream = w.pointer<void>();
  if (!w.fits) return DSEL_ERR_SHAPE;
  return dsel_logits(x, dtype, rows, vocab, x_stride, tokens, token_dtype, width, tokens_stride, prompt_len,
                     total_len, repetition, frequency, presence, bias_offsets, bias_ids, bias_values, bias_count,
                     mask, mask_stride, mask_count, mask_rows, out, out_stride, stream);
}

int index_score(Words w) {
  auto* q = w.pointer<const void>();
  const int dtype = w.narrow();
  const int64_t tokens = w.wide();
  const int32_t heads = w.narrow();
  const int32_t dim = w.narrow();
  const int64_t q_token_stride = w.wide();
  const int64_t q_head_stride = w.wide();
  auto* weights = w.pointer<const float>();
  const int64_t weights_stride = w.wide();
  auto* keys = w.pointer<const void>();
  const int32_t pages = w.narrow();
  const int32_t page_size = w.narrow();
  const int64_t page_stride = w.wide();
  const int64_t key_stride = w.wide();
  auto* key_scale = w.pointer<const float>();
  const int64_t scale_page_stride = w.wide();
  auto* table = w.pointer<const int32_t>();
  const int32_t seqs = w.narrow();
  const int32_t table_width = w.narrow();
  const int64_t table_stride = w.wide();
  auto* seq_ids = w.pointer<const int32_t>();
  auto* end = w.pointer<const int32_t>();
  auto* out = w.pointer<void>();
  const int out_dtype = w.narrow();
  const int64_t row_stride = w.wide();
  auto* stream = w.pointer<void>();
  if (!w.fits) return DSEL_ERR_SHAPE;
  return dsel_index_score(q, dtype, tokens, heads, dim, q_token_stride, q_head_stride, weights, weights_stride, keys,
                          pages, page_size, page_stride, key_stride, key_scale, scale_page_stride, table, seqs,
                          table_width, table_stride, seq_ids, end, out, out_dtype, row_stride, stream);
}

int sparse_attn(Words w) {
  auto* q = w.pointer<const void>();
  const int dtype = w.narrow();
  const int64_t tokens = w.wide();
  const int32_t q_heads = w.narrow();
  const int32_t kv_heads = w.narrow();
  const int32_t dim = w.narrow();
  const int64_t q_token_stride = w.wide();
  const int64_t q_head_stride = w.wide();
  auto* k = w.pointer<const void>();
  auto* v = w.pointer<const void>();
  const int32_t pages = w.narrow();
  const int32_t page_size = w.narrow();
  const int64_t k_page_stride = w.wide();
  const int64_t k_row_stride = w.wide();
  const int64_t k_head_stride = w.wide();
  const int64_t v_page_stride = w.wide();
  const int64_t v_row_stride = w.wide();
  const int64_t v_head_stride = w.wide();
  auto* table = w.pointer<const int32_t>();
  const int32_t seqs = w.narrow();
  const int32_t table_width = w.narrow();
  const int64_t table_stride = w.wide();
  auto* seq_ids = w.pointer<const int32_t>();
  auto* end = w.pointer<const int32_t>();
  auto* indices = w.pointer<const void>();
  const int index_dtype = w.narrow();
  const int32_t take = w.narrow();
  const int64_t idx_token_stride = w.wide();
  const int64_t idx_head_stride = w.wide();
  const int32_t block = w.narrow();
  const float scale = w.real();
  auto* out = w.pointer<void>();
  auto* lse = w.pointer<float>();
  auto* stream = w.pointer<void>();
  if (!w.fits) return DSEL_ERR_SHAPE;
  return dsel_sparse_attn(q, dtype, tokens, q_heads, kv_heads, dim, q_token_stride, q_head_stride, k, v, pages,
                          page_size, k_page_stride, k_row_stride, k_head_stride, v_page_stride, v_row_stride,
                          v_head_stride, table, seqs, table_width, table_stride, seq_ids, end, indices, index_dtype,
                          take, idx_token_stride, idx_head_stride, block, scale, out, lse, stream);
}

}  // namespace

DSEL_API int dsel_call(int call, const void* words) {
  if (words == nullptr) return DSEL_ERR_NULL;
  const Words w = {static_cast<const unsigned char*>(words)};
  switch (call) {
    case DSEL_CALL_LOGITS: return logits(w);
    case DSEL_CALL_INDEX_SCORE: return index_score(w);
    case DSEL_CALL_SPARSE_ATTN: return sparse_attn(w);
    default: return DSEL_ERR_UNAVAILABLE;
  }
}
