// dsel_logits: penalties for repeated tokens, biases and a grammar mask on the
// rows that dsel_topk_sample draws from.
//
// Per row, with c[v] = how often v occurs among the row's answer tokens and
// seen[v] = whether it occurs in its prompt or answer:
//   y = float(x[v]);  seen[v]: y = y > 0 ? y / repetition : y * repetition
//   y = y - frequency * c[v] - presence * [c[v] > 0];  y = y + (the row's biases of v, in list order)
//   y = -inf where the mask's bit v is 0, and in the columns that pad the row
//
// What bounds it: the logits are read once and written once (HBM), a row's tokens
// are a few KB.  So one CTA owns a slice of a row's vocabulary: its logits go to
// registers first (the loads fly while the rest is done), the row's tokens are
// counted into shared memory (one 32-bit word per vocabulary entry of the slice:
// integer atomics, so the result does not depend on their order), and one pass
// over the registers applies everything and writes the row.  Every CTA of a row
// scans the row's tokens itself: they come from L2, and a scan costs a few
// instructions per token against a second launch and a count array in HBM.
//
// Measured (one B200, 256 rows of 129,280 f32, up to 16,384 tokens each): 95.5 us, of which
// the stream alone takes 42.1 (the copy rate), the mask 3, the biases 7, the scans 18 and
// the entries they met 17 to 25: bound by instructions (64% of issue slots busy).  Tried and
// dropped: penalties written sparsely after a pure stream (134 us: each phase waits for
// the one before), prompt and answer in two branch-free scans (117 us), a warp of its own
// for the biases (102 us), scans shared in clusters of eight through distributed shared memory
// (126 us).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dsel_ops.cuh"

namespace dsel {
namespace {

// 256 threads: with 512 (slices of 8,192, half the scans) 256 rows take 90.4 us, but 64 rows 20.5 against 19.4
// and one row 3.7 against 3.3.
constexpr int kLgThreads = 256;
constexpr int kLgVecs = 4;                            // vectors of 4 elements each thread holds
constexpr int kLgSlice = kLgThreads * kLgVecs * 4;    // vocabulary entries of a CTA
constexpr uint32_t kInPrompt = 0x80000000u;           // count word: seen in the prompt; low bits: answer count

struct LogitsParams {
  const void* x;
  int64_t x_stride;
  const void* tokens;
  int64_t tokens_stride;
  const int32_t* prompt_len;
  const int32_t* total_len;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_offsets;
  const int32_t* bias_ids;
  const float* bias_values;
  int64_t bias_count;
  const uint32_t* mask;
  int64_t mask_stride;
  int64_t mask_count;
  const int32_t* mask_rows;
  float* out;
  int64_t out_stride;
  int32_t vocab;
  int32_t width;
  int32_t slices;   // CTAs per row
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 b = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xFFFF0000u), __uint_as_float(b.y << 16),
                     __uint_as_float(b.y & 0xFFFF0000u));
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Counts the row's first `to` tokens that fall in [base, base + len).  Each CTA of a row scans them all, so a
// token costs a quarter of a load, a subtraction and a comparison.
struct Counter {
  uint32_t* counts;
  int32_t base;
  uint32_t len;
  int32_t prompt;
  __device__ __forceinline__ void add(int32_t id, int32_t i) const {
    const uint32_t d = uint32_t(id) - uint32_t(base);   // (an id below base, or negative, wraps past len)
    if (d < len) {
      if (i < prompt)
        atomicOr(&counts[d], kInPrompt);
      else
        atomicAdd(&counts[d], 1u);
    }
  }
  __device__ __forceinline__ void add(int64_t id, int32_t i) const {
    if (id >= 0 && id <= INT32_MAX) add(int32_t(id), i);
  }
};

__device__ __forceinline__ void count_tokens(const int64_t* __restrict__ t, int32_t to, const Counter& c) {
  constexpr int kUnroll = 8;
  for (int32_t i0 = int32_t(threadIdx.x); i0 < to; i0 += kLgThreads * kUnroll) {
    int64_t id[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) id[u] = i0 + u * kLgThreads < to ? t[i0 + u * kLgThreads] : -1;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) c.add(id[u], i0 + u * kLgThreads);
  }
}

__device__ __forceinline__ void count_tokens(const int32_t* __restrict__ t, int32_t to, const Counter& c) {
  constexpr int kUnroll = 4;
  const int32_t off = int32_t((16u - (reinterpret_cast<uintptr_t>(t) & 15u)) & 15u) / 4;   // up to a 16-byte boundary
  const int32_t head = off < to ? off : to;
  const int32_t quads = (to - head) / 4, tail = head + quads * 4;
  const int32_t tid = int32_t(threadIdx.x);
  if (tid < head) c.add(t[tid], tid);
  if (tid < to - tail) c.add(t[tail + tid], tail + tid);
  const int4* q = reinterpret_cast<const int4*>(t + head);
  for (int32_t i0 = tid; i0 < quads; i0 += kLgThreads * kUnroll) {
    int4 id[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      id[u] = i0 + u * kLgThreads < quads ? q[i0 + u * kLgThreads] : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t dx = uint32_t(id[u].x) - uint32_t(c.base), dy = uint32_t(id[u].y) - uint32_t(c.base);
      const uint32_t dz = uint32_t(id[u].z) - uint32_t(c.base), dw = uint32_t(id[u].w) - uint32_t(c.base);
      if (min(min(dx, dy), min(dz, dw)) >= c.len) continue;   // none of the four is in the slice
      const int32_t i = head + (i0 + u * kLgThreads) * 4;
      c.add(id[u].x, i);
      c.add(id[u].y, i + 1);
      c.add(id[u].z, i + 2);
      c.add(id[u].w, i + 3);
    }
  }
}

template <typename T, typename tok_t, bool kAligned>
__global__ void __launch_bounds__(kLgThreads) logits_kernel(const __grid_constant__ LogitsParams p) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* counts = smem;                                         // [kLgSlice]
  float* bias = reinterpret_cast<float*>(smem + kLgSlice);         // [kLgSlice], only when the call has biases
  const int64_t row = blockIdx.x / uint32_t(p.slices);
  const int32_t slice = int32_t(blockIdx.x - row * p.slices);
  const int32_t base = slice * kLgSlice;
  const int32_t tid = int32_t(threadIdx.x);

  for (int i = tid; i < kLgSlice / 4; i += kLgThreads) {
    reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
    if (p.bias_ids != nullptr) reinterpret_cast<uint4*>(bias)[i] = make_uint4(0, 0, 0, 0);
  }
  grid_wait();   // nothing above touches global memory

  // the row's numbers, then the slice's logits: all on their way before anything is waited for
  const float rep = p.repetition != nullptr ? p.repetition[row] : 1.f;
  const float freq = p.frequency != nullptr ? p.frequency[row] : 0.f;
  const float pres = p.presence != nullptr ? p.presence[row] : 0.f;
  int32_t total = p.total_len != nullptr ? p.total_len[row] : p.width;
  const int32_t prompt = p.prompt_len != nullptr ? p.prompt_len[row] : 0;
  int64_t mrow = -1, b0 = 0, b1 = 0;
  if (p.mask != nullptr) mrow = p.mask_rows != nullptr ? int64_t(p.mask_rows[row]) : row;
  if (p.bias_ids != nullptr) {
    b0 = p.bias_offsets[row];
    b1 = p.bias_offsets[row + 1];
  }
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  float4 y[kLgVecs];
#pragma unroll
  for (int j = 0; j < kLgVecs; ++j) {
    const int32_t e = base + (j * kLgThreads + tid) * 4;
    if (kAligned && e + 4 <= p.vocab) {
      y[j] = load4<T>(x + e);
    } else {
      y[j].x = e + 0 < p.vocab ? load1(x + e + 0) : 0.f;
      y[j].y = e + 1 < p.vocab ? load1(x + e + 1) : 0.f;
      y[j].z = e + 2 < p.vocab ? load1(x + e + 2) : 0.f;
      y[j].w = e + 3 < p.vocab ? load1(x + e + 3) : 0.f;
    }
  }
  // the mask's words of those vectors (bits of one vector lie in one word)
  uint32_t allowed[kLgVecs];
  const bool masked = mrow >= 0 && mrow < p.mask_count;
#pragma unroll
  for (int j = 0; j < kLgVecs; ++j) {
    const int32_t e = base + (j * kLgThreads + tid) * 4;
    allowed[j] = 0xFu;
    if (masked && e < p.vocab) allowed[j] = p.mask[mrow * p.mask_stride + (e >> 5)] >> (e & 31);
    const int32_t left = p.vocab - e;   // columns from vocab on are never allowed
    if (left < 4) allowed[j] &= left > 0 ? (1u << left) - 1u : 0u;
  }

  // A positive logit is divided as a product with the reciprocal: two roundings for one, but a division for
  // each element took a third of the kernel's instructions.
  const float inverse = 1.f / rep;
  const int32_t slice_end = p.vocab - base < kLgSlice ? p.vocab : base + kLgSlice;
  b0 = b0 < 0 ? 0 : b0;
  b1 = b1 > p.bias_count ? p.bias_count : b1;
  const bool biased = b0 < b1;
  // neutral penalties change no logit, so such a row's tokens are not read
  const bool counted = p.tokens != nullptr && (rep != 1.f || freq != 0.f || pres != 0.f) && base < p.vocab;
  __syncthreads();   // the count words are zero
  // biases: one warp walks the row's list, so repeated entries add up in list order
  if (biased) {
    if (tid < 32) {
      for (int64_t b = b0; b < b1; b += 32) {
        const bool in = b + tid < b1;
        const int32_t id = in ? p.bias_ids[b + tid] : -1;
        const float v = in ? p.bias_values[b + tid] : 0.f;
        const bool mine = id >= base && id < slice_end;
        if (!__any_sync(0xFFFFFFFFu, mine)) continue;
        uint32_t same = __match_any_sync(0xFFFFFFFFu, mine ? id : -1 - tid);
        const bool first = mine && (__ffs(same) - 1) == tid;
        float sum = first ? bias[id - base] : 0.f;
        while (__any_sync(0xFFFFFFFFu, same != 0u)) {
          const int src = same != 0u ? __ffs(same) - 1 : tid;
          const float add = __shfl_sync(0xFFFFFFFFu, v, src);
          if (same != 0u) sum += add;
          same &= same - 1u;
        }
        if (first) bias[id - base] = sum;
        __syncwarp();
      }
    }
  }
  if (counted) {
    total = total < 0 ? 0 : (total > p.width ? p.width : total);
    const Counter c = {counts, base, uint32_t(slice_end - base), prompt};
    count_tokens(static_cast<const tok_t*>(p.tokens) + row * p.tokens_stride, total, c);
  }
  __syncthreads();
  grid_launch();   // a dependent launch may begin its own set-up

  float* out = p.out + row * p.out_stride;
  const float ninf = -__int_as_float(0x7F800000);
#pragma unroll
  for (int j = 0; j < kLgVecs; ++j) {
    const int32_t o = (j * kLgThreads + tid) * 4;
    const int32_t e = base + o;
    if (e >= p.out_stride) break;
    float v[4] = {y[j].x, y[j].y, y[j].z, y[j].w};
    if (counted) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(counts + o);
      const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
      if ((c4.x | c4.y | c4.z | c4.w) != 0u) {   // few: but some lane of a warp mostly has one, so no branches within
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t n = c[i] & ~kInPrompt;
          const float seen = v[i] * (v[i] > 0.f ? inverse : rep);
          const float less = n != 0u ? freq * float(n) + pres : 0.f;
          v[i] = c[i] != 0u ? seen - less : v[i];
        }
      }
    }
    if (biased) {
      const float4 b = *reinterpret_cast<const float4*>(bias + o);
      v[0] += b.x, v[1] += b.y, v[2] += b.z, v[3] += b.w;
    }
    float4 r;
    r.x = (allowed[j] & 1u) != 0u ? v[0] : ninf;
    r.y = (allowed[j] & 2u) != 0u ? v[1] : ninf;
    r.z = (allowed[j] & 4u) != 0u ? v[2] : ninf;
    r.w = (allowed[j] & 8u) != 0u ? v[3] : ninf;
    *reinterpret_cast<float4*>(out + e) = r;   // out_stride is a multiple of 16
  }
}

template <typename T, typename tok_t>
int launch_logits(const LogitsParams& p, int64_t rows, bool aligned, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> allowed[2];
  const uint32_t smem = kLgSlice * 4 * (p.bias_ids != nullptr ? 2 : 1);
  auto kern = aligned ? logits_kernel<T, tok_t, true> : logits_kernel<T, tok_t, false>;
  if (allow_smem(reinterpret_cast<const void*>(kern), 2 * kLgSlice * 4, dev, &allowed[aligned]) != cudaSuccess) return DSEL_ERR_CUDA;
  return launch_dependent(kern, unsigned(rows * p.slices), kLgThreads, 1, smem, st, p) == cudaSuccess ? DSEL_OK
                                                                                                      : DSEL_ERR_CUDA;
}

}  // namespace
}  // namespace dsel

using namespace dsel;

DSEL_API int dsel_logits(const void* x, int dtype, int64_t rows, int32_t vocab, int64_t x_stride, const void* tokens,
                         int token_dtype, int32_t width, int64_t tokens_stride, const int32_t* prompt_len,
                         const int32_t* total_len, const float* repetition, const float* frequency,
                         const float* presence, const int32_t* bias_offsets, const int32_t* bias_ids,
                         const float* bias_values, int64_t bias_count, const void* mask, int64_t mask_stride,
                         int64_t mask_count, const int32_t* mask_rows, float* out, int64_t out_stride, void* stream) {
  if (dtype != DSEL_BF16 && dtype != DSEL_F32) return DSEL_ERR_DTYPE;
  if (rows < 0) return DSEL_ERR_ROWS;
  if (vocab < 1 || vocab > INT32_MAX - 16 * kLgSlice) return DSEL_ERR_SHAPE;
  if (x_stride < vocab || out_stride < vocab || out_stride % kStrideReq != 0 || out_stride > INT32_MAX - 16 * kLgSlice)
    return DSEL_ERR_STRIDE;
  if (tokens != nullptr) {
    if (token_dtype != DSEL_I32 && token_dtype != DSEL_I64) return DSEL_ERR_INDEX_DTYPE;
    if (width < 0 || width > INT32_MAX - 16 * kLgThreads) return DSEL_ERR_SHAPE;
    if (tokens_stride < width) return DSEL_ERR_STRIDE;
  }
  if (bias_count < 0 || mask_count < 0) return DSEL_ERR_SHAPE;
  if (mask != nullptr) {
    if (mask_stride < (int64_t(vocab) + 31) / 32) return DSEL_ERR_STRIDE;
    if (mask_rows == nullptr && mask_count < rows) return DSEL_ERR_SHAPE;
  }
  if (rows == 0) return DSEL_OK;
  if (x == nullptr || out == nullptr) return DSEL_ERR_NULL;
  if ((bias_ids == nullptr) != (bias_offsets == nullptr) || (bias_ids == nullptr) != (bias_values == nullptr))
    return DSEL_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(out) & 15u) != 0) return DSEL_ERR_ALIGN;
  const int eb = dtype == DSEL_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(x) & uintptr_t(eb - 1)) != 0) return DSEL_ERR_ALIGN;
  const int32_t slices = int32_t((out_stride + kLgSlice - 1) / kLgSlice);
  if (rows > INT32_MAX / slices) return DSEL_ERR_ROWS;
  // in place only where every element is read and written by one thread
  if (ranges_meet(x, (rows - 1) * x_stride + vocab, eb, out, rows * out_stride, 4) &&
      !(x == out && dtype == DSEL_F32 && (x_stride == out_stride || rows == 1)))   // (one row: no stride counts)
    return DSEL_ERR_OVERLAP;
  LogitsParams p = {};
  p.slices = slices;
  int dev = 0, sms = 0;
  if (const int st = current_device(&dev, &sms); st != DSEL_OK) return st;
  p.x = x;
  p.x_stride = x_stride;
  p.tokens = width > 0 ? tokens : nullptr;
  p.tokens_stride = tokens_stride;
  p.prompt_len = prompt_len;
  p.total_len = total_len;
  p.repetition = repetition;
  p.frequency = frequency;
  p.presence = presence;
  p.bias_offsets = bias_offsets;
  p.bias_ids = bias_count > 0 ? bias_ids : nullptr;
  p.bias_values = bias_values;
  p.bias_count = bias_count;
  p.mask = static_cast<const uint32_t*>(mask);
  p.mask_stride = mask_stride;
  p.mask_count = mask_count;
  p.mask_rows = mask_rows;
  p.out = out;
  p.out_stride = out_stride;
  p.vocab = vocab;
  p.width = width;
  // a vector of 4 elements at every 4th column: 16 bytes of f32, 8 of bf16
  const bool aligned = (reinterpret_cast<uintptr_t>(x) % uintptr_t(4 * eb)) == 0 && (x_stride % 4 == 0 || rows == 1);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool wide = token_dtype == DSEL_I64;
  if (dtype == DSEL_BF16)
    return wide ? launch_logits<__nv_bfloat16, int64_t>(p, rows, aligned, dev, cs)
                : launch_logits<__nv_bfloat16, int32_t>(p, rows, aligned, dev, cs);
  return wide ? launch_logits<float, int64_t>(p, rows, aligned, dev, cs) : launch_logits<float, int32_t>(p, rows, aligned, dev, cs);
}
