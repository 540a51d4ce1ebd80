// dsel_sparse_attn: attention of each query over the cached blocks that its TopK
// indices name.
//
//   z[n] = scale * q[t][h] . k[n]   over the listed positions n < end[t]
//   o[t][h] = sum_n exp(z[n] - m) v[n] / sum_n exp(z[n] - m),   lse = m + log(sum)
//
// What bounds it: every query has its own list, so the keys and values are gathered
// once per (query, key head): 4 * dim bytes for 4 * dim * group operations (group =
// query heads that share a key head), far below what the tensor cores need.  The work
// is to keep enough gathers in flight.  So the list of a (query, key head) is dealt out
// in tiles of 16 or 32 positions to the key groups (one or more warps) of a cluster of
// up to eight CTAs; each group runs its own ring of 16-byte asynchronous copies and its
// own running reference (near the maximum) and sum, with no barrier but its own; the
// groups' partial sums meet once, at the end, through distributed shared memory (one
// launch, no workspace).
// A group has a warp for every 16 query heads: legacy m16n8k16 products, since a tile
// has 16 to 64 rows and its operands arrive row by row in any order.
//
// Probabilities are rounded to the operands' type for the product with v (the matrix
// instruction takes both of one type); their sum is kept of the float32 values.  float16
// ends at 2^-25, so there they are taken 2^11 times as large: else the terms of a long list
// far below its largest score would be in the sum and not in the product.
//
// Measured (one B200): 64 queries of 32 heads over 4, 32 blocks of 64 positions each 47 us
// (269 MB, 0.88 of the copy rate); 1,024 queries of one sequence over 16 such blocks
// 230 us (the 2.1 GB that they gather come out of L2 at 9.3 TB/s; 440 instructions a tile
// of 16 bound it); 64 queries of 64 heads over one, 512 positions each 13.6 us (latency: the
// index, the page, the row, then the join, each a round trip).
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dsel_ops.cuh"

namespace dsel {
namespace {

constexpr int kAtWarps = 4;
constexpr int kAtThreads = kAtWarps * 32;
// Positions per tile.  A group of one warp owns a whole ring, so its tiles are small: the four rings of a CTA take
// 96 KB with three stages (two CTAs an SM) and 64 KB with two (three CTAs); with tiles of 32 one CTA fitted,
// and a 1,024-query chunk took 443 us.  Groups of two and four warps share theirs.
constexpr int at_tile(int row_warps) { return row_warps == 1 ? 16 : 32; }
constexpr int kAtSm = 228 * 1024;   // shared memory of an SM
constexpr int kAtMaxStages = 3;
constexpr int kAtMaxCluster = 8;
constexpr int kPitchPad = 8;       // floats: rows of the partial sums fall on different banks

struct AttnParams {
  const uint8_t* q;
  int64_t q_token_bytes, q_head_bytes;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_page_bytes, k_row_bytes, k_head_bytes;
  int64_t v_page_bytes, v_row_bytes, v_head_bytes;
  const int32_t* table;
  int64_t table_stride;
  const void* indices;
  int64_t idx_token_stride, idx_head_stride;
  const int32_t* seq_ids;
  const int32_t* end;
  void* out;
  float* lse;
  float scale_log2;     // |scale| * log2(e): the softmax runs on powers of two
  uint32_t q_flip;      // sign bits of a pair of 16-bit values where scale < 0
  uint32_t q_keep;      // no bits where scale is 0: the products are, and scale_log2 is 1
  int32_t idx_i64;
  int32_t pages, page_size, page_shift;
  int32_t seqs, table_width, seq_mode;
  int32_t kv_heads, group, row_tiles;
  int32_t take, block, block_shift;
  int32_t tiles;        // tiles of the whole list
  int32_t rows_even;    // places lie row_bytes apart across pages too, in k as in v: one 32-bit place says where
  int32_t stages;
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool kBf16>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Warps that share a key group: its own barrier, or none for a single warp.
template <int kRowWarps>
__device__ __forceinline__ void group_sync(int group) {
  if (kRowWarps == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kRowWarps * 32) : "memory");
}

// Position in its sequence of entry l of the list, or -1: none, or behind `end`.
__device__ __forceinline__ int32_t list_position(const AttnParams& p, const void* idx, int32_t l, int32_t end) {
  if (p.block_shift >= 0 && !p.idx_i64) {   // the plain case in 32 bits: an index that passes the test gives a position
    const int32_t j = l >> p.block_shift;
    if (j >= p.take) return -1;
    const uint32_t i = static_cast<const uint32_t*>(idx)[j];
    if (end <= 0 || i > uint32_t(end - 1) >> p.block_shift) return -1;
    const int32_t pos = int32_t(i << p.block_shift) + (l - (j << p.block_shift));
    return pos < end ? pos : -1;
  }
  const int32_t j = l / p.block;
  if (j >= p.take) return -1;
  const int64_t i = p.idx_i64 ? static_cast<const int64_t*>(idx)[j] : int64_t(static_cast<const int32_t*>(idx)[j]);
  if (i < 0 || i > int64_t(end)) return -1;
  const int64_t pos = i * p.block + (l - j * p.block);
  return pos < int64_t(end) ? int32_t(pos) : -1;
}

// The page of a position and its place in it; page < 0: none.
struct Place {
  int32_t page, row;
};
__device__ __forceinline__ Place locate(const AttnParams& p, const int32_t* table, int32_t pos) {
  Place at = {-1, 0};
  if (pos >= 0) {
    const int32_t i = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
    if (i < p.table_width) at.page = table[i];
    if (at.page >= p.pages) at.page = -1;
    at.row = pos - i * p.page_size;
  }
  return at;
}

template <bool kBf16, int kDim, int kRowWarps>
__global__ void __launch_bounds__(kAtThreads, kRowWarps == 1 ? 3 : 1) attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kGroups = kAtWarps / kRowWarps;          // key groups of the CTA
  constexpr int kRows = 16 * kRowWarps;                  // query heads of the CTA
  constexpr int kRowBytes = kDim * 2;
  constexpr int kPieces = kRowBytes / 16;
  constexpr int kAtTile = at_tile(kRowWarps);
  constexpr int kTileBytes = kAtTile * kRowBytes;        // keys of a tile; its values follow
  constexpr int kPitch = kDim + kPitchPad;
  // How far (in powers of two) a score may lie above its row's reference, and what a probability of 1 is in the
  // product with v.  In float16 both together stay below 2^16: terms down to 2^-36 count, each within 2^-36.
  constexpr float kAhead = kBf16 ? 8.f : 4.f;
  constexpr float kUnit = kBf16 ? 1.f : 2048.f;
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  const int grp = warp / kRowWarps, rw = warp % kRowWarps;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int32_t unit = int32_t(blockIdx.x / ranks);
  const int32_t rt = unit % p.row_tiles;
  const int32_t th = unit / p.row_tiles;
  const int32_t kvh = th % p.kv_heads;
  const int32_t t = th / p.kv_heads;
  grid_wait();
  grid_launch();

  int32_t end = p.end[t];
  const int32_t seq = p.seq_mode == 0 ? p.seq_ids[t] : (p.seq_mode == 1 ? t : 0);
  if (seq < 0 || seq >= p.seqs) end = 0;
  const int32_t* table = p.table + (end > 0 ? int64_t(seq) * p.table_stride : 0);
  const int64_t idx_off = int64_t(t) * p.idx_token_stride + int64_t(kvh) * p.idx_head_stride;
  const void* idx = static_cast<const uint8_t*>(p.indices) + idx_off * (p.idx_i64 ? 8 : 4);
  const uint8_t* kbase = p.k + int64_t(kvh) * p.k_head_bytes;
  const uint8_t* vbase = p.v + int64_t(kvh) * p.v_head_bytes;

  // this warp's query heads as A fragments (with a negative scale their negatives: scores then only grow with
  // the products, and the maximum is that of the products)
  const int row0 = rt * kRows + rw * 16;    // first head of the group
  uint32_t qf[kDim / 16][4];
  {
    const uint8_t* qb = p.q + int64_t(t) * p.q_token_bytes + (lane & 3) * 4;
    const int ra = row0 + (lane >> 2), rb = ra + 8;
    const uint8_t* qa = qb + int64_t(kvh * p.group + ra) * p.q_head_bytes;
    const uint8_t* qc = qb + int64_t(kvh * p.group + rb) * p.q_head_bytes;
#pragma unroll
    for (int s = 0; s < kDim / 16; ++s) {
      qf[s][0] = ra < p.group ? *reinterpret_cast<const uint32_t*>(qa + s * 32) : 0u;
      qf[s][1] = rb < p.group ? *reinterpret_cast<const uint32_t*>(qc + s * 32) : 0u;
      qf[s][2] = ra < p.group ? *reinterpret_cast<const uint32_t*>(qa + s * 32 + 16) : 0u;
      qf[s][3] = rb < p.group ? *reinterpret_cast<const uint32_t*>(qc + s * 32 + 16) : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[s][i] = (qf[s][i] ^ p.q_flip) & p.q_keep;
    }
  }

  float o[kDim / 8][4];
#pragma unroll
  for (int i = 0; i < kDim / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m0 = -__int_as_float(0x7F800000), m1 = m0, l0 = 0.f, l1 = 0.f;

  const uint32_t ring = shared_addr(smem) + uint32_t(grp * p.stages) * (2 * kTileBytes);
  const int32_t step = int32_t(ranks) * kGroups;
  const int32_t first = int32_t(rank) * kGroups + grp;
  const int32_t mine = p.tiles > first ? (p.tiles - first + step - 1) / step : 0;   // tiles of this group

  // Two loads lie between a list entry and its rows (the index, the page): each is fetched ahead of its use,
  // 32 entries (one a lane) at a time.
  constexpr int kBatch = 32 / kAtTile;     // tiles of a look-up
  auto entry = [&](int32_t i) {            // this lane's position in the group's tiles i .. i + kBatch - 1
    const int32_t tile = i + lane / kAtTile;
    return tile < mine ? list_position(p, idx, (first + tile * step) * kAtTile + lane % kAtTile, end) : -1;
  };
  int32_t pos_next = entry(0);
  Place at = {-1, 0};
  uint32_t exist = 0u;                     // bit l: lane l's position of the look-up exists
  int32_t slot = -1;
  constexpr int kPerPass = 32 / kPieces;   // rows that a warp copies at once
  constexpr uint32_t kFullTile = kAtTile == 32 ? 0xFFFFFFFFu : (1u << kAtTile) - 1u;
  const int piece = lane % kPieces, my_row = rw * (kAtTile / kRowWarps) + lane / kPieces;
  uint32_t put[4];                         // where a lane's piece of row my_row + kPerPass * j lies in a tile (j mod 4)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = my_row + kPerPass * j;
    put[j] = uint32_t(row) * kRowBytes + (uint32_t(piece ^ (row & 7)) << 4);
  }
  const uint8_t* kpiece = kbase + piece * 16;
  const uint8_t* vpiece = vbase + piece * 16;
  uint32_t fill = ring;                    // the stage that is filled next
  const uint32_t ring_end = ring + uint32_t(p.stages) * (2 * kTileBytes);
  auto issue = [&](int32_t i) -> uint32_t {   // starts the copies of the group's tile i; which of its positions exist
    const uint32_t dst = fill;
    fill += 2 * kTileBytes;
    if (fill == ring_end) fill = ring;
    if (i >= mine) return 0u;
    const int sub = kBatch > 1 ? i % kBatch : 0;
    if (sub == 0) {
      at = locate(p, table, pos_next);
      pos_next = entry(i + kBatch);
      exist = __ballot_sync(0xFFFFFFFFu, at.page >= 0);
      slot = at.page >= 0 && p.rows_even ? at.page * p.page_size + at.row : -1;
    }
    const uint32_t any = (exist >> (sub * kAtTile)) & kFullTile;
    if (any == 0u) return 0u;
    const int from = sub * kAtTile + my_row;   // the lane that knows this lane's first row
    if (p.rows_even && any == kFullTile) {
#pragma unroll
      for (int j = 0; j < kAtTile / kRowWarps / kPerPass; ++j) {
        const int32_t s = __shfl_sync(0xFFFFFFFFu, slot, from + kPerPass * j);
        const int64_t o = int64_t(s) * int32_t(p.k_row_bytes);
        const uint32_t to = dst + put[j & 3] + uint32_t((j >> 2) * 4 * kPerPass * kRowBytes);
        copy16(to, kpiece + o);
        copy16(to + kTileBytes, vpiece + o);
      }
    } else {
#pragma unroll 2
      for (int j = 0; j < kAtTile / kRowWarps / kPerPass; ++j) {
        const int64_t page = __shfl_sync(0xFFFFFFFFu, at.page, from + kPerPass * j);
        const int64_t place = __shfl_sync(0xFFFFFFFFu, at.row, from + kPerPass * j);
        const int row = my_row + kPerPass * j;
        const uint32_t to = dst + uint32_t(row) * kRowBytes + (uint32_t(piece ^ (row & 7)) << 4);
        const bool in = page >= 0;
        copy16(to, in ? kpiece + page * p.k_page_bytes + place * p.k_row_bytes : p.k, in);
        copy16(to + kTileBytes, in ? vpiece + page * p.v_page_bytes + place * p.v_row_bytes : p.v, in);
      }
    }
    return any;
  };

  // Where this lane's rows of the operand fragments lie in a tile: of keys for the product with q (rows as
  // they are), of values for the product with the probabilities (transposed on the way); depth step d: j = d mod 4.
  uint32_t key_at[4], value_at[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t kr = uint32_t((lane & 7) + ((lane >> 4) << 3)), vr = uint32_t(lane & 15);
    key_at[j] = kr * kRowBytes + (((uint32_t(2 * j) + ((lane >> 3) & 1u)) ^ (lane & 7u)) << 4);
    value_at[j] = kTileBytes + vr * kRowBytes + (((uint32_t(2 * j) + (uint32_t(lane) >> 4)) ^ (lane & 7u)) << 4);
  }
  constexpr float kNone = -__builtin_huge_valf();

  uint32_t live[kAtMaxStages];   // which positions of the tiles in flight exist
#pragma unroll
  for (int s = 0; s < kAtMaxStages; ++s) live[s] = 0u;
#pragma unroll
  for (int s = 0; s < kAtMaxStages - 1; ++s) {
    if (s < p.stages - 1) live[s] = issue(s);
    copy_commit();
  }
  uint32_t tile_at = ring;
  for (int32_t i = 0; i < mine; ++i) {
    // (with fewer than kAtMaxStages stages the ring is only that deep: the newest group is this tile's own)
    const uint32_t newest = issue(i + p.stages - 1);
    copy_commit();
    if (p.stages == 3) {
      live[2] = newest;
      copy_wait<2>();
    } else if (p.stages == 2) {
      live[1] = newest;
      copy_wait<1>();
    } else {
      live[0] = newest;
      copy_wait<0>();
    }
    group_sync<kRowWarps>(grp);
    const uint32_t here = live[0], kt = tile_at;
    live[0] = live[1];
    live[1] = live[2];
    tile_at += 2 * kTileBytes;
    if (tile_at == ring_end) tile_at = ring;
    if (here != 0u) {
      constexpr bool kSplit = kAtTile == 16;   // two sums of half the depth each: shorter chains where there are few
      float s[kAtTile / 8][4], s2[kSplit ? kAtTile / 8 : 1][4];
#pragma unroll
      for (int n = 0; n < kAtTile / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = 0.f;
          if (kSplit) s2[n][e] = 0.f;
        }
#pragma unroll
      for (int d = 0; d < kDim / 16; ++d) {
#pragma unroll
        for (int n = 0; n < kAtTile / 16; ++n) {   // 16 keys: two column tiles, both halves of the depth
          uint32_t b[4];
          ldmatrix4(kt + key_at[d & 3] + uint32_t(n * 16 * kRowBytes + (d >> 2) * 128), b);
          mma16816<kBf16>(kSplit && (d & 1) != 0 ? s2[2 * n] : s[2 * n], qf[d], b[0], b[1]);
          mma16816<kBf16>(kSplit && (d & 1) != 0 ? s2[2 * n + 1] : s[2 * n + 1], qf[d], b[2], b[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < kAtTile / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kSplit) s[n][e] += s2[n][e];
      if (here != kFullTile) {   // positions that do not exist do not count
        const uint32_t cols = here >> ((lane & 3) * 2);
#pragma unroll
        for (int n = 0; n < kAtTile / 8; ++n) {
          if (((cols >> (n * 8)) & 1u) == 0u) s[n][0] = s[n][2] = kNone;
          if (((cols >> (n * 8 + 1)) & 1u) == 0u) s[n][1] = s[n][3] = kNone;
        }
      }
      float x0 = m0, x1 = m1;
#pragma unroll
      for (int n = 0; n < kAtTile / 8; ++n) {
        x0 = fmaxf(x0, fmaxf(s[n][0], s[n][1]));
        x1 = fmaxf(x1, fmaxf(s[n][2], s[n][3]));
      }
      x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 2));
      // The reference m of a row moves only where a score is 2^kAhead above it: terms and sums then are at most that
      // much larger, which no type here minds, and the sums of nearly every tile need no new factor (with a move for
      // every new maximum some row of a warp had one in most tiles).
      const bool up0 = (x0 - m0) * p.scale_log2 > kAhead, up1 = (x1 - m1) * p.scale_log2 > kAhead;
      if (__any_sync(0xFFFFFFFFu, up0 || up1)) {
        // (a row without a score so far has m = -inf and holds zeros)
        const float f0 = up0 ? pow2((m0 - x0) * p.scale_log2) : 1.f, f1 = up1 ? pow2((m1 - x1) * p.scale_log2) : 1.f;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < kDim / 8; ++n) {
          o[n][0] *= f0;
          o[n][1] *= f0;
          o[n][2] *= f1;
          o[n][3] *= f1;
        }
        m0 = up0 ? x0 : m0;
        m1 = up1 ? x1 : m1;
      }
      // (product - reference) * scale
      const float z0 = m0 == kNone ? 0.f : m0, z1 = m1 == kNone ? 0.f : m1;
#pragma unroll
      for (int n = 0; n < kAtTile / 8; ++n) {
        s[n][0] = pow2((s[n][0] - z0) * p.scale_log2);
        s[n][1] = pow2((s[n][1] - z0) * p.scale_log2);
        s[n][2] = pow2((s[n][2] - z1) * p.scale_log2);
        s[n][3] = pow2((s[n][3] - z1) * p.scale_log2);
        l0 += s[n][0] + s[n][1];
        l1 += s[n][2] + s[n][3];
      }
#pragma unroll
      for (int n = 0; n < kAtTile / 16; ++n) {
        const uint32_t a[4] = {pack16<kBf16>(s[2 * n][0] * kUnit, s[2 * n][1] * kUnit),
                               pack16<kBf16>(s[2 * n][2] * kUnit, s[2 * n][3] * kUnit),
                               pack16<kBf16>(s[2 * n + 1][0] * kUnit, s[2 * n + 1][1] * kUnit),
                               pack16<kBf16>(s[2 * n + 1][2] * kUnit, s[2 * n + 1][3] * kUnit)};
#pragma unroll
        for (int d = 0; d < kDim / 16; ++d) {
          uint32_t b[4];
          ldmatrix4t(kt + value_at[d & 3] + uint32_t(n * 16 * kRowBytes + (d >> 2) * 128), b);
          mma16816<kBf16>(o[2 * d], a, b[0], b[1]);
          mma16816<kBf16>(o[2 * d + 1], a, b[2], b[3]);
        }
      }
    }
    group_sync<kRowWarps>(grp);   // the stage may be filled again
  }
  copy_wait<0>();
  l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 1);
  l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 2);
  l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 1);
  l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 2);

  // ---- the groups' partial sums meet ----
  __syncthreads();   // the rings are no longer read
  float* part = reinterpret_cast<float*>(smem);                       // [kGroups][kRows][kPitch]
  float* ml = part + kGroups * kRows * kPitch;                        // [kGroups][kRows][2]: maximum, sum
  float* wt = ml + kGroups * kRows * 2;                               // [ranks * kGroups][kRows], then [kRows] totals
  {
    const int r = rw * 16 + (lane >> 2);
    float* pa = part + (grp * kRows + r) * kPitch + (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < kDim / 8; ++n) {
      *reinterpret_cast<float2*>(pa + n * 8) = make_float2(o[n][0], o[n][1]);
      *reinterpret_cast<float2*>(pa + 8 * kPitch + n * 8) = make_float2(o[n][2], o[n][3]);
    }
    if ((lane & 3) == 0) {
      ml[(grp * kRows + r) * 2] = m0;
      ml[(grp * kRows + r) * 2 + 1] = l0;
      ml[(grp * kRows + r + 8) * 2] = m1;
      ml[(grp * kRows + r + 8) * 2 + 1] = l1;
    }
  }
  if (ranks > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const int64_t out0 = int64_t(t) * p.kv_heads * p.group + kvh * p.group;   // the key head's first row of the output
  if (ranks == 1) {   // all parts are here
    for (int i = int(threadIdx.x); i < kRows * kDim / 4; i += kAtThreads) {
      const int r = i / (kDim / 4), c = (i % (kDim / 4)) * 4;
      const int head = rt * kRows + r;
      if (head >= p.group) continue;
      float2 x[kGroups];
      float top = kNone, sum = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        x[g] = *reinterpret_cast<const float2*>(ml + (g * kRows + r) * 2);
        top = fmaxf(top, x[g].x);
      }
      const float z = top == kNone ? 0.f : top;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float f = pow2((x[g].x - z) * p.scale_log2);
        const float4 b = *reinterpret_cast<const float4*>(part + (g * kRows + r) * kPitch + c);
        sum += x[g].y * f;
        a.x += b.x * f;
        a.y += b.y * f;
        a.z += b.z * f;
        a.w += b.w * f;
      }
      const float inv = sum == 0.f ? 0.f : (1.f / kUnit) / sum;
      const uint2 y = make_uint2(pack16<kBf16>(a.x * inv, a.y * inv), pack16<kBf16>(a.z * inv, a.w * inv));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + ((out0 + head) * kDim + c) * 2) = y;
      if (c == 0 && p.lse != nullptr)
        p.lse[out0 + head] = sum == 0.f ? kNone : (z * p.scale_log2 + log2f(sum)) * 0.6931471805599453f;
    }
    return;
  }
  // Remote loads are issued four at a time: one takes as long as the four.
  const int parts = int(ranks) * kGroups;                             // at least 2, a power of two
  float* sums = wt + parts * kRows;                                   // [parts][kRows] sums, then [kRows] totals
  float* total = sums + parts * kRows;
  if (int(threadIdx.x) < kRows) {
    const int r = int(threadIdx.x);
    float top = kNone;
    for (int i = 0; i < parts; i += 4) {
      float2 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = i + j < parts ? i + j : parts - 1;
        x[j] = peer_load2(peer_addr(shared_addr(ml + ((k % kGroups) * kRows + r) * 2), uint32_t(k / kGroups)));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = i + j < parts ? i + j : parts - 1;
        wt[k * kRows + r] = x[j].x;
        sums[k * kRows + r] = x[j].y;
        top = fmaxf(top, x[j].x);
      }
    }
    const float z = top == kNone ? 0.f : top;
    float sum = 0.f;
    for (int i = 0; i < parts; ++i) {
      const float f = pow2((wt[i * kRows + r] - z) * p.scale_log2);
      wt[i * kRows + r] = f;
      sum += sums[i * kRows + r] * f;
    }
    total[r] = sum;
    const int head = rt * kRows + r;
    if (rank == 0 && p.lse != nullptr && head < p.group)
      p.lse[out0 + head] = sum == 0.f ? kNone : (z * p.scale_log2 + log2f(sum)) * 0.6931471805599453f;
  }
  __syncthreads();
  for (int i = int(rank) * kAtThreads + int(threadIdx.x); i < kRows * kDim / 4; i += int(ranks) * kAtThreads) {
    const int r = i / (kDim / 4), c = (i % (kDim / 4)) * 4;
    const int head = rt * kRows + r;
    if (head >= p.group) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t here_at = shared_addr(part + r * kPitch + c);
    for (int j = 0; j < parts; j += 4) {
      float4 x[4];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        const int k = j + q4 < parts ? j + q4 : parts - 1;
        x[q4] = peer_load4(peer_addr(here_at, uint32_t(k / kGroups)) + uint32_t((k % kGroups) * kRows * kPitch * 4));
      }
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        if (j + q4 < parts) {
          const float f = wt[(j + q4) * kRows + r];
          a.x += x[q4].x * f;
          a.y += x[q4].y * f;
          a.z += x[q4].z * f;
          a.w += x[q4].w * f;
        }
      }
    }
    const float sum = total[r];
    const float inv = sum == 0.f ? 0.f : (1.f / kUnit) / sum;
    const uint2 y = make_uint2(pack16<kBf16>(a.x * inv, a.y * inv), pack16<kBf16>(a.z * inv, a.w * inv));
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + ((out0 + head) * kDim + c) * 2) = y;
  }
  cluster_sync_all();   // no CTA leaves while a peer may still read its sums
}

template <bool kBf16, int kDim, int kRowWarps>
int launch_attn(AttnParams p, int64_t units, int dev, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> allowed;
  auto kern = attn_kernel<kBf16, kDim, kRowWarps>;
  constexpr int kGroups = kAtWarps / kRowWarps;
  constexpr int kStageBytes = kGroups * 2 * at_tile(kRowWarps) * kDim * 2;
  p.tiles = int32_t((int64_t(p.take) * p.block + at_tile(kRowWarps) - 1) / at_tile(kRowWarps));
  // CTAs per (query, key head): as many as fill the SMs twice, but none without a tile for each of its groups
  int cluster = 1;
  while (cluster < kAtMaxCluster && units * cluster * 2 <= int64_t(sms) * 2 && cluster * 2 * kGroups <= p.tiles) cluster *= 2;
  const int64_t each = (p.tiles + int64_t(cluster) * kGroups - 1) / (int64_t(cluster) * kGroups);
  // Three stages keep the most copies in flight of CTAs that all run at once; where there are more, two let three
  // CTAs of single-warp groups share an SM (1,024-query chunk 309 -> 244 us; 256 CTAs at once 51 -> 54 us).
  const int most = kRowWarps == 1 && units * cluster > 2 * int64_t(sms) ? 2 : kAtMaxStages;
  p.stages = each < 1 ? 1 : (each > most ? most : int(each));
  const int merge = kAtWarps * 16 * (kDim + kPitchPad + 2) * 4 + (2 * cluster * kGroups + 1) * 16 * kRowWarps * 4;
  int smem = p.stages * kStageBytes > merge ? p.stages * kStageBytes : merge;
  // Few CTAs are spread over the SMs by asking for so much that no SM takes more than its share (64 queries x 512
  // keys of 64 heads, clusters of four: 14.0 us, and 17.2 where three CTAs fit an SM and clusters crowd some).
  const int64_t share = (units * cluster + sms - 1) / sms;
  if (share <= 2 && smem < kAtSm / int(share + 1) + 1024) smem = kAtSm / int(share + 1) + 1024;
  if (units * cluster > INT32_MAX) return DSEL_ERR_ROWS;
  if (allow_smem(reinterpret_cast<const void*>(kern), kAtSm / 2 + 1024, dev, &allowed) != cudaSuccess)
    return DSEL_ERR_CUDA;
  return launch_dependent(kern, unsigned(units * cluster), kAtThreads, cluster, uint32_t(smem), st, p) == cudaSuccess
             ? DSEL_OK
             : DSEL_ERR_CUDA;
}

template <bool kBf16, int kDim>
int launch_rows(AttnParams& p, int64_t tokens, int dev, int sms, cudaStream_t st) {
  // a warp for every 16 heads that share keys, up to 64 rows a CTA
  const int rows = p.group <= 16 ? 16 : p.group <= 32 ? 32 : 64;
  p.row_tiles = (p.group + rows - 1) / rows;
  const int64_t units = tokens * p.kv_heads * p.row_tiles;
  if (rows == 16) return launch_attn<kBf16, kDim, 1>(p, units, dev, sms, st);
  if (rows == 32) return launch_attn<kBf16, kDim, 2>(p, units, dev, sms, st);
  return launch_attn<kBf16, kDim, 4>(p, units, dev, sms, st);
}

int log2_of(int32_t n) {
  for (int s = 0; s < 31; ++s)
    if ((int64_t(1) << s) == n) return s;
  return -1;
}

}  // namespace
}  // namespace dsel

using namespace dsel;

DSEL_API int dsel_sparse_attn(const void* q, int dtype, int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t dim,
                              int64_t q_token_stride, int64_t q_head_stride, const void* k, const void* v,
                              int32_t pages, int32_t page_size, int64_t k_page_stride, int64_t k_row_stride,
                              int64_t k_head_stride, int64_t v_page_stride, int64_t v_row_stride,
                              int64_t v_head_stride, const int32_t* table, int32_t seqs, int32_t table_width,
                              int64_t table_stride, const int32_t* seq_ids, const int32_t* end, const void* indices,
                              int index_dtype, int32_t take, int64_t idx_token_stride, int64_t idx_head_stride,
                              int32_t block, float scale, void* out, float* lse, void* stream) {
  if (dtype != DSEL_BF16 && dtype != DSEL_F16) return DSEL_ERR_DTYPE;
  if (index_dtype != DSEL_I32 && index_dtype != DSEL_I64) return DSEL_ERR_INDEX_DTYPE;
  if (tokens < 0 || tokens > INT32_MAX / 2) return DSEL_ERR_ROWS;
  if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || (dim != 64 && dim != 128)) return DSEL_ERR_SHAPE;
  if (pages < 0 || page_size < 1 || seqs < 0 || table_width < 0) return DSEL_ERR_SHAPE;
  if (seq_ids == nullptr && seqs != 1 && int64_t(seqs) != tokens) return DSEL_ERR_SHAPE;
  if (take < 0 || block < 1 || int64_t(take) * block > INT32_MAX / 2) return DSEL_ERR_SHAPE;
  if (q_head_stride < dim || q_token_stride < 0 || k_page_stride < 0 || v_page_stride < 0 || k_row_stride < dim ||
      v_row_stride < dim || k_head_stride < 0 || v_head_stride < 0 || table_stride < table_width ||
      idx_token_stride < 0 || idx_head_stride < 0)
    return DSEL_ERR_STRIDE;
  if (((q_token_stride | q_head_stride | k_page_stride | k_row_stride | k_head_stride | v_page_stride | v_row_stride |
        v_head_stride) & 7) != 0)
    return DSEL_ERR_STRIDE;   // rows are copied in 16-byte pieces
  if (tokens == 0) return DSEL_OK;
  // A cache without pages, or a table without places, has no positions: no query is of any sequence, and neither is read.
  const bool no_keys = pages == 0 || seqs == 0 || table_width == 0;
  if (q == nullptr || end == nullptr || out == nullptr || (indices == nullptr && take > 0) ||
      (!no_keys && (k == nullptr || v == nullptr || table == nullptr)))
    return DSEL_ERR_NULL;
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
        reinterpret_cast<uintptr_t>(out)) & 15u) != 0)
    return DSEL_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (const int st = current_device(&dev, &sms); st != DSEL_OK) return st;
  AttnParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.q_token_bytes = q_token_stride * 2;
  p.q_head_bytes = q_head_stride * 2;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.k_page_bytes = k_page_stride * 2;
  p.k_row_bytes = k_row_stride * 2;
  p.k_head_bytes = k_head_stride * 2;
  p.v_page_bytes = v_page_stride * 2;
  p.v_row_bytes = v_row_stride * 2;
  p.v_head_bytes = v_head_stride * 2;
  p.table = table;
  p.table_stride = table_stride;
  p.indices = indices;
  p.idx_token_stride = idx_token_stride;
  p.idx_head_stride = idx_head_stride;
  p.idx_i64 = index_dtype == DSEL_I64;
  p.seq_ids = seq_ids;
  p.end = end;
  p.out = out;
  p.lse = lse;
  p.scale_log2 = float((scale < 0 ? -double(scale) : double(scale)) * 1.4426950408889634);
  p.q_flip = scale < 0 ? 0x80008000u : 0u;
  p.q_keep = 0xFFFFFFFFu;
  if (p.scale_log2 == 0.f) {   // -inf, the score of what does not exist, takes no factor of 0
    p.scale_log2 = 1.f;
    p.q_keep = 0u;
  }
  p.pages = pages;
  p.page_size = page_size;
  p.page_shift = log2_of(page_size);
  p.seqs = no_keys ? 0 : seqs;
  p.table_width = table_width;
  p.seq_mode = seq_ids != nullptr ? 0 : (seqs == 1 ? 2 : 1);
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.take = take;
  p.block = block;
  p.block_shift = log2_of(block);
  p.rows_even = k_page_stride == page_size * k_row_stride && v_page_stride == k_page_stride &&
                v_row_stride == k_row_stride && int64_t(pages) * page_size <= INT32_MAX &&
                k_row_stride * 2 <= INT32_MAX;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dtype == DSEL_BF16)
    return dim == 64 ? launch_rows<true, 64>(p, tokens, dev, sms, cs) : launch_rows<true, 128>(p, tokens, dev, sms, cs);
  return dim == 64 ? launch_rows<false, 64>(p, tokens, dev, sms, cs) : launch_rows<false, 128>(p, tokens, dev, sms, cs);
}
