// dsel_index_score: the Lightning Indexer's score of every cached key for each
// query, the rows that dsel_topk selects from.
//
//   score[t][s] = scale[s] * sum_h weights[t][h] * max(0, q[t][h] . key[s])   for s < end[t], else -inf
//
// A product of key tiles with query heads, so it runs on the tensor cores: the 128
// keys of a tile are the rows of D (one TMEM lane each), the heads of one or more
// queries its columns (one f32 column each), the head dimension is the depth.  With
// the heads in columns, the weighted sum over heads is a loop over the registers of
// the thread that owns a key: no shuffle, and its scores leave as coalesced rows.
//
// What bounds it: one query per sequence (decoding) reads 2 * dim bytes of key for
// 2 * heads * dim operations: HBM.  A chunk of queries over the same keys is bound by
// the tensor cores (2 * heads * dim operations per score), beside which the sum over
// heads costs 1.5 instructions per (key, head): the epilogue of one accumulator runs
// under the products of the other.
//
// Roles of a persistent CTA: 8 warps read accumulators, sum over heads and store; two
// bring key tiles (and one of them the queries) by TMA; one, in decoding two, issue the
// products.  Pages of a power of two of at least 8 keys are boxes of a tensor map; pages
// of other sizes end anywhere in a tile, so there the two warps address each key by
// itself and copy it in 16-byte pieces.
//
// Measured (one B200, 64 heads of 128): 64 queries over 64 K to 128 K keys each, bf16
// 254 to 259 us (1,637 MB, 0.97 to 0.98 of the copy rate), e4m3 with scales 141 us in short
// runs at full clocks to 173 us in long ones (852 MB, 0.92 to 0.75: a tile of 16 KB costs the same
// barrier round trips as one of 32); 1,024 queries over 65,536 keys 890 to 990 us, in short and
// long runs, with the power limit (1,091 GFLOP, 1,100 to 1,230 TFLOP/s).
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dsel_ops.cuh"
#include "dsel_wait.cuh"

namespace dsel {

namespace {

__device__ int g_score_status;   // DSEL_ERR_DEVICE_TIMEOUT when a wait gave up, DSEL_ERR_ALIGN: shared memory unaligned

constexpr int kTile = 128;            // keys per tile (TMEM lanes)
constexpr int kPanel = kTile * 128;   // a tile's panel: 128 rows of 128 bytes, 128-byte swizzle
constexpr int kEpiWarps = 8;
constexpr int kProdWarps = 2;
constexpr int kProdThreads = kProdWarps * 32;
constexpr int kProdKeys = kTile / kProdWarps;   // keys of a tile that a copying warp brings
constexpr int kMmaWarps = 2;
constexpr int kScThreads = (kEpiWarps + kProdWarps + kMmaWarps) * 32;
constexpr int kMaxAccs = 8;
constexpr int kMaxRing = 8;
constexpr int kScoreSmem = 227 * 1024;   // all of a CTA's shared memory
constexpr int kBarBytes = 512;          // the barriers and the accumulators' address
constexpr uint64_t kWaitLimit = 2000000000ull;   // 2 s, in ns

struct ScoreParams {
  CUtensorMap q_map;      // [tokens][heads][dim], boxes of one accumulator's queries, 128 bytes of depth
  CUtensorMap key_map;    // [pages][page_size][dim], boxes of box_keys keys; used where box_keys > 0
  int32_t box_keys;       // keys of a box: the page, or a tile of a longer one; 0: keys are copied one by one
  const float* weights;
  int64_t weights_stride;
  const uint8_t* keys;
  int64_t page_bytes, key_bytes;
  const float* key_scale;
  int64_t scale_page_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* seq_ids;
  const int32_t* end;
  void* out;
  int64_t row_stride;
  int32_t pages, page_size, page_shift;   // page_shift >= 0: page_size is 1 << page_shift
  int32_t seqs, table_width;
  int32_t tokens, heads, row_bytes;       // row_bytes: dim * element size
  int32_t col_tiles;                      // accumulators per key tile: 1 or 2
  int32_t ring, lag;                      // key tiles in shared memory; copied tiles in flight before the oldest is awaited
  int32_t q_bufs;                         // query buffers
  int32_t chunk;                          // key tiles per work item
  int32_t balanced;                       // shares instead of ranges (see Walk)
  int32_t chunks, items;
  int32_t seq_mode;                       // 0: seq_ids, 1: token t is sequence t, 2: one sequence
  int32_t out_f32;
};

// ---- PTX ----
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  return warp_wait(bar, parity, kWaitLimit, &g_score_status);
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// True in one lane of a converged warp, the same one every time (a form from which the compiler sees that
// what follows runs once: the tensor instructions take uniform registers).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0u;
}
// Shared-memory descriptor of a K-major operand in 128-byte-swizzled panels: address,
// 1024 bytes between groups of 8 rows, descriptor version 1, swizzle mode 2 (128 bytes).
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
template <bool kByte>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  if (kByte)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// A fragment of 16 keys (TMEM lanes) and 8 * N columns: in group j of 8 columns a thread gets
// columns 2 (lane % 4) and the next of keys lane / 4 (r[4j], r[4j + 1]) and lane / 4 + 8.  The
// values may be used after tmem_wait<N> on the same array.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t* r);
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t* r);   // (the registers are operands: no use moves ahead of it)
template <>
__device__ __forceinline__ void tmem_load<2>(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_wait<2>(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}
template <>
__device__ __forceinline__ void tmem_load<4>(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_wait<4>(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ float relu(uint32_t x) {   // a NaN stays one
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(__uint_as_float(x)));
  return y;
}

// a * b + c of two floats in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// A work item: up to 32 consecutive queries (one per lane) and a range of key tiles.
// Queries of one sequence that follow each other share its key tiles: a run.
struct Item {
  int32_t token0, count;   // queries of the item
  int32_t seq, end;        // this lane's query: its sequence (-1: none) and its visible keys
  uint32_t starts;         // bit i: lane i starts a run
  int32_t tile0, limit;           // first key tile
};

// Stores y as float32 or bfloat16 where `on`, without a branch: the code around it stays one block.
__device__ __forceinline__ void store_if(bool on, bool f32, uint64_t at, float y) {
  const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b16 h;\n\t"
      "setp.ne.u32 p, %0, 0;\n\tsetp.ne.u32 q, %1, 0;\n\tcvt.u16.u32 h, %4;\n\t"
      "@p st.global.b16 [%2], h;\n\t@q st.global.f32 [%2], %3;\n\t}" ::"r"(uint32_t(on && !f32)),
      "r"(uint32_t(on && f32)), "l"(at), "f"(y), "r"(h)
      : "memory");
}

// A place in a ring of `size` and how often the ring went round (its parity); no division on the way.
struct Cursor {
  uint32_t at, rounds;
  __device__ __forceinline__ void step(uint32_t size) {
    if (++at == size) {
      at = 0;
      ++rounds;
    }
  }
};

// Key tiles that query t sees.
__device__ __forceinline__ int32_t tiles_of(const ScoreParams& p, int32_t t) {
  const int32_t seq = p.seq_mode == 0 ? p.seq_ids[t] : (p.seq_mode == 1 ? t : 0);
  const int32_t end = p.end[t];
  if (seq < 0 || seq >= p.seqs || end < 0) return 0;
  return int32_t(((end > p.row_stride ? p.row_stride : int64_t(end)) + kTile - 1) / kTile);
}

// The work of a CTA, item by item: which queries, and from which of their key tiles on.
//   dealt:    ranges of `chunk` tiles of every query group, one grid apart;
//   balanced: an equal share of all queries' tiles, one after another, found by summing what each query sees
//             (one query an item).
struct Walk {
  int32_t item, group, tile0;
  int32_t left;   // balanced: tiles left of the share
  __device__ __forceinline__ bool more(const ScoreParams& p) const {
    return p.balanced ? left > 0 && group < p.tokens : item < p.items;
  }
};
__device__ __forceinline__ void deal(const ScoreParams& p, Walk& w, int32_t item) {
  w.item = item;
  w.group = item / p.chunks;
  w.tile0 = (item - w.group * p.chunks) * p.chunk;
}
__device__ __forceinline__ Walk first_walk(const ScoreParams& p) {
  Walk w = {0, 0, 0, 0};
  if (!p.balanced) {
    deal(p, w, int32_t(blockIdx.x));
    return w;
  }
  const int lane = int(threadIdx.x & 31);
  const int32_t each = (p.tokens + 31) / 32, t0 = lane * each;   // queries of a lane
  int64_t mine = 0;
  for (int32_t j = 0; j < each; ++j) mine += t0 + j < p.tokens ? tiles_of(p, t0 + j) : 0;
  int64_t upto = mine;   // tiles of this lane's queries and all before
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += v;
  }
  const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  const int64_t from = total * blockIdx.x / gridDim.x, to = total * (blockIdx.x + 1) / gridDim.x;
  if (from >= to) return w;
  const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, upto > from)) - 1;
  int64_t at = __shfl_sync(0xFFFFFFFFu, upto - mine, owner);   // tiles before the owner's queries
  w.group = owner * each;
  for (;;) {   // (ends: the owner's queries reach past `from`)
    const int32_t n = tiles_of(p, w.group);
    if (at + n > from) break;
    at += n;
    ++w.group;
  }
  w.tile0 = int32_t(from - at);
  w.left = int32_t(to - from);
  return w;
}

// What the queries of an item come with, read an item ahead of its use.
struct ItemRead {
  int32_t seq, end;
};
__device__ __forceinline__ ItemRead read_item(const ScoreParams& p, const Walk& w, int per_item) {
  ItemRead r = {-1, 0};
  const int lane = int(threadIdx.x & 31);
  const int64_t t = int64_t(w.group) * per_item + lane;
  if (w.more(p) && lane < per_item && t < p.tokens) {
    r.seq = p.seq_mode == 0 ? p.seq_ids[t] : (p.seq_mode == 1 ? int32_t(t) : 0);
    r.end = p.end[t];
  }
  return r;
}
__device__ __forceinline__ Item make_item(const ScoreParams& p, const Walk& w, int per_item, const ItemRead& r) {
  Item it;
  const int lane = int(threadIdx.x & 31);
  it.tile0 = w.tile0;
  it.limit = p.balanced ? w.left : p.chunk;
  it.token0 = w.group * per_item;
  it.count = p.tokens - it.token0 < per_item ? p.tokens - it.token0 : per_item;
  it.seq = r.seq < 0 || r.seq >= p.seqs ? -1 : r.seq;
  it.end = r.end < 0 || it.seq < 0 ? 0 : (r.end > p.row_stride ? int32_t(p.row_stride) : r.end);
  const int32_t before = __shfl_up_sync(0xFFFFFFFFu, it.seq, 1);
  it.starts = __ballot_sync(0xFFFFFFFFu, lane < it.count && (lane == 0 || before != it.seq));
  return it;
}

// The run that starts at lane a: its end lane, its sequence, the key tiles of this item that any of its queries sees.
struct Run {
  int a, b;
  int32_t seq, end, tiles;
};

__device__ __forceinline__ Run load_run(const ScoreParams& p, const Item& it, int a) {
  Run r;
  const int lane = int(threadIdx.x & 31);
  const uint32_t later = a < 31 ? it.starts & ~((2u << a) - 1u) : 0u;
  r.a = a;
  r.b = later != 0u ? __ffs(later) - 1 : it.count;
  r.seq = __shfl_sync(0xFFFFFFFFu, it.seq, a);
  r.end = __reduce_max_sync(0xFFFFFFFFu, lane >= a && lane < r.b ? it.end : 0);
  const int32_t n = (r.end + kTile - 1) / kTile - it.tile0;
  r.tiles = n < 0 ? 0 : (n > it.limit ? it.limit : n);
  return r;
}

// To the next item; the one that ends is `it`.
__device__ __forceinline__ void step_walk(const ScoreParams& p, Walk& w, const Item& it) {
  if (p.balanced) {
    w.left -= load_run(p, it, 0).tiles;
    ++w.group;
    w.tile0 = 0;
  } else {
    deal(p, w, w.item + int32_t(gridDim.x));
  }
}

// Where a key lies: its page as the table gives it (-1: none), and its place in the page.
struct KeyPage {
  int32_t page, place;
};
__device__ __forceinline__ KeyPage fetch_page(const ScoreParams& p, const int32_t* table, int32_t pos, int32_t end) {
  KeyPage at = {-1, 0};
  if (pos < end) {
    const int32_t i = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
    at.place = pos - i * p.page_size;
    if (i < p.table_width) at.page = table[i];
  }
  return at;
}

// kByte: e4m3 operands.  kHeads: heads per query, padded.  kCols: columns of an accumulator.
// kFull: no head is padding (the test for it would cost the sum as much as its arithmetic).
template <bool kByte, int kHeads, int kCols, bool kFull>
__global__ void __launch_bounds__(kScThreads, 1) score_kernel(const __grid_constant__ ScoreParams p,
                                                             const uint32_t idesc) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kPerTile = kCols / kHeads;   // queries of an accumulator
  // One query an accumulator: key tiles go round as many as fit, so that products run ahead while the
  // epilogue starts on a work item; warpgroup and product warp b take every other tile.  Several: two of
  // 256 columns, and both warpgroups take each, half of its queries each, while the other one is filled.
  constexpr bool kShare = kPerTile > 1;
  constexpr int kAccs = kShare ? 2 : (512 / kCols < kMaxAccs ? 512 / kCols : kMaxAccs);
  const uint32_t ring0 = shared_addr(smem);
  const int panels = (p.row_bytes + 127) / 128;
  const uint32_t stage_bytes = uint32_t(panels) * kPanel;
  const uint32_t q0 = ring0 + uint32_t(p.ring) * stage_bytes;
  const uint32_t q_panel = uint32_t(kCols) * 128u;                       // one accumulator's queries, one panel
  const uint32_t q_bytes = uint32_t(p.col_tiles * panels) * q_panel;     // one query buffer
  uint8_t* tail = smem + p.ring * stage_bytes + p.q_bufs * q_bytes;
  const uint32_t full0 = shared_addr(tail), empty0 = full0 + 8 * kMaxRing;
  const uint32_t done0 = full0 + 16 * kMaxRing, free0 = done0 + 8 * kMaxAccs, qfull0 = free0 + 8 * kMaxAccs,
                 qfree0 = qfull0 + 16;
  const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
  const int per_item = kPerTile * p.col_tiles;
  static_assert((2 * kMaxRing + 2 * kMaxAccs + 4) * 8 + 8 <= kBarBytes, "barriers outgrew their reservation");
  uint32_t* tmem_base_sh = reinterpret_cast<uint32_t*>(tail + (2 * kMaxRing + 2 * kMaxAccs + 4) * 8);
  if ((ring0 & 1023u) != 0u) {   // the swizzled panels need it; the dynamic window starts aligned when it is alone
    if (threadIdx.x == 0) atomicExch(&g_score_status, DSEL_ERR_ALIGN);
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.ring; ++i) {
      bar_init(full0 + 8 * i, p.box_keys > 0 ? 1 : kProdThreads);
      bar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      bar_init(done0 + 8 * i, 1);
      bar_init(free0 + 8 * i, kShare ? 256 : 128);   // the warpgroups that read an accumulator
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(qfull0 + 8 * i, 1);
      bar_init(qfree0 + 8 * i, kShare ? 1 : kMmaWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  constexpr uint32_t kTmemCols = kAccs * kCols;   // a power of two of at least 32
  if (warp == kEpiWarps + kProdWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_addr(tmem_base_sh)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_sh;
  grid_wait();
  grid_launch();

  if (warp < kEpiWarps) {
    // ---------------- sum over heads, stores ----------------
    constexpr int kMine = kShare ? kPerTile / 2 : 1;       // queries of an accumulator that this warpgroup sums
    constexpr int kMyCols = kMine * kHeads;
    constexpr int kSets = kShare ? 2 : 1;                  // accumulators with queries of their own (col_tiles)
    constexpr int kChunk = kMyCols < 32 ? kMyCols : 32;    // columns read at a time, the next while one is summed
    constexpr int kChunks = kMyCols / kChunk;
    constexpr int kGroups = kChunk / 8;
    constexpr int kPerQuery = kHeads < kChunk ? kHeads : kChunk;
    const int b = warp >> 2;                       // warpgroup
    const int row = (warp & 3) * 32 + (lane >> 2) + (lane & 3) * 8;   // the key of a tile whose sum ends up here
    const uint32_t acc0 = tmem + (uint32_t(warp & 3) << 21);          // lane quarter in bits 16..
    uint32_t parity = 0;  // bit a: accumulator a's next fill
    uint32_t turn = 0;    // key tiles so far (col_tiles == 1: accumulators take turns)
    bool ok = true;
    // -inf from column `from` to `to` (multiples of 16) of a query's row: both warpgroups' threads, 16 bytes each
    auto fill = [&](int32_t token, int64_t from, int64_t to) {
      const int step = p.out_f32 ? 4 : 8;
      const uint32_t none = p.out_f32 ? 0xFF800000u : 0xFF80FF80u;
      for (int64_t pos = from + int64_t(threadIdx.x) * step; pos < to; pos += kEpiWarps * 32 * step) {
        const int64_t o = (int64_t(token) * p.row_stride + pos) * (p.out_f32 ? 4 : 2);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + o) = make_uint4(none, none, none, none);
      }
    };
    if (p.balanced) {   // what no query sees, in pieces, while the first tiles are on their way
      constexpr int64_t kPieceCols = 8192;
      const int64_t pieces = (p.row_stride + kPieceCols - 1) / kPieceCols;
      for (int64_t u = blockIdx.x; u < pieces * p.tokens; u += gridDim.x) {
        const int32_t token = int32_t(u / pieces);
        const int64_t col = u % pieces * kPieceCols, seen = int64_t(tiles_of(p, token)) * kTile;
        fill(token, seen > col ? seen : col, col + kPieceCols < p.row_stride ? col + kPieceCols : p.row_stride);
      }
    }
    Walk walk = first_walk(p);
    ItemRead ahead = read_item(p, walk, per_item);
    while (walk.more(p) && ok) {
      const Item it = make_item(p, walk, per_item, ahead);
      step_walk(p, walk, it);
      ahead = read_item(p, walk, per_item);
      // the weights of this thread's columns
      float w[kSets][kMyCols / 4];
#pragma unroll
      for (int n = 0; n < kSets; ++n)
#pragma unroll
        for (int i = 0; i < kMyCols / 4; ++i) {
          const int col = (i >> 1) * 8 + (lane & 3) * 2 + (i & 1);
          const int qi = n * kPerTile + (kShare ? b * kMine : 0) + col / kHeads, h = col % kHeads;
          w[n][i] = qi < it.count && qi < per_item && h < p.heads
                        ? p.weights[int64_t(it.token0 + qi) * p.weights_stride + h]
                        : 0.f;
        }
      // Queries that were summed, four sums in each of four lanes: finish() leaves one key's in every lane
      // and stores it.  It runs beside the next sum, whose arithmetic fills its waits.
      struct {
        float s[kChunk / kPerQuery][4];
        int32_t pos, q, lo, hi;   // stored: queries q.. in [lo, hi)
        uint64_t at;              // address of query 0's score of this key
        float scale;
        bool live;
      } last = {};
      const bool out_f32 = p.out_f32 != 0;
      auto finish = [&]() {
#pragma unroll
        for (int i = 0; i < kChunk / kPerQuery; ++i) {
          const float* v = last.s[i];
          const bool odd = (lane & 1) != 0, high = (lane & 2) != 0;
          const float a0 = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[1], 1);
          const float a1 = (odd ? v[3] : v[2]) + __shfl_xor_sync(0xFFFFFFFFu, odd ? v[2] : v[3], 1);
          float y = ((high ? a1 : a0) + __shfl_xor_sync(0xFFFFFFFFu, high ? a0 : a1, 2)) * last.scale;
          const int qi = last.q + i;
          const int32_t end = __shfl_sync(0xFFFFFFFFu, it.end, qi & 31);
          if (!last.live || last.pos >= end) y = -__int_as_float(0x7F800000);
          // (queries of other runs are summed with the others and not stored)
          store_if(qi >= last.lo && qi < last.hi && last.pos < p.row_stride, out_f32,
                   last.at + ((int64_t(qi) * int32_t(p.row_stride)) << (out_f32 ? 2 : 1)), y);
        }
      };
      const int64_t pos0 = int64_t(it.tile0) * kTile;
      const int64_t pos_end = pos0 + int64_t(p.chunk) * kTile < p.row_stride ? pos0 + int64_t(p.chunk) * kTile : p.row_stride;
      for (int a = 0; a < it.count && ok;) {
        const Run run = load_run(p, it, a);
        a = run.b;
        const int32_t* table = p.table + int64_t(run.seq < 0 ? 0 : run.seq) * p.table_stride;
        // Each key's scale is read one tile of this warpgroup ahead of its use, its page two.
        const int skip = kShare ? 1 : 2;
        int32_t k = kShare ? 0 : int32_t((turn & 1u) != uint32_t(b));
        const uint32_t turn0 = turn;
        turn += uint32_t(run.tiles);
        auto page_of = [&](int32_t tile) {
          return fetch_page(p, table, (it.tile0 + tile) * kTile + row, tile < run.tiles ? run.end : 0);
        };
        auto exists = [&](const KeyPage& at) { return at.page >= 0 && at.page < p.pages; };
        auto scale_of = [&](const KeyPage& at) {
          return p.key_scale != nullptr && exists(at) ? p.key_scale[int64_t(at.page) * p.scale_page_stride + at.place] : 1.f;
        };
        KeyPage at = page_of(k), next = page_of(k + skip);
        float scale = scale_of(at);
        for (; k < run.tiles && ok; k += skip) {
          const int32_t pos = (it.tile0 + k) * kTile + row;
          const bool live = exists(at);
          const float scale_now = scale;
          scale = scale_of(next);
          at = next;
          next = page_of(k + 2 * skip);
#pragma unroll
          for (int n = 0; n < kSets; ++n) {
            // the accumulator's queries in the run, and this warpgroup's of them
            if (n >= p.col_tiles || run.b <= n * kPerTile || run.a >= (n + 1) * kPerTile) continue;
            const int first = n * kPerTile + (kShare ? b * kMine : 0);
            const int lo = run.a > first ? run.a : first;
            const int hi = run.b < first + kMine ? run.b : first + kMine;
            const uint32_t acc_i = kShare && p.col_tiles == 2 ? uint32_t(n) : (turn0 + uint32_t(k)) & uint32_t(kAccs - 1);
            if (!bar_wait(done0 + 8 * acc_i, (parity >> acc_i) & 1u)) {
              ok = false;
              break;
            }
            parity ^= 1u << acc_i;
            tc_fence_after();
            if (lo >= hi) {   // only the other warpgroup has queries here
              tc_fence_before();
              bar_arrive(free0 + 8 * acc_i);
              continue;
            }
            const uint32_t acc = acc0 + acc_i * uint32_t(kCols) + uint32_t(kShare ? b * kMyCols : 0);
            uint32_t x[2][2][4 * kGroups];
            auto read = [&](int c) {
              tmem_load<kGroups>(acc + uint32_t(c * kChunk), x[c & 1][0]);
              tmem_load<kGroups>(acc + (16u << 16) + uint32_t(c * kChunk), x[c & 1][1]);
            };
            float2 s[4];   // sums of keys lane / 4 + 8 j, even and odd columns
            read(0);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              tmem_wait<kGroups>(x[c & 1][0]);
              tmem_wait<kGroups>(x[c & 1][1]);
              if (c + 1 < kChunks) {
                read(c + 1);
              } else {   // nothing of the accumulator is left to read
                tc_fence_before();
                bar_arrive(free0 + 8 * acc_i);
              }
              if ((kHeads <= kChunk || c * kChunk % kHeads == 0)) finish();   // its waits pass under this sum
#pragma unroll
              for (int q = 0; q < kChunk / kPerQuery; ++q) {
                if (c * kChunk % kHeads == 0) s[0] = s[1] = s[2] = s[3] = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = q * kPerQuery / 8; j < (q + 1) * kPerQuery / 8; ++j) {
                  const float2 wj = make_float2(w[n][(c * kGroups + j) * 2], w[n][(c * kGroups + j) * 2 + 1]);
#pragma unroll
                  for (int k4 = 0; k4 < 4; ++k4) {
                    const uint32_t* xe = &x[c & 1][k4 >> 1][4 * j + 2 * (k4 & 1)];
                    float2 y = make_float2(relu(xe[0]), relu(xe[1]));
                    if (!kFull) {   // columns behind the last head count for nothing, whatever they hold
                      const int h = (c * kChunk + j * 8) % kHeads + (lane & 3) * 2;
                      if (h >= p.heads) y.x = 0.f;
                      if (h + 1 >= p.heads) y.y = 0.f;
                    }
                    s[k4] = fma2(y, wj, s[k4]);
                  }
                }
                if (kHeads <= kChunk || (c + 1) * kChunk % kHeads == 0) {   // the query's last columns
#pragma unroll
                  for (int k4 = 0; k4 < 4; ++k4) last.s[q][k4] = s[k4].x + s[k4].y;
                }
              }
              if (kHeads <= kChunk || (c + 1) * kChunk % kHeads == 0) {
                last.pos = pos;
                last.q = first + c * kChunk / kHeads;
                last.lo = lo;
                last.hi = hi;
                last.at = reinterpret_cast<uint64_t>(p.out) +
                          uint64_t((int64_t(it.token0) * p.row_stride + pos) << (out_f32 ? 2 : 1));
                last.scale = scale_now;
                last.live = live;
              }
            }
          }
        }
        finish();
        last.hi = 0;
        // -inf behind the run's last tile
        if (!p.balanced)
          for (int qi = run.a; qi < run.b; ++qi) fill(it.token0 + qi, pos0 + int64_t(run.tiles) * kTile, pos_end);
      }
    }
  } else if (warp < kEpiWarps + kProdWarps) {
    // ---------------- key tiles and queries ----------------
    const int pw = warp - kEpiWarps;
    const uint32_t ring = uint32_t(p.ring);
    Cursor tile = {0, 0}, told = {0, 0}, qbuf = {0, 0};   // next tile; next copied tile to announce; next queries
    int pending = 0;                                      // tiles copied but not yet announced
    bool ok = true;
    auto tell = [&]() {   // announce the oldest copied tile that is not yet: it is complete, and visible to the products
      fence_async_shared();
      bar_arrive(full0 + 8 * told.at);
      told.step(ring);
      --pending;
    };
    auto flush = [&]() {
      copy_wait<0>();
      while (pending > 0) tell();
    };
    // the item's queries, before its first tile
    auto load_queries = [&](const Item& it) {
      const uint32_t buf = qbuf.at, was = (qbuf.rounds & 1u) ^ 1u;
      qbuf.step(uint32_t(p.q_bufs));
      if (pw != 0) return true;
      // the products that read this buffer may still wait for tiles not yet announced
      if (p.box_keys == 0 && !__all_sync(0xFFFFFFFFu, bar_try(qfree0 + 8 * buf, was))) flush();
      if (!bar_wait(qfree0 + 8 * buf, was)) return false;
      if (elect_one()) {
        bar_expect(qfull0 + 8 * buf, q_bytes);
        for (int n = 0; n < p.col_tiles; ++n)
          for (int i = 0; i < panels; ++i)
            tma_load(q0 + buf * q_bytes + uint32_t(n * panels + i) * q_panel, &p.q_map, qfull0 + 8 * buf,
                     i * (kByte ? 128 : 64), 0, it.token0 + n * kPerTile);
      }
      __syncwarp();
      return true;
    };
    if (p.box_keys > 0) {
      {
        // The warps take every other tile.  Lane i brings its page i (or its part of a longer page); 32 pages
        // are looked up at once, that many ahead of their use.
        uint32_t turn = 0;
        const int boxes = kTile / p.box_keys, per_batch = 32 / boxes;
        const uint32_t box_bytes = uint32_t(p.box_keys) * 128u;
        Walk walk = first_walk(p);
        ItemRead ahead = read_item(p, walk, per_item);
        while (walk.more(p) && ok) {
          const Item it = make_item(p, walk, per_item, ahead);
          step_walk(p, walk, it);
          ahead = read_item(p, walk, per_item);
          bool queries = false;   // loaded for this item
          for (int a = 0; a < it.count && ok;) {
            const Run run = load_run(p, it, a);
            a = run.b;
            const int32_t* table = p.table + int64_t(run.seq < 0 ? 0 : run.seq) * p.table_stride;
            const int32_t start = it.tile0 * kTile;
            auto fetch = [&](int32_t k) {   // the pages of tiles k .. k + per_batch - 1
              return fetch_page(p, table, start + k * kTile + lane * p.box_keys, k < run.tiles ? run.end : 0).page;
            };
            int32_t batch = -1, next = fetch(0);
            for (int32_t k = 0; k < run.tiles; ++k) {
              const int in_batch = k & (per_batch - 1);
              if (in_batch == 0) {
                batch = next;
                next = fetch(k + per_batch);
              }
              const int32_t page = __shfl_sync(0xFFFFFFFFu, batch, (in_batch * boxes + lane) & 31);
              const int32_t pos = start + k * kTile + lane * p.box_keys;
              if (!queries) {
                queries = true;
                if (!load_queries(it)) {
                  ok = false;
                  break;
                }
              }
              if (int(turn++ & 1u) == pw) {
                const uint32_t slot = tile.at;
                if (!bar_wait(empty0 + 8 * slot, (tile.rounds & 1u) ^ 1u)) {
                  ok = false;
                  break;
                }
                // (keys behind the last page are left as they are: their sums are not used)
                const bool in = lane < boxes && pos < run.end;
                const int n = __popc(__ballot_sync(0xFFFFFFFFu, in));
                if (elect_one()) bar_expect(full0 + 8 * slot, uint32_t(n * panels) * box_bytes);
                __syncwarp();
                if (in) {   // a page outside the cache is outside the map: zeros
                  const uint32_t dst = ring0 + slot * stage_bytes + uint32_t(lane) * box_bytes;
                  for (int i = 0; i < panels; ++i)
                    tma_load(dst + uint32_t(i) * kPanel, &p.key_map, full0 + 8 * slot, i * (kByte ? 128 : 64),
                             pos & (p.page_size - 1), page);
                }
                __syncwarp();
              }
              tile.step(ring);
            }
          }
        }
        // after a wait that gave up: no copy stays in flight (the last use of each place)
        for (uint32_t i = 0; !ok && i < ring; ++i) {
          const uint32_t uses = tile.rounds + (i < tile.at ? 1u : 0u);
          if (uses > 0) bar_wait(full0 + 8 * i, (uses - 1) & 1u);   // (or the other warp's, given up on as well)
        }
      }
    } else {
      const int per_row = p.row_bytes / 16;   // 16-byte pieces of a key: 2, 4, 6, 8, 12 or 16
      const int inverse = (65536 + per_row - 1) / per_row;   // i * inverse / 65536 is i / per_row for every piece of a tile
      Walk walk = first_walk(p);
      ItemRead ahead = read_item(p, walk, per_item);
      while (walk.more(p) && ok) {
        const Item it = make_item(p, walk, per_item, ahead);
        step_walk(p, walk, it);
        ahead = read_item(p, walk, per_item);
        bool queries = false;   // loaded for this item
        for (int a = 0; a < it.count && ok;) {
          const Run run = load_run(p, it, a);
          a = run.b;
          const int32_t* table = p.table + int64_t(run.seq < 0 ? 0 : run.seq) * p.table_stride;
          // each lane looks up two keys of a tile, a tile ahead of their use
          const int32_t mine = it.tile0 * kTile + pw * kProdKeys + lane;
          KeyPage next0 = fetch_page(p, table, mine, run.tiles > 0 ? run.end : 0);
          KeyPage next1 = fetch_page(p, table, mine + 32, run.tiles > 0 ? run.end : 0);
          for (int32_t k = 0; k < run.tiles; ++k) {
            const KeyPage at0 = next0, at1 = next1;
            const int32_t end = k + 1 < run.tiles ? run.end : 0;
            next0 = fetch_page(p, table, mine + (k + 1) * kTile, end);
            next1 = fetch_page(p, table, mine + (k + 1) * kTile + 32, end);
            if (!queries) {
              queries = true;
              if (!load_queries(it)) {
                ok = false;
                break;
              }
            }
            const uint32_t slot = tile.at;
            if (!bar_wait(empty0 + 8 * slot, (tile.rounds & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            const int64_t off0 = at0.page >= 0 && at0.page < p.pages
                                     ? int64_t(at0.page) * p.page_bytes + int64_t(at0.place) * p.key_bytes
                                     : -1;
            const int64_t off1 = at1.page >= 0 && at1.page < p.pages
                                     ? int64_t(at1.page) * p.page_bytes + int64_t(at1.place) * p.key_bytes
                                     : -1;
            const uint32_t dst0 = ring0 + slot * stage_bytes + uint32_t(pw) * (kProdKeys * 128);
            // consecutive lanes bring consecutive pieces
#pragma unroll 4
            for (int i = lane; i < kProdKeys * per_row; i += 32) {
              const int r = (i * inverse) >> 16, piece = i - r * per_row;
              const int64_t o0 = __shfl_sync(0xFFFFFFFFu, off0, r & 31), o1 = __shfl_sync(0xFFFFFFFFu, off1, r & 31);
              const int64_t o = r < 32 ? o0 : o1;
              copy16(dst0 + uint32_t(piece >> 3) * kPanel + uint32_t(r) * 128u + (uint32_t((piece ^ r) & 7) << 4),
                     p.keys + (o < 0 ? 0 : o + piece * 16), o >= 0);
            }
            copy_commit();
            tile.step(ring);
            if (++pending > p.lag) {
              if (p.lag >= 4)
                copy_wait<4>();
              else if (p.lag == 3)
                copy_wait<3>();
              else if (p.lag == 2)
                copy_wait<2>();
              else
                copy_wait<1>();
              tell();
            }
          }
        }
      }
      flush();   // also on the way out after a wait that gave up: no copy stays in flight
    }
  } else {
    // ---------------- products ----------------
    Cursor tile = {0, 0}, qbuf = {0, 0};
    const int mw = warp - kEpiWarps - kProdWarps;
    uint32_t parity = 0;   // bit a: accumulator a's next fill
    uint32_t turn = 0;     // key tiles so far
    bool ok = mw == 0 || !kShare;
    const int steps = p.row_bytes / 32;
    const uint64_t key_operand = operand(ring0), q_operand = operand(q0);
    Walk walk = first_walk(p);
    ItemRead ahead = read_item(p, walk, per_item);
    while (walk.more(p) && ok) {
      const Item it = make_item(p, walk, per_item, ahead);
      step_walk(p, walk, it);
      ahead = read_item(p, walk, per_item);
      bool any = false;
      for (int a = 0; a < it.count && ok;) {
        const Run run = load_run(p, it, a);
        a = run.b;
        for (int32_t k = 0; k < run.tiles && ok; ++k) {
          if (!any && !bar_wait(qfull0 + 8 * qbuf.at, qbuf.rounds & 1u)) {
            ok = false;
            break;
          }
          any = true;
          if (!kShare && int(turn & 1u) != mw) {   // the other warp's
            parity ^= 1u << (turn & uint32_t(kAccs - 1));
            tile.step(uint32_t(p.ring));
            ++turn;
            continue;
          }
          if (!bar_wait(full0 + 8 * tile.at, tile.rounds & 1u)) {
            ok = false;
            break;
          }
          // (addresses in descriptors count 16 bytes)
          const uint64_t keys = key_operand + uint64_t(tile.at * (stage_bytes >> 4));
#pragma unroll
          for (int n = 0; n < (kShare ? 2 : 1); ++n) {
            // only accumulators with a query of the run
            if (n >= p.col_tiles || run.b <= n * kPerTile || run.a >= (n + 1) * kPerTile) continue;
            const uint32_t b = kShare && p.col_tiles == 2 ? uint32_t(n) : turn & uint32_t(kAccs - 1);
            if (!bar_wait(free0 + 8 * b, ((parity >> b) & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            parity ^= 1u << b;
            tc_fence_after();
            if (elect_one()) {   // always the same thread: a commit covers its own products
              const uint64_t queries = q_operand + uint64_t((qbuf.at * q_bytes + uint32_t(n * panels) * q_panel) >> 4);
              const uint32_t d = tmem + b * uint32_t(kCols);
#pragma unroll
              for (int s = 0; s < 8; ++s)
                if (s < steps)
                  mma<kByte>(d, keys + uint64_t((s >> 2) * (kPanel >> 4) + (s & 3) * 2),
                             queries + uint64_t((s >> 2) * (kCols * 128 >> 4) + (s & 3) * 2), idesc, s > 0);
              tc_commit(done0 + 8 * b);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) tc_commit(empty0 + 8 * tile.at);
          __syncwarp();
          tile.step(uint32_t(p.ring));
          ++turn;
        }
      }
      if (any) {
        if (ok && elect_one()) tc_commit(qfree0 + 8 * qbuf.at);
        __syncwarp();
        qbuf.step(uint32_t(p.q_bufs));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kEpiWarps + kProdWarps) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The map of a [planes][rows][dim] tensor with boxes of `box_planes` x `box_rows` x `inner` elements.
bool encode(CUtensorMap* map, int dtype, const void* base, int64_t dim, int64_t rows, int64_t planes, int64_t row_bytes,
            int64_t plane_bytes, int inner, int box_rows, int box_planes) {
  static std::atomic<EncodeFn> known;
  EncodeFn fn = known.load(std::memory_order_relaxed);
  if (fn == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || f == nullptr) {
      cudaGetLastError();
      return false;
    }
    fn = reinterpret_cast<EncodeFn>(f);
    known.store(fn, std::memory_order_relaxed);
  }
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(rows), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(row_bytes), cuuint64_t(plane_bytes)};
  const cuuint32_t box[3] = {cuuint32_t(inner), cuuint32_t(box_rows), cuuint32_t(box_planes)};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUtensorMapDataType type = dtype == DSEL_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == DSEL_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return fn(map, type, 3, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kByte, int kHeads, int kCols, bool kFull>
int launch_score(const ScoreParams& p, int dtype, int grid, int smem, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> allowed;
  auto kern = score_kernel<kByte, kHeads, kCols, kFull>;
  if (allow_smem(reinterpret_cast<const void*>(kern), kScoreSmem, dev, &allowed) != cudaSuccess) return DSEL_ERR_CUDA;
  // D f32, A and B of the operands' type (f16 0, bf16 1; e4m3 0), both K-major, N / 8, M / 16
  const uint32_t type = dtype == DSEL_BF16 ? 1u : 0u;
  const uint32_t idesc =
      (1u << 4) | (type << 7) | (type << 10) | (uint32_t(kCols / 8) << 17) | (uint32_t(kTile / 16) << 24);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(kScThreads, 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, idesc) == cudaSuccess ? DSEL_OK : DSEL_ERR_CUDA;
}

template <bool kByte, int kHeads>
int launch_heads(const ScoreParams& p, int dtype, bool wide, int grid, int smem, int dev, cudaStream_t st) {
  if (p.heads == kHeads)
    return wide ? launch_score<kByte, kHeads, 256, true>(p, dtype, grid, smem, dev, st)
                : launch_score<kByte, kHeads, kHeads, true>(p, dtype, grid, smem, dev, st);
  return wide ? launch_score<kByte, kHeads, 256, false>(p, dtype, grid, smem, dev, st)
              : launch_score<kByte, kHeads, kHeads, false>(p, dtype, grid, smem, dev, st);
}

template <bool kByte>
int launch_type(const ScoreParams& p, int dtype, int hp, bool wide, int grid, int smem, int dev, cudaStream_t st) {
  switch (hp) {
    case 16: return launch_heads<kByte, 16>(p, dtype, wide, grid, smem, dev, st);
    case 32: return launch_heads<kByte, 32>(p, dtype, wide, grid, smem, dev, st);
    case 64: return launch_heads<kByte, 64>(p, dtype, wide, grid, smem, dev, st);
    default: return launch_heads<kByte, 128>(p, dtype, wide, grid, smem, dev, st);
  }
}

}  // namespace

int score_status(int* out, cudaStream_t st) {
  int zero = 0;
  if (cudaMemcpyFromSymbolAsync(out, g_score_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaMemcpyToSymbolAsync(g_score_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return DSEL_ERR_CUDA;
  return DSEL_OK;
}

}  // namespace dsel

using namespace dsel;

DSEL_API int dsel_index_score(const void* q, int dtype, int64_t tokens, int32_t heads, int32_t dim,
                              int64_t q_token_stride, int64_t q_head_stride, const float* weights,
                              int64_t weights_stride, const void* keys, int32_t pages, int32_t page_size,
                              int64_t page_stride, int64_t key_stride, const float* key_scale,
                              int64_t scale_page_stride, const int32_t* table, int32_t seqs, int32_t table_width,
                              int64_t table_stride, const int32_t* seq_ids, const int32_t* end, void* out,
                              int out_dtype, int64_t row_stride, void* stream) {
  if (dtype != DSEL_BF16 && dtype != DSEL_F16 && dtype != DSEL_E4M3) return DSEL_ERR_DTYPE;
  if (out_dtype != DSEL_BF16 && out_dtype != DSEL_F32) return DSEL_ERR_DTYPE;
  if (tokens < 0 || tokens > INT32_MAX / 2) return DSEL_ERR_ROWS;
  const int eb = dtype == DSEL_E4M3 ? 1 : 2;
  if (heads < 1 || heads > 128 || dim < 32 || dim > 128 || dim % 32 != 0) return DSEL_ERR_SHAPE;
  if (pages < 0 || page_size < 1 || seqs < 0 || table_width < 0) return DSEL_ERR_SHAPE;
  if (seq_ids == nullptr && seqs != 1 && int64_t(seqs) != tokens) return DSEL_ERR_SHAPE;
  if (row_stride < 1 || row_stride % kStrideReq != 0 || row_stride > INT32_MAX - 1024 * kTile) return DSEL_ERR_STRIDE;
  if (q_head_stride < dim || (tokens > 1 && q_token_stride < dim) || weights_stride < heads || key_stride < dim || page_stride < 0 ||
      table_stride < table_width || scale_page_stride < 0)
    return DSEL_ERR_STRIDE;
  // rows of operands are copied in 16-byte pieces
  if (q_head_stride * eb % 16 != 0 || q_token_stride * eb % 16 != 0 || key_stride * eb % 16 != 0 ||
      page_stride * eb % 16 != 0)
    return DSEL_ERR_STRIDE;
  if (tokens == 0) return DSEL_OK;
  // A cache without pages, or a table without places, has no keys: no query is of any sequence, and neither is read.
  const bool no_keys = pages == 0 || seqs == 0 || table_width == 0;
  if (q == nullptr || weights == nullptr || end == nullptr || out == nullptr ||
      (!no_keys && (keys == nullptr || table == nullptr)))
    return DSEL_ERR_NULL;
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(keys) | reinterpret_cast<uintptr_t>(out)) & 15u) != 0)
    return DSEL_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (const int st = current_device(&dev, &sms); st != DSEL_OK) return st;

  ScoreParams p = {};
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.keys = static_cast<const uint8_t*>(keys);
  p.page_bytes = page_stride * eb;
  p.key_bytes = key_stride * eb;
  p.key_scale = key_scale;
  p.scale_page_stride = scale_page_stride;
  p.table = table;
  p.table_stride = table_stride;
  p.seq_ids = seq_ids;
  p.end = end;
  p.out = out;
  p.row_stride = row_stride;
  p.pages = pages;
  p.page_size = page_size;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((int64_t(1) << s) == page_size) p.page_shift = s;
  p.seqs = no_keys ? 0 : seqs;
  p.table_width = table_width;
  p.tokens = int32_t(tokens);
  p.heads = heads;
  p.row_bytes = dim * eb;
  p.seq_mode = seq_ids != nullptr ? 0 : (seqs == 1 ? 2 : 1);
  p.out_f32 = out_dtype == DSEL_F32;

  // One query an accumulator where each sequence has one (decoding: bound by the keys' bytes, so a narrow
  // accumulator and a deep ring); else as many as 256 columns hold, and two accumulators per key tile
  // when a sequence has more queries than one holds: each tile then serves twice the queries.
  const int hp = heads <= 16 ? 16 : heads <= 32 ? 32 : heads <= 64 ? 64 : 128;
  const int64_t per_seq = seqs > 0 ? (tokens + seqs - 1) / seqs : 1;
  const bool wide = per_seq > 1;
  const int cols = wide ? 256 : hp;
  p.col_tiles = wide && per_seq > 256 / hp ? 2 : 1;
  const int stage = (p.row_bytes + 127) / 128 * kPanel;
  const int qbytes = p.col_tiles * ((p.row_bytes + 127) / 128) * cols * 128;
  const int room = kScoreSmem - kBarBytes;
  p.q_bufs = (room - 2 * qbytes) / stage >= 4 ? 2 : 1;
  p.ring = (room - p.q_bufs * qbytes) / stage;
  if (p.ring > kMaxRing) p.ring = kMaxRing;
  p.lag = p.ring - 2 > 4 ? 4 : p.ring - 2;
  const int smem = p.ring * stage + p.q_bufs * qbytes + kBarBytes;

  // Queries come as boxes of one accumulator; keys as boxes of a page where the pages fit tiles.
  const int inner = 128 / eb;   // elements of 128 bytes
  const int64_t q_head = heads > 1 ? q_head_stride * eb : p.row_bytes;
  const int64_t q_token = tokens > 1 ? q_token_stride * eb : heads * q_head;
  if (!encode(&p.q_map, dtype, q, dim, heads, tokens, q_head, q_token, inner, hp, cols / hp)) return DSEL_ERR_STRIDE;
  p.box_keys = p.page_shift >= 3 && !no_keys ? (page_size < kTile ? page_size : kTile) : 0;
  if (p.box_keys > 0 && !encode(&p.key_map, dtype, keys, dim, page_size, pages, p.key_bytes,
                                pages > 1 ? p.page_bytes : int64_t(page_size) * p.key_bytes, inner, p.box_keys, 1))
    p.box_keys = 0;

  // Key tiles per work item: the count whose items fill whole rounds of the SMs best, an item's own
  // cost (its queries) counted as one tile of a narrow accumulator, two of a wide one.
  const int64_t per_item = int64_t(cols / hp) * p.col_tiles;
  const int64_t groups = (tokens + per_item - 1) / per_item;
  const int64_t tiles = (row_stride + kTile - 1) / kTile;
  const int most = p.col_tiles == 2 ? 64 : 16;
  int64_t best = -1;
  for (int c = 1; c <= most && c <= tiles; ++c) {
    const int64_t items = groups * ((tiles + c - 1) / c);
    if (items > INT32_MAX / 2) continue;
    const int64_t cost = (items + sms - 1) / sms * (c + (wide ? 2 : 1));
    if (best < 0 || cost <= best) {
      best = cost;
      p.chunk = c;
    }
  }
  if (best < 0) return DSEL_ERR_ROWS;
  p.chunks = int32_t((tiles + p.chunk - 1) / p.chunk);
  p.items = int32_t(groups * p.chunks);
  // A query an item, not too many of them to sum on the way in: every CTA takes the same number of tiles in one go,
  // however ragged the sequences.  (Ranges of 16 tiles dealt out: e4m3 decoding 167 us, an item's start costs four of
  // its tiles; equal shares took 140; ranges of 32: the same, and bf16 262 us for 255, since some CTAs got one
  // more than others.)
  // Where every tile has a CTA of its own, the sum would only come before it (1 x 8,192: 5.7 us for 4.8).
  const int64_t most_tiles = tokens * tiles;
  p.balanced = !wide && tokens <= 1024 && most_tiles > sms;
  const int grid = p.balanced ? sms : (p.items < sms ? p.items : sms);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return dtype == DSEL_E4M3 ? launch_type<true>(p, dtype, hp, wide, grid, smem, dev, cs)
                            : launch_type<false>(p, dtype, hp, wide, grid, smem, dev, cs);
}
