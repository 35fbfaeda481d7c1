// What the two kernels of mdw_tree_attention share: the call's parameters, the cut of its work into shares, types
// and small steps. tree_attention.cu has the kernel for many rows, the join and the entry points,
// tree_attention_rows.cu the kernel for up to 32 rows.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "mdw_attn.cuh"
#include "mdw_device.cuh"

namespace mdw {

constexpr int kTileKeys = 128;        // keys of a tile (one pipeline stage)
constexpr int kTileRows = 128;        // rows of a row block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnParams {
  const void* v;             // the cache's values and page stride, for keys read on their own
  int64_t page_stride;
  const float* k_scale;
  const float* v_scale;
  const void* q;
  void* out;
  float* lse;
  int64_t ldq, ldo;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* row_start;
  const uint64_t* tree_mask;
  uint32_t* status;
  long long spin_budget;
  float scale;
  int B, T, Hq, Hkv, group, max_new, max_pages, num_pages, page_shift, item_cost;
  // workspace
  int32_t* total;          // [2] tiles of the whole call, blocks with a share
  struct Cut* cuts;        // [grid] the item that a block's share starts inside of
  int32_t* lost;           // [grid] whether a block gave up: what its part belongs to is not stored
  float2* part_ml;         // [2 * grid][128] (c m, sum) of partial items
  float* part_o;           // [2 * grid][128][D] their unnormalised outputs
};

// An item that a share boundary cuts; rows = 0: the share starts with a whole item.
struct Cut {
  int row0, rows, first, h;        // request's first row, rows of the block (of rows x heads), its first one, kv head
  int start, tiles;                // first tile of the item, its tiles
};

// ------------------------------------------------------------------ requests and shares

// An item costs its tiles and, for its rows, its first scores and its result, as much time as so many more: they count
// when the work is cut into shares. 16 ragged trees: 84 us at 3, 79 to 81 at 5 to 7, 85 at 9; the kernel for few rows,
// 32 of them over E4M3: 79 us at 2, 72 at 4, 75 at 7; one token in 64 requests 66 us at 1, 64 at 2, 68 at 5.
constexpr int kItemCost = 6, kItemCost32 = 4, kItemCost16 = 2;

struct Request {
  int row0, rows, ctx, keys;       // first row, rows, cached tokens, keys; rows < 0: not valid
  __device__ __forceinline__ int blocks(const AttnParams& p) const { return (rows * p.group + kTileRows - 1) / kTileRows; }
  __device__ __forceinline__ int tiles() const { return (keys + kTileKeys - 1) / kTileKeys; }
  __device__ __forceinline__ int64_t work(const AttnParams& p) const {
    return rows <= 0 ? 0 : (int64_t)p.Hkv * blocks(p) * (tiles() + p.item_cost);
  }
};
__device__ __forceinline__ Request load_request(const AttnParams& p, int b) {
  Request r;
  r.row0 = p.row_start[b];
  const int64_t rows = (int64_t)p.row_start[b + 1] - r.row0;
  r.ctx = p.ctx_len[b];
  const int64_t keys = r.ctx + rows;
  const bool ok = r.row0 >= 0 && rows >= 0 && r.row0 + rows <= p.T && rows <= p.max_new && r.ctx >= 0 &&
                  keys <= (int64_t)p.max_pages << p.page_shift;
  r.rows = ok ? (int)rows : -1;
  r.keys = (int)keys;
  return r;
}

// Equal contiguous shares of `total` units: block c has [start(c), start(c + 1)). An item's units are its tiles and
// then its item cost; a share that has tiles of an item writes a partial result of it, one that ends
// among its last units has the whole rest.
struct Shares {
  int blocks, base, rest;
  __device__ __forceinline__ Shares(int total, int grid) {
    blocks = total < grid ? total : grid;
    base = blocks > 0 ? total / blocks : 0;
    rest = total - base * blocks;
  }
  __device__ __forceinline__ int start(int c) const { return c * base + min(c, rest); }
  __device__ __forceinline__ int owner(int t) const {
    const int wide = rest * (base + 1);
    return t < wide ? t / (base + 1) : rest + (t - wide) / base;
  }
};

// The walk of one warp over its block's share, tile by tile; every warp of a block sees the same. A lane holds
// one of 32 consecutive requests, so that the next one costs no load.
struct Walk {
  Request mine, r;                 // the lane's request; the current item's
  int b, h, rb, tile, tiles;       // current item and tile, tiles of the item
  int units;                       // units left in the share, the current item's from `tile` on first

  __device__ __forceinline__ void take(int lane_) {
    r.row0 = __shfl_sync(0xffffffffu, mine.row0, lane_);
    r.rows = __shfl_sync(0xffffffffu, mine.rows, lane_);
    r.ctx = __shfl_sync(0xffffffffu, mine.ctx, lane_);
    r.keys = __shfl_sync(0xffffffffu, mine.keys, lane_);
    tiles = r.tiles();
  }
  __device__ __forceinline__ void load32(const AttnParams& p, int first, int lane) {
    mine.rows = 0;
    if (first + lane < p.B) mine = load_request(p, first + lane);
  }
  __device__ void begin(const AttnParams& p, int lane) {
    units = 0;
    int64_t total = 0;
    for (int i = 0; i < p.B; i += 32) {
      load32(p, i, lane);
      if (mine.rows < 0 && blockIdx.x == 0) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
      int64_t w = mine.work(p);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      total += w;
    }
    const bool many = total > 0x7fffffff;       // beyond any real batch: nothing is computed
    if (many && blockIdx.x == 0) raise_status(p.status, MDW_ERR_UNSUPPORTED_SHAPE);
    const Shares shares(many ? 0 : (int)total, gridDim.x);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      p.total[0] = many ? 0 : (int)total;
      p.total[1] = shares.blocks;
    }
    if ((int)blockIdx.x >= shares.blocks) return;
    const int at = shares.start(blockIdx.x);
    units = shares.start(blockIdx.x + 1) - at;
    int before = 0;
    for (int i = 0; i < p.B; i += 32) {
      if (p.B > 32) load32(p, i, lane);
      const int w = (int)mine.work(p);
      int sum = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > at);
      if (hit) {
        const int l = __ffs(hit) - 1;
        before += __shfl_sync(0xffffffffu, sum - w, l);
        b = i + l;
        take(l);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    const int in = at - before, whole = tiles + p.item_cost, item = in / whole;
    tile = in - item * whole;
    h = item / r.blocks(p);
    rb = item - h * r.blocks(p);
    Cut cut{};
    if (tile > 0 && tile < tiles) cut = Cut{r.row0, min(r.rows * p.group - rb * kTileRows, kTileRows), rb * kTileRows, h, at - tile, tiles};
    if (threadIdx.x == 0) {
      p.cuts[blockIdx.x] = cut;
      p.lost[blockIdx.x] = 0;                   // (the same thread sets it when the block ends)
    }
    if (tile >= tiles) {                        // the tiles before belong to the last share
      units -= whole - tile;
      if (units > 0) next_item(p, lane);
    }
  }
  // Tiles of the current item in the share; afterwards done() moves on.
  __device__ __forceinline__ int count() const { return min(tiles - tile, units); }
  __device__ __forceinline__ bool more() const { return units > 0; }
  __device__ __forceinline__ void done(const AttnParams& p, int lane) {
    units -= tiles + p.item_cost - tile;
    if (units > 0) next_item(p, lane);
  }
  __device__ __forceinline__ void next_item(const AttnParams& p, int lane) {
    tile = 0;
    if (++rb == r.blocks(p)) {
      rb = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if ((++b & 31) == 0) load32(p, b, lane);
          take(b & 31);
        } while (r.rows <= 0);
      }
    }
  }
};

// ------------------------------------------------------------------ small steps

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int row, int head, int page) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
               :: "r"(dst), "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c of a row over an E4M3 cache, which holds the scales of the keys and of the row's elements: where it falls below fp32 it stays
// positive, for a key that a row does not see is one with a score of -inf times c.
__device__ __forceinline__ float positive(float c) { return c == 0.f ? 1.401298464e-45f : c; }

// Types of the two matrix products: the query's own, f16 over an E4M3 cache (exact for its values).
template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
  static constexpr uint32_t kExponent = 0x7F807F80u;
  static constexpr float kShift = 0.f;
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <> struct Mma<__half> {
  static constexpr uint32_t kExponent = 0x7C007C00u;
  // f16 probabilities are kept times 2^7, so that those below 2^-14 of the largest do not lose bits, and
  // 2^8 more (kSlack) do not overflow
  static constexpr float kShift = 7.f;
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
// The base of a row's exponents follows its maximum only when that has grown by more than this (log2): any
// base gives the same result, and a new one costs a pass over the output in tensor memory.
constexpr float kSlack = 8.f;

// Visibility of 32 keys from `key` on (bit j: key + j) for a row with node mask `bits`.
__device__ __forceinline__ uint32_t visible32(uint64_t bits, int key, int ctx) {
  const int ahead = ctx - key;                                  // cached tokens among and after them
  if (ahead >= 32) return 0xffffffffu;
  if (ahead > 0) return ((1u << ahead) - 1u) | (uint32_t)(bits << ahead);
  return -ahead < 64 ? (uint32_t)(bits >> -ahead) : 0u;
}

// Values that are not finite. A product with a probability of zero makes NaN of an infinite value: one that f16 rounds to zero, one that
// exp2 does, the zeros of the keys of other copies. The sum of such values with positive weights is the infinity, or NaN if one of them is
// NaN or both infinities occur. So where a column of an item came out as NaN over finite sums, the block looks its values up: which
// columns meet +inf and -inf (NaN is both) in the context, and in each node. Rare, and so after the item's results are stored:
// finite caches cost a comparison per output, a token of NaN in the longest of 16 requests 94 -> 270 us (a search by every thread for
// itself took 8 ms).
constexpr int kJoinThreads = 256;    // threads that join an item's results, in both kernels, on barrier 1
__device__ __forceinline__ bool join_barrier_or(bool mine) {
  uint32_t any;
  asm volatile("{ .reg .pred p, q; setp.ne.u32 q, %1, 0; bar.red.or.pred p, 1, %2, q; selp.u32 %0, 1, 0, p; }"
               : "=r"(any) : "r"((uint32_t)mine), "n"(kJoinThreads) : "memory");
  return any != 0;
}
// Words of found [1 + nodes][D / 32][+inf, -inf]; row 0 is the context.
template <int D> __device__ __forceinline__ constexpr int found_words(int nodes) { return (1 + nodes) * (D / 32) * 2; }
// All kJoinThreads threads; v: the head's values of page 0; keys [first, end).
template <typename T, int D>
static __device__ __noinline__ void find_infinities(uint32_t* found, int id, const uint16_t* v, int64_t page_stride, const int32_t* table, int page_shift,
                                                    int num_pages, int ctx, int first, int end) {
  constexpr uint32_t kExponent = Mma<T>::kExponent;
  constexpr int kPieces = D / 8, kStep = kJoinThreads / kPieces;
  const int piece = id % kPieces;
  uint32_t seen[2] = {0, 0};                                    // of the context
#pragma unroll 8
  for (int key = first + id / kPieces; key < end; key += kStep) {
    const int page = table[key >> page_shift];
    if (page < 0 || page >= num_pages) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(v + page * page_stride + (int64_t)(key & ((1 << page_shift) - 1)) * D + 8 * piece);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t here[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t e = w[j / 2] >> (16 * (j & 1)) & 0xffffu, size = e & 0x7fffu, inf = kExponent & 0xffffu;
      here[0] |= (uint32_t)(size > inf || e == inf) << j;
      here[1] |= (uint32_t)(size > inf || e == (inf | 0x8000u)) << j;
    }
    if (key < ctx) {
      seen[0] |= here[0];
      seen[1] |= here[1];
    } else {
      for (int k = 0; k < 2; ++k)
        if (here[k]) atomicOr(&found[((1 + key - ctx) * (D / 32) + piece / 4) * 2 + k], here[k] << (piece % 4 * 8));
    }
  }
  for (int k = 0; k < 2; ++k)
    if (seen[k]) atomicOr(&found[piece / 4 * 2 + k], seen[k] << (piece % 4 * 8));
}
// A thread's columns of a row that sees the nodes `bits`, in out or part: those that meet one of the infinities (and are it, or NaN).
template <typename T, int D>
static __device__ __noinline__ void mend_columns(T* out, float* part, int column, int columns, const uint32_t* found, uint64_t bits) {
  uint32_t high = 0, low = 0;
  for (int i = 0; i < columns; ++i) {
    const int word = (column + i) / 32, bit = (column + i) % 32;
    if (i == 0 || bit == 0) {
      high = found[2 * word];
      low = found[2 * word + 1];
      for (uint64_t left = bits; left; left &= left - 1) {
        const int row = __ffsll(left) * (D / 32) + word;
        high |= found[2 * row];
        low |= found[2 * row + 1];
      }
    }
    if (!((high ^ low) >> bit & 1)) continue;
    const float x = high >> bit & 1 ? INFINITY : -INFINITY;
    if (out) out[i] = Elem<T>::from_float(x);
    else part[i] = x;
  }
}
// After an item's results are stored and join_barrier_or() of the threads that have NaN over finite sums (odd).
template <typename T, int D>
__device__ __forceinline__ void mend_item(const AttnParams& p, const Walk& w, uint32_t* found, int id, bool odd, T* out, float* part, int column, int columns,
                                          uint64_t bits) {
  for (int i = id; i < found_words<D>(w.r.rows); i += kJoinThreads) found[i] = 0;
  __syncwarp();
  join_barrier_or(false);
  find_infinities<T, D>(found, id, static_cast<const uint16_t*>(p.v) + ((int64_t)w.h << p.page_shift) * D, p.page_stride,
                        p.block_table + (size_t)w.b * p.max_pages, p.page_shift, p.num_pages, w.r.ctx, w.tile * kTileKeys,
                        min(w.r.keys, (w.tile + w.count()) * kTileKeys));
  __syncwarp();
  join_barrier_or(false);
  if (odd) mend_columns<T, D>(out, part, column, columns, found, bits);
  __syncwarp();
  join_barrier_or(false);
}

// Up to kFewRows rows a request and kv head: the kernel of tree_attention_rows.cu. A stage of its copies, and so a box
// of them, has kFewBytes of keys at most.
constexpr int kFewRows = 32, kFewBytes = 4096;
cudaError_t launch_few_rows(const AttnParams& p, bool bf16, bool e4m3, int D, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev,
                            cudaStream_t s);

}  // namespace mdw
