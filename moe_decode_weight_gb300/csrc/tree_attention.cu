// mdw_tree_attention: attention of trees of drafted tokens over the paged key/value cache.
//
// Mathematics. For a row and the keys it sees, with z_j = q . k_j and c = scale * log2(e):
//   o = sum_j 2^(c z_j - c m) v_j / sum_j 2^(c z_j - c m),   lse = ln2 (c m + log2 sum_j 2^(c z_j - c m)),
// for any m; a running maximum keeps the exponents below 0. Partial results (c m, sum, weighted
// values) over disjoint key sets join by rescaling to the larger c m, so the keys of a row can be
// split over warps and blocks and joined in a fixed order. Scores, sums and outputs are fp32. The probabilities
// are rounded to 16 bits for the second product, since an instruction multiplies operands of one type
// and a second product for the rest would double its work: outputs are off by 0.0022 of their norm instead of 0.0017, which is
// their own rounding to bf16 (4-token window; f16, 64-node trees: 0.00029 instead of 0.00021).
//
// Split. The query heads of one kv head and the nodes of one tree are the rows of one tile (node major,
// up to 128 rows), so a key is read from memory once for all of them. The work is the list of
// (request, kv head, row block, 128-key tile), cut into equal contiguous shares, one per block, one block
// per SM: ragged lengths balance, and only the first and last item of a share are partial. Their sums
// go to the workspace and a second, dependent launch joins them.
//
// Both products run on tcgen05 with the rows as the 128 lanes of tensor memory: scores = rows x keys into 128
// columns, then probabilities x values onto D columns of output, the probabilities read from tensor memory.
// Up to 64 (32) rows are laid down two (four) times, and every copy takes the exponentials of a half
// (quarter) of the keys, so that all four schedulers share them; its other probabilities are zeros, and
// the copies' outputs are joined at the end of the item. The tiles of an item alternate between
// two streams with scores, output, maximum and sum of their own, so that one stream's exponentials run
// while the tensor cores work for the other.
//
// Requests of up to 32 rows a kv head have a kernel of their own (tree_attention_rows.cu; few_rows() below chooses).
//
// What bounds it is the stream of keys and values up to 64 rows a block (16 ragged trees of up to 16 nodes x 4 heads, 12k
// keys: 80 us, 5.1 TB/s), and the chain of a tile above (64-node trees of 8 heads: 47 us; a tile of 128 rows
// takes a stream some 5,000 cycles: scores, maximum, exponentials, output). 152 SMs need about 128 KB each in flight to draw the
// memory's full rate (a copy alone, with nothing done to the tiles, reaches 7.1 TB/s so, 16-token
// pages in random order). Keys and values therefore share one ring in the order in which the products
// free them (K0 K1 V0 K2 V1 K3 ...), and a tile is held only while its product runs. The roles of a block:
//   warp 0       requests the tiles by TMA (a box per page, head and 128 bytes of a row, swizzled)
//   warp 1       issues the matrix products
//   warps 2, 3   lay down the rows of the next item while the last one's are in the exponentials, and keep
//                non-finite values that not every row sees out of the products
//   warps 12-15  over an E4M3 cache only: do the latter and turn the tiles into f16 ones, exactly
//   warps 4-7    exponentials of the even tiles, one thread per lane; warps 8-11 of the odd tiles
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mdw_internal.h"
#include "mdw_tcgen05.cuh"
#include "tree_attention.cuh"

namespace mdw {
namespace {

// ------------------------------------------------------------------ the kernel

template <typename T, bool kE4M3, int D>
struct Shape {
  using C = typename std::conditional<kE4M3, __half, T>::type;     // type of the products
  static constexpr int kBytes = kE4M3 ? 1 : 2;
  static constexpr int kRowBytes = D * kBytes < 128 ? D * kBytes : 128;   // one key's row in a copied tile
  static constexpr int kHalves = D * kBytes / kRowBytes;                  // boxes of a page (128 bytes of each key)
  static constexpr int kCopied = kTileKeys * D * kBytes;                  // a copied tile of keys or of values
  static constexpr int kOperand = kTileKeys * D * 2;                      // a 16-bit one
  static constexpr int kSlots = (kE4M3 ? 4 : 5) * (128 / D);              // copied tiles in the ring
  static constexpr int kBuffers = kE4M3 ? 3 * (128 / D) : 0;              // converted tiles
  static constexpr int kClean = kE4M3 ? kBuffers : kSlots;                // operands of the products
  static constexpr int kHelpers = kE4M3 ? 128 : 64;                       // threads of warps 12-15, or of 2 and 3
  static constexpr int kThreads = 32 * (kE4M3 ? 16 : 12);
  static constexpr int kRowsAt = 0, kSlotsAt = kTileRows * D * 2, kBuffersAt = kSlotsAt + kSlots * kCopied;
  // columns of an output that join at a time: few registers over E4M3 (a batch of trees 80 us, with 16 84) and for heads of 64
  // (64-node trees 46.6, 47.6), fewer barriers otherwise (64 requests 75, with 8 77)
  static constexpr int kPiece = kE4M3 || D == 64 ? 8 : 16, kJoinAt = kBuffersAt + kBuffers * kOperand;
  static constexpr int kSmall = kJoinAt + 2 * kTileRows * kPiece * 4;     // small arrays and barriers
  static constexpr int kSmem = kSmall + 2 * kTileRows * 8 + 3 * kTileRows * 4 + 1024;
  // tensor memory columns of a stream: scores (the probabilities take their first half when D = 128), output
  static constexpr int kOut = 128, kProb = D == 128 ? 0 : 192, kStream = 256;

  // 16-byte piece of a key's row in a copied tile, as the TMA swizzle places it.
  static __device__ __forceinline__ uint32_t copied(uint32_t tile, int key, int piece) {
    if constexpr (kRowBytes == 128) return tile + (piece >> 3) * (kTileKeys * 128) + key * 128 + (((piece & 7) ^ (key & 7)) << 4);
    else return tile + key * 64 + ((piece ^ ((key >> 1) & 3)) << 4);
  }
  // The same in a 16-bit operand of 128 rows.
  static __device__ __forceinline__ uint32_t operand(uint32_t tile, int row, int piece) {
    return tile + (piece >> 3) * (128 * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
  }
};

// Place of the keys and of the values of tile i in the order K0 K1 V0 K2 V1 K3 ... of an item of `count` tiles.
__device__ __forceinline__ int keys_unit(int i) { return i < 2 ? i : 2 * i - 1; }
__device__ __forceinline__ int values_unit(int i, int count) { return min(2 * i + 2, 2 * count - 1); }
__device__ __forceinline__ bool is_keys(int unit, int count) {
  return unit == 0 || (unit < 2 ? count > 1 : (unit & 1) && (unit + 1) / 2 < count);
}

// Barriers and small arrays of a block.
struct Small {
  uint32_t full, empty;            // per slot: copied; free again
  uint32_t clean, buffer_free;     // per operand: fit for the product; (converted ones) free again
  uint32_t rows_ready, rows_free;  // the item's rows are in shared memory; its last score product is done
  uint32_t scores, probs, output;  // per stream: scores; probabilities; output of a tile complete
  uint32_t end;
  uint32_t* bad_pages;             // per slot: pages of the tile that lie outside the cache
  uint32_t* tile_bad;              // the same per operand, and then (last two) of the tile in each stream
  uint32_t (*odd)[4];              // per operand: keys with non-finite values (taken out)
  volatile int* dead;
  uint32_t* tmem;
  float2* ml;                      // [2][128] (c m, sum) of the streams' lanes
  float* row_c;                    // [3][128] c of the lanes, by item mod 3: when the rows of item k + 3 are laid
                                   // down, the first tile of item k + 2 has its scores, so item k is done
};

// Those of 32 keys of a tile (from in_tile on) that lie on a page of the cache.
__device__ __forceinline__ uint32_t on_pages32(uint32_t bad, int in_tile, int page_shift) {
  uint32_t v = 0;
  if (!(bad >> (in_tile >> page_shift) & 1)) v |= 0xffffu;
  if (!(bad >> ((in_tile + 16) >> page_shift) & 1)) v |= 0xffff0000u;
  return v;
}

// Rows are laid down 128 / copy_rows times.
__device__ __forceinline__ int copy_rows(int rows) { return rows <= 32 ? 32 : (rows <= 64 ? 64 : 128); }

// What a thread of the exponentials keeps of its lane over an item.
struct Lane {
  float c, mc, l;                  // c; base of the exponents (less kShift); sum
  uint64_t bits;                   // nodes the row sees
  int row, head;                   // of q, out and lse
  bool valid;
};

// Exponentials of one tile for a lane: `cols` keys from key0 on (the share of the lane's copy). The tile holds keys
// that not every row sees unless `all`. Scores lie in the columns from `scores` on, probabilities go to `probs`
// (two to a column), the output so far is in `out`. 32 keys at a time, in loops that stay rolled: the warps of the two
// streams are at different places of this code, and unrolled over the tile it did not stay in the instruction cache
// (64-node trees 56 us instead of 50).
template <typename T, bool kE4M3, int D>
__device__ __forceinline__ void exponentials(const AttnParams& p, Lane& w, uint32_t scores, uint32_t probs, uint32_t out, int key0, int cols,
                                             int tile_key, const Request& r, int b, int h, bool all, uint32_t bad, const uint32_t* odd) {
  using S = Shape<T, kE4M3, D>;
  using M = Mma<typename S::C>;
  float v[32], most = -INFINITY;
  uint32_t see = ~0u;
  auto hide = [&](int at) {
    see = visible32(w.bits, tile_key + key0 + at, r.ctx) & on_pages32(bad, key0 + at, p.page_shift);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = see >> e & 1 ? v[e] : -INFINITY;
  };
#pragma unroll 1
  for (int at = cols - 32; at >= 0; at -= 32) {                // the first part is held when the maximum is known
    float top = tc_ld32_max(v, scores + key0 + at);
    tc_wait_ld();
    if (!all) {
      hide(at);
      top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; ++e) top = fmaxf(top, v[e]);
    }
    most = fmaxf(most, top);
  }
  const float now = most == -INFINITY ? -INFINITY : fmaf(most, w.c, -M::kShift);
  const bool grown = w.valid && now > w.mc + kSlack;            // also from -inf
  if (__any_sync(0xffffffffu, grown)) {
    const float f = grown ? (w.mc == -INFINITY ? 0.f : exp2_fast(w.mc - now)) : 1.f;
    if (__any_sync(0xffffffffu, grown && w.l != 0.f)) {
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
        float o[32];
        tc_ld32(o, out + i);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= f;
        tc_st32(out + i, o);
      }
    }
    w.l *= f;
    if (grown) w.mc = now;
  }
  const float from = w.mc == -INFINITY ? 0.f : w.mc;
#pragma unroll 1
  for (int at = 0; at < cols; at += 32) {
    if (at > 0) {
      tc_ld32(v, scores + key0 + at);
      tc_wait_ld();
      if (!all) hide(at);
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      v[e] = exp2_fast(fmaf(v[e], w.c, -from));
      sum[e & 3] += v[e];
    }
    w.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    uint32_t packed[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) packed[e] = M::pack(v[2 * e], v[2 * e + 1]);
    tc_st16(probs + (key0 + at) / 2, packed);
    if (!all) {
      // rare: keys with values that are NaN or infinite; the rows that see one add them themselves
      for (uint32_t left = odd[(key0 + at) / 32]; left; left &= left - 1) {
        const int k = __ffs(left) - 1, key = tile_key + key0 + at + k;
        float pk = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) pk = e == k ? v[e] : pk;
        const bool seen = w.valid && (see >> k & 1);
        const int64_t page = p.block_table[(size_t)b * p.max_pages + (key >> p.page_shift)];
        const int64_t src = page * p.page_stride + (((int64_t)h << p.page_shift) + (key & ((1 << p.page_shift) - 1))) * D;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float o[32];
          tc_wait_st();
          tc_ld32(o, out + i);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x;
            if constexpr (kE4M3) x = __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(static_cast<const uint8_t*>(p.v)[src + i + e])));
            else x = Elem<T>::to_float(static_cast<const T*>(p.v)[src + i + e]);
            if (seen && !isfinite(x)) o[e] += pk * x;
          }
          tc_st32(out + i, o);
        }
      }
    }
  }
  if (cols < kTileKeys) {                                       // (their columns may have held scores of this share until now)
    const uint32_t none[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
    for (int j = 0; j < kTileKeys; j += 32)
      if (j < key0 || j >= key0 + cols) tc_st16(probs + j / 2, none);
  }
  tc_wait_st();
}

template <typename T, bool kE4M3, int D>
__global__ void __launch_bounds__(Shape<T, kE4M3, D>::kThreads, 1)
tree_attention_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<T, kE4M3, D>;
  using M = Mma<typename S::C>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Small sm;
  {
    uint8_t* at = smem + S::kSmall;
    sm.ml = reinterpret_cast<float2*>(at);
    sm.row_c = reinterpret_cast<float*>(sm.ml + 2 * kTileRows);
    uint32_t bar = smem_u32(sm.row_c + 3 * kTileRows);
    auto take = [&](int n) { const uint32_t r = bar; bar += 8 * n; return r; };
    sm.full = take(S::kSlots);
    sm.empty = take(S::kSlots);
    sm.clean = take(S::kClean);
    sm.buffer_free = take(S::kBuffers);
    sm.rows_ready = take(1);
    sm.rows_free = take(1);
    sm.scores = take(2);
    sm.probs = take(2);
    sm.output = take(2);
    sm.end = take(1);
    uint32_t* word = reinterpret_cast<uint32_t*>(smem + (bar - base));
    sm.odd = reinterpret_cast<uint32_t (*)[4]>(word);
    sm.bad_pages = word + 4 * S::kClean;
    sm.tile_bad = sm.bad_pages + S::kSlots;
    sm.dead = reinterpret_cast<volatile int*>(sm.tile_bad + S::kClean + 2);
    sm.tmem = sm.tile_bad + S::kClean + 3;
  }
  if (base & 1023) {                                            // the swizzled tiles need the alignment asked for above
    if (threadIdx.x == 0) raise_status(p.status, MDW_ERR_UNSUPPORTED_SHAPE);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.total[0] = p.total[1] = 0;
    return;
  }
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(sm.full + 8 * i, 1);
      mbar_init(sm.empty + 8 * i, kE4M3 ? S::kHelpers : 1);
    }
    for (int i = 0; i < S::kClean; ++i) mbar_init(sm.clean + 8 * i, S::kHelpers);
    for (int i = 0; i < S::kBuffers; ++i) mbar_init(sm.buffer_free + 8 * i, 1);
    mbar_init(sm.rows_ready, 64);
    mbar_init(sm.rows_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.scores + 8 * i, 2);
      mbar_init(sm.probs + 8 * i, 4);
      mbar_init(sm.output + 8 * i, 1);
    }
    mbar_init(sm.end, 1);
    *sm.dead = 0;
    mbar_init_fence();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Walk walk;
  walk.begin(p, lane);
  if (!walk.more()) return;                                     // the whole block
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *sm.tmem, 0);
  const uint32_t rows_at = base + S::kRowsAt;
  auto wait = [&](uint32_t bar, uint32_t parity) { mbar_wait(bar, parity, p.spin_budget, p.status, sm.dead); };
  auto slot_at = [&](int slot) { return base + S::kSlotsAt + slot * S::kCopied; };
  auto operand_at = [&](int i) { return kE4M3 ? base + S::kBuffersAt + i * S::kOperand : slot_at(i); };

  if (warp == 0) {
    // ---- copies: lane i serves a tile's i-th page
    const int box_rows = min(1 << p.page_shift, kTileKeys), pages = kTileKeys / box_rows;
    const uint32_t page_bytes = (uint32_t)box_rows * D * S::kBytes;
    int slot = 0;
    uint32_t phase = 0;
    bool lost = false;
    while (walk.more() && !lost) {
      const Request r = walk.r;
      const int tile0 = walk.tile, count = walk.count(), head = walk.h;
      const int32_t* table = p.block_table + (size_t)walk.b * p.max_pages;
      auto look = [&](int i) {                                  // page of the lane in tile i; -1: none wanted, -2: outside the cache
        const int key = (tile0 + i) * kTileKeys + lane * box_rows;
        if (i >= count || lane >= pages || key >= r.keys) return -1;
        const int id = table[key >> p.page_shift];
        return id >= 0 && id < p.num_pages ? id : -2;
      };
      // pages of the tile whose values come next and of the two after it
      int id0 = look(0), id1 = look(1), id2 = look(2);
      for (int u = 0; u < 2 * count; ++u) {
        const bool keys = is_keys(u, count);
        const int id = keys && u > 0 ? id1 : id0, i = keys ? (u + 1) / 2 : (u == 2 * count - 1 ? count - 1 : u / 2 - 1);
        const unsigned good = __ballot_sync(0xffffffffu, id >= 0), bad = __ballot_sync(0xffffffffu, id == -2);
        wait(sm.empty + 8 * slot, phase ^ 1);
        if (__any_sync(0xffffffffu, *sm.dead)) { lost = true; break; }
        const uint32_t bar = sm.full + 8 * slot, to = slot_at(slot);
        if (lane == 0) {
          sm.bad_pages[slot] = bad;
          if (bad) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
          mbar_arrive_tx(bar, page_bytes * __popc(good));
        }
        __syncwarp();
        if (id >= 0) {
          const int row = ((tile0 + i) * kTileKeys + lane * box_rows) & ((1 << p.page_shift) - 1);
#pragma unroll
          for (int k = 0; k < S::kHalves; ++k)
            tma_load(to + k * (kTileKeys * S::kRowBytes) + lane * box_rows * S::kRowBytes, keys ? &kmap : &vmap, bar,
                     k * (S::kRowBytes / S::kBytes), row, head, id);
        }
        if (++slot == S::kSlots) { slot = 0; phase ^= 1; }
        if (!keys) {
          id0 = id1;
          id1 = id2;
          id2 = look(i + 3);
        }
      }
      walk.done(p, lane);
    }
    // Every copy arrives before the block ends, also where a wait runs out after the last one was requested: warp 0 waits
    // for each slot's last one (a slot that was never filled has its phase before the first, which is over).
    for (int i = 0; i < S::kSlots; ++i) mbar_drain(sm.full + 8 * i, i < slot ? phase : phase ^ 1);
  } else if (warp == 1) {
    // ---- products. Scores of the first two tiles of an item, then in turn the output of tile i and the scores
    // of tile i + 2, whose columns hold the probabilities that output reads.
    int unit0 = 0, items = 0, done[2] = {0, 0};                 // units before this item; items; outputs of each stream
    while (walk.more()) {
      const int count = walk.count();
      auto scores = [&](int i) {
        const int unit = unit0 + keys_unit(i), at = unit % S::kClean, s = i & 1;
        // (also where nothing is done to keys: the helper warps wait for every copy, and one that came to a slot after its
        // next copy would wait for the one after that, and hold up everything)
        wait(sm.clean + 8 * at, unit / S::kClean & 1);
        tc_fence_after();
        const uint32_t rows_low = operand_low(rows_at, 16), keys_low = operand_low(operand_at(at), 16), to = tmem + s * S::kStream;
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            const uint32_t off = ((t >> 2) * (128 * 128) + (t & 3) * 32) >> 4;
            tc_mma(to, rows_low + off, keys_low + off, mma_shape(M::kBf16, false, kTileKeys), t > 0);
          }
          tc_commit(sm.scores + 8 * s);
          sm.tile_bad[S::kClean + s] = kE4M3 ? sm.tile_bad[at] : sm.bad_pages[at];
          mbar_arrive(sm.scores + 8 * s);
          tc_commit((kE4M3 ? sm.buffer_free : sm.empty) + 8 * at);
          if (i == count - 1) tc_commit(sm.rows_free);
        }
        __syncwarp();
      };
      wait(sm.rows_ready, items & 1);
      // the columns of the scores hold probabilities until the last output that reads them is complete
      for (int i = 0; i < 2 && i < count; ++i) {
        if (done[i] > 0) wait(sm.output + 8 * i, (done[i] - 1) & 1);
        scores(i);
      }
      for (int i = 0; i < count; ++i) {
        const int unit = unit0 + values_unit(i, count), at = unit % S::kClean, s = i & 1;
        wait(sm.clean + 8 * at, unit / S::kClean & 1);
        wait(sm.probs + 8 * s, done[s] & 1);
        tc_fence_after();
        const uint32_t values_low = operand_low(operand_at(at), 128 * 128), stream = tmem + s * S::kStream;
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < kTileKeys / 16; ++t)
            tc_mma_tmem(stream + S::kOut, stream + S::kProb + 8 * t, values_low + t * (2048 >> 4), mma_shape(M::kBf16, true, D), true);
          tc_commit(sm.output + 8 * s);
          tc_commit((kE4M3 ? sm.buffer_free : sm.empty) + 8 * at);
        }
        __syncwarp();
        if (i + 2 < count) {
          // where the probabilities have columns of their own, the scores may follow at once: their completion
          // includes the output's
          if (S::kProb < kTileKeys) wait(sm.output + 8 * s, done[s] & 1);
          scores(i + 2);
        }
        ++done[s];
      }
      unit0 += 2 * count;
      ++items;
      walk.done(p, lane);
    }
    if (lane == 0) tc_commit(sm.end);
    __syncwarp();
    mbar_drain(sm.end, 0);                                      // nothing is in flight when the columns are given back
  } else if (warp < 4 || warp >= 12) {
    // ---- warps 2, 3: the rows of an item, as soon as the last item's scores are complete. They (or warps 12-15 over
    // an E4M3 cache) also go over the tiles: where not every row sees all of a tile, non-finite values are
    // taken out and noted per key (the rows that see them add them); E4M3 tiles are converted
    const int id = kE4M3 ? threadIdx.x - 384 : threadIdx.x - 64;
    int slot = 0, buffer = 0, items = 0;
    uint32_t phase = 0, buffer_phase = 0;
    while (walk.more()) {
      const Request r = walk.r;
      const int tile0 = walk.tile, count = walk.count(), h = walk.h;
      if (warp < 4) {
        if (items > 0) wait(sm.rows_free, (items - 1) & 1);
        const int first = walk.rb * kTileRows, rows = min(r.rows * p.group - first, kTileRows), per = copy_rows(rows);
#pragma unroll 1
        for (int at = threadIdx.x - 64; at < kTileRows; at += 64) {
          const int mine = at & (per - 1), flat = first + mine, node = flat / p.group;
          if (mine >= rows) continue;
          const T* src = static_cast<const T*>(p.q) + (int64_t)(r.row0 + node) * p.ldq + (int64_t)(h * p.group + flat - node * p.group) * D;
          if constexpr (!kE4M3) {
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) sts16(S::operand(rows_at, at, i), *reinterpret_cast<const uint4*>(src + 8 * i));
          } else {
            float f = 1.f, c = p.scale * kLog2e * p.k_scale[h];
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
              // bf16 rows enter f16, the type of the converted keys, times a power of two that puts their largest element in [1, 4):
              // elements below 2^-17 of it are off by up to 2^-25 of it, far below the fp32 sums' own error
              float top = 0.f;
#pragma unroll 8
              for (int i = 0; i < D / 8; ++i) {
                T x[8];
                const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * i);
                memcpy(x, &v, 16);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(Elem<T>::to_float(x[e])));
              }
              const int ex = top > 0.f && isfinite(top) ? min((int)(__float_as_uint(top) >> 23) - 127, 126) : 0;
              f = __uint_as_float((uint32_t)(127 - ex) << 23);
              c *= ex >= -126 ? __uint_as_float((uint32_t)(127 + ex) << 23) : 5.877471754111438e-39f;
            }
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
              T x[8];
              uint4 v = *reinterpret_cast<const uint4*>(src + 8 * i);
              memcpy(x, &v, 16);
              v = make_uint4(M::pack(Elem<T>::to_float(x[0]) * f, Elem<T>::to_float(x[1]) * f), M::pack(Elem<T>::to_float(x[2]) * f, Elem<T>::to_float(x[3]) * f),
                             M::pack(Elem<T>::to_float(x[4]) * f, Elem<T>::to_float(x[5]) * f), M::pack(Elem<T>::to_float(x[6]) * f, Elem<T>::to_float(x[7]) * f));
              sts16(S::operand(rows_at, at, i), v);
            }
            sm.row_c[items % 3 * kTileRows + at] = positive(c);
          }
        }
        fence_async_proxy();
        mbar_arrive(sm.rows_ready);
        ++items;
        if (kE4M3) {
          walk.done(p, lane);
          continue;
        }
      }
      for (int u = 0; u < 2 * count; ++u) {
        const bool keys = is_keys(u, count);
        const int i = keys ? (u + 1) / 2 : (u == 2 * count - 1 ? count - 1 : u / 2 - 1), tile_key = (tile0 + i) * kTileKeys;
        wait(sm.full + 8 * slot, phase);
        const uint32_t bad = sm.bad_pages[slot], from = slot_at(slot);
        const int b = kE4M3 ? buffer : slot;
        const bool all = keys || (tile_key + kTileKeys <= r.ctx && bad == 0);
        if constexpr (kE4M3) wait(sm.buffer_free + 8 * b, buffer_phase ^ 1);
        if (id == 0) sm.tile_bad[b] = bad;
        if (!all) {
          if (id < 4) sm.odd[b][id] = 0;
          asm volatile("bar.sync 2, %0;" :: "n"(S::kHelpers) : "memory");
        }
        auto note = [&](uint32_t non, int key) {
          if (non && tile_key + key < r.keys && !(bad >> (key >> p.page_shift) & 1)) atomicOr(&sm.odd[b][key >> 5], 1u << (key & 31));
        };
        if constexpr (!kE4M3) {
          if (!all)
            for (int j = id; j < kTileKeys * (D / 8); j += S::kHelpers) {
              const int key = j / (D / 8);
              const uint32_t at = S::copied(from, key, j % (D / 8));
              const uint4 v = lds16(at);
              const uint32_t e = M::kExponent;
              const uint4 non = make_uint4(__vcmpeq2(v.x & e, e), __vcmpeq2(v.y & e, e), __vcmpeq2(v.z & e, e), __vcmpeq2(v.w & e, e));
              if (non.x | non.y | non.z | non.w) {
                sts16(at, make_uint4(v.x & ~non.x, v.y & ~non.y, v.z & ~non.z, v.w & ~non.w));
                note(1u, key);
              }
            }
        } else {
          const uint32_t to = operand_at(b);
          // thread: one 16-byte piece of every kStep-th key, at the same place of the swizzle each time
          constexpr int kPieces = D / 16, kStep = S::kHelpers / kPieces;
          const int key0 = id / kPieces, piece = id % kPieces;
          const bool swap = piece >= 4;                         // the two halves of an operand share banks: even pieces of one with odd ones of the other
          const uint32_t src = S::copied(from, key0, piece), lo = S::operand(to, key0, 2 * piece), hi = S::operand(to, key0, 2 * piece + 1);
#pragma unroll
          for (int k0 = 0; k0 < kTileKeys / kStep; k0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = lds16(src + (k0 + k) * kStep * S::kRowBytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (!all) {
                // the only non-finite code is S.1111.111
                const uint32_t m = 0x7f7f7f7fu;
                const uint4 non = make_uint4(__vcmpeq4(v[k].x & m, m), __vcmpeq4(v[k].y & m, m), __vcmpeq4(v[k].z & m, m), __vcmpeq4(v[k].w & m, m));
                note(non.x | non.y | non.z | non.w, key0 + (k0 + k) * kStep);
                v[k] = make_uint4(v[k].x & ~non.x, v[k].y & ~non.y, v[k].z & ~non.z, v[k].w & ~non.w);
              }
              const uint32_t a0 = swap ? v[k].z : v[k].x, a1 = swap ? v[k].w : v[k].y, b0 = swap ? v[k].x : v[k].z, b1 = swap ? v[k].y : v[k].w;
              sts16((swap ? hi : lo) + (k0 + k) * kStep * 128, make_uint4(e4m3x2_to_f16x2(a0 & 0xffffu), e4m3x2_to_f16x2(a0 >> 16),
                                                                          e4m3x2_to_f16x2(a1 & 0xffffu), e4m3x2_to_f16x2(a1 >> 16)));
              sts16((swap ? lo : hi) + (k0 + k) * kStep * 128, make_uint4(e4m3x2_to_f16x2(b0 & 0xffffu), e4m3x2_to_f16x2(b0 >> 16),
                                                                          e4m3x2_to_f16x2(b1 & 0xffffu), e4m3x2_to_f16x2(b1 >> 16)));
            }
          }
          mbar_arrive(sm.empty + 8 * slot);
        }
        if (kE4M3 || !all) fence_async_proxy();
        mbar_arrive(sm.clean + 8 * b);
        if (++slot == S::kSlots) { slot = 0; phase ^= 1; }
        if (kE4M3 && ++buffer == S::kBuffers) { buffer = 0; buffer_phase ^= 1; }
      }
      walk.done(p, lane);
    }
  } else {
    // ---- exponentials: thread = lane of tensor memory
    const int s = warp >= 8 ? 1 : 0, at_lane = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
    const uint32_t scores = tmem + s * S::kStream + lanes, probs = scores + S::kProb, out = scores + S::kOut;
    int unit0 = 0, items = 0, done = 0;                         // units before this item; items; tiles of this stream
    while (walk.more()) {
      const Request r = walk.r;
      const int first = walk.rb * kTileRows, rows = min(r.rows * p.group - first, kTileRows), h = walk.h;
      const int tile0 = walk.tile, count = walk.count();
      const bool whole = count == walk.tiles;
      // rows in a copy, the lane's row and the first key of its share of a tile
      const int per = copy_rows(rows), mine = at_lane & (per - 1), key0 = at_lane & ~(per - 1);
      const bool active = (warp & 3) * 32 % per < rows;
      Lane w;
      w.valid = mine < rows;
      const int flat = first + (w.valid ? mine : 0), node = flat / p.group;
      w.row = r.row0 + node;
      w.head = h * p.group + flat - node * p.group;
      w.c = p.scale * kLog2e * (kE4M3 ? p.k_scale[h] : 1.f);
      w.bits = 0;
      if (w.valid) {
        w.bits = p.tree_mask ? p.tree_mask[w.row] : ~0ull >> (63 - node);
        if (r.rows < 64) w.bits &= (1ull << r.rows) - 1;
      }
      w.mc = -INFINITY;
      w.l = 0.f;
      if (active) {
        float zero[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) zero[e] = 0.f;
#pragma unroll
        for (int i = 0; i < D; i += 32) tc_st32(out + i, zero);
        tc_wait_st();
      }
      for (int i = s; i < count; i += 2) {
        const int tile_key = (tile0 + i) * kTileKeys;
        wait(sm.scores + 8 * s, done & 1);
        if (kE4M3 && i == s) w.c = sm.row_c[items % 3 * kTileRows + at_lane];
        const uint32_t bad = sm.tile_bad[S::kClean + s];
        const bool all = tile_key + kTileKeys <= r.ctx && bad == 0;
        const int value = unit0 + values_unit(i, count);
        if (!all) wait(sm.clean + 8 * (value % S::kClean), value / S::kClean & 1);
        // (the notes of a block that gave up are another tile's: they name keys behind the sequence, or pages outside the cache)
        const bool lost = __any_sync(0xffffffffu, !all && *sm.dead);
        if (active && !lost) {
          tc_fence_after();
          const uint32_t* odd = sm.odd[value % S::kClean];
          exponentials<T, kE4M3, D>(p, w, scores, probs, out, key0, per, tile_key, r, walk.b, h, all, bad, odd);
          tc_fence_before();
        }
        ++done;
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.probs + 8 * s);
      }

      // ---- the item's result: the two streams of a lane and the copies of a row on one base; this thread adds the
      // streams of half of the columns, and the copies add up over shared memory
      constexpr int kHalf = D / 2, kPiece = S::kPiece;
      if (count > s) wait(sm.output + 8 * s, (done - 1) & 1);
      __syncwarp();
      tc_fence_after();
      sm.ml[s * kTileRows + at_lane] = make_float2(w.mc, w.l);
      tc_fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tc_fence_after();
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * kTileRows / 32; ++j)
        if (32 * j % per == 0) m = fmaxf(m, sm.ml[mine + 32 * j].x);
      const float from = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int j = 0; j < 2 * kTileRows / 32; ++j)
        if (32 * j % per == 0) sum += sm.ml[mine + 32 * j].y * exp2_fast(sm.ml[mine + 32 * j].x - from);
      float fa = exp2_fast(sm.ml[at_lane].x - from), fb = exp2_fast(sm.ml[kTileRows + at_lane].x - from);
      if (whole) {
        const float f = sum == 0.f ? 0.f : (kE4M3 ? p.v_scale[h] : 1.f) / sum;
        fa *= f;
        fb *= f;
      }
      const int slot = 2 * blockIdx.x + (tile0 > 0 ? 0 : 1);
      bool nan = false;
#pragma unroll 1
      for (int i = s * kHalf; i < (s + 1) * kHalf; i += kPiece) {
        float o[kPiece];
        if (active) {
          float x[kPiece];
          tc_ld(x, tmem + lanes + S::kOut + i);
          tc_ld(o, tmem + lanes + S::kStream + S::kOut + i);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < kPiece; ++e) o[e] = fa * x[e] + fb * o[e];
        }
        // columns 4 c .. 4 c + 3 of lane x at (128 c + x) * 16 bytes
        const uint32_t place = base + S::kJoinAt + s * (kPiece / 4 * kTileRows * 16) + at_lane * 16;
        if (per < kTileRows) {
          if (at_lane >= per)
#pragma unroll
            for (int e = 0; e < kPiece; e += 4)
              sts16(place + e / 4 * kTileRows * 16, make_uint4(__float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]), __float_as_uint(o[e + 3])));
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (at_lane < per)
            for (int copy = per; copy < kTileRows; copy += per)
#pragma unroll
              for (int e = 0; e < kPiece; e += 4) {
                const uint4 v = lds16(place + copy * 16 + e / 4 * kTileRows * 16);
                o[e] += __uint_as_float(v.x);
                o[e + 1] += __uint_as_float(v.y);
                o[e + 2] += __uint_as_float(v.z);
                o[e + 3] += __uint_as_float(v.w);
              }
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        if (at_lane < per && w.valid && !*sm.dead) {
          if constexpr (!kE4M3)
#pragma unroll
            for (int e = 0; e < kPiece; ++e) nan |= isnan(o[e]);
          if (whole) {
            T* dst = static_cast<T*>(p.out) + (int64_t)w.row * p.ldo + (int64_t)w.head * D + i;
#pragma unroll
            for (int e = 0; e < kPiece; e += 8) {
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (sum != 0.f)
                v = make_uint4(Mma<T>::pack(o[e], o[e + 1]), Mma<T>::pack(o[e + 2], o[e + 3]), Mma<T>::pack(o[e + 4], o[e + 5]), Mma<T>::pack(o[e + 6], o[e + 7]));
              *reinterpret_cast<uint4*>(dst + e) = v;
            }
          } else {
            float* dst = p.part_o + ((size_t)slot * kTileRows + mine) * D + i;
#pragma unroll
            for (int e = 0; e < kPiece; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        __syncwarp();
      }
      if (s == 0 && at_lane < per && w.valid && !*sm.dead) {
        if (!whole) p.part_ml[(size_t)slot * kTileRows + mine] = make_float2(m, sum);
        else if (p.lse) p.lse[(int64_t)w.row * p.Hq + w.head] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
      }
      __syncwarp();
      tc_fence_before();
      // outputs and sums are read; the next item may begin
      if constexpr (kE4M3) {
        asm volatile("bar.sync 1, 256;" ::: "memory");
      } else if (const bool odd = nan && isfinite(sum); join_barrier_or(odd)) {
        T* out = whole ? static_cast<T*>(p.out) + (int64_t)w.row * p.ldo + (int64_t)w.head * D + s * kHalf : nullptr;
        mend_item<T, D>(p, walk, reinterpret_cast<uint32_t*>(smem + S::kJoinAt), threadIdx.x - 128, odd, out,
                        p.part_o + ((size_t)slot * kTileRows + mine) * D + s * kHalf, s * kHalf, kHalf, w.bits);
      }
      tc_fence_after();
      unit0 += 2 * count;
      ++items;
      walk.done(p, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *sm.dead) p.lost[blockIdx.x] = 1;
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
  }
}

// Joins the partial items: block x belongs to the boundary before share x + 1, and works if it is the first one
// inside its item. One warp per row, a lane D / 32 columns, the shares' sums in order.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(const AttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  // (loaded together: cuts of blocks without a share hold what an earlier call left, and are not used)
  const int total = p.total[0], blocks = p.total[1];
  const Cut cut = p.cuts[blockIdx.x + 1];
  if ((int)blockIdx.x + 1 >= blocks || cut.rows == 0) return;
  const Shares shares(total, blocks);
  if (shares.start(blockIdx.x) > cut.start) return;             // an earlier boundary is inside too
  const int c0 = blockIdx.x, parts = shares.owner(cut.start + cut.tiles - 1) - c0 + 1;
  int lost = lane < parts ? p.lost[c0 + lane] : 0;              // (looked at when the sums are there)
  for (int i = lane + 32; i < parts; i += 32) lost |= p.lost[c0 + i];
  for (int row = blockIdx.y * 4 + (threadIdx.x >> 5); row < cut.rows; row += 4 * gridDim.y) {
    // the item's first part is the last of its block's share, the others are the first of theirs
    auto slot = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * kTileRows + row; };
    float2 ml = make_float2(-INFINITY, 0.f);                    // of part `lane`
    if (lane < parts) ml = p.part_ml[slot(lane)];
    constexpr int kAhead = 8;                                   // parts whose outputs are loaded with the sums
    float v[kAhead][kPer];
    auto load = [&](int first) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float* src = p.part_o + slot(min(first + u, parts - 1)) * D + lane * kPer;
        if constexpr (kPer == 4) *reinterpret_cast<float4*>(v[u]) = __ldcg(reinterpret_cast<const float4*>(src));
        else *reinterpret_cast<float2*>(v[u]) = __ldcg(reinterpret_cast<const float2*>(src));
      }
    };
    load(0);
    float mc = ml.x;
    for (int i = lane + 32; i < parts; i += 32) mc = fmaxf(mc, p.part_ml[slot(i)].x);
    mc = warp_max(mc);
    const float base = mc == -INFINITY ? 0.f : mc;
    float o[kPer], f = 0.f, l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = 0.f;
    for (int i = 0; i < parts; i += kAhead) {
      if (i % 32 == 0) {
        if (i > 0) ml = i + lane < parts ? p.part_ml[slot(i + lane)] : make_float2(-INFINITY, 0.f);
        f = exp2_fast(ml.x - base);
        l = fmaf(ml.y, f, l);
      }
      if (i > 0) load(i);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float g = __shfl_sync(0xffffffffu, f, (i + u) & 31);
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] = i + u < parts ? fmaf(v[u][j], g, o[j]) : o[j];
      }
    }
    l = warp_sum(l);
    if (__any_sync(0xffffffffu, lost)) return;                  // a part is missing
    const int flat = cut.first + row, node = flat / p.group, head = cut.h * p.group + flat - node * p.group;
    const float norm = l == 0.f ? 0.f : (p.v_scale ? p.v_scale[cut.h] : 1.f) / l;
    T* dst = static_cast<T*>(p.out) + (int64_t)(cut.row0 + node) * p.ldo + (int64_t)head * D + lane * kPer;
    uint32_t packed[kPer / 2];
#pragma unroll
    for (int j = 0; j < kPer; j += 2) packed[j / 2] = l == 0.f ? 0u : Mma<T>::pack(o[j] * norm, o[j + 1] * norm);
    if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
    else *reinterpret_cast<uint32_t*>(dst) = packed[0];
    if (p.lse && lane == 0) p.lse[(int64_t)(cut.row0 + node) * p.Hq + head] = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
  }
}

// ------------------------------------------------------------------ host

// Which kernel. Up to 16 rows: few_rows_kernel (one token over 131k E4M3 keys 51 us, the other kernel 86; 1,500 16-bit keys
// 10.4 and 14.7; 131k 16-bit keys 90 and 88). Up to 32 rows, of which two warps share the copies: the same over E4M3 caches
// and heads of 64 (batches of trees 72 and 79 us, 51 and 64, 51 and 59). Over a 16-bit cache with heads of 128 neither is always the
// faster one: a window of 20 rows over 1,500 keys takes 11.5 and 14.8 us, over 9,600 keys (two tiles a block) 17.8 and
// 18.2, over 40,000 31.5 and 29.5, a batch of trees 88 and 77. The lengths are on the device, so the choice goes by what the
// block table has room for, two tiles a block: a short window with a table of 32k tokens takes the slower kernel, and its
// last bits follow the table's width.
bool few_rows(const AttnParams& p, int key_bytes, int grid) {
  const int rows = p.max_new * p.group;
  if (rows <= 16) return true;
  if (rows > kFewRows) return false;
  const int64_t tiles = (((int64_t)p.max_pages << p.page_shift) + kTileKeys - 1) / kTileKeys * p.B * p.Hkv;
  return key_bytes < 256 || tiles <= 2 * grid;
}

// The cache as [pages][heads][page size][head dim]; a box is up to `most` rows of one page and head, 128 bytes (or
// a whole 64-byte row) wide.
bool encode_cache(CUtensorMap* map, const mdw_kv_cache* c, void* data, int most) {
  const bool fp8 = c->dtype == MDW_DT_E4M3;
  const cuuint64_t e = fp8 ? 1 : 2, d = c->head_dim, ps = c->page_size;
  const cuuint64_t dims[4] = {d, ps, (cuuint64_t)c->kv_heads, (cuuint64_t)c->num_pages};
  const cuuint64_t strides[3] = {d * e, d * ps * e, (cuuint64_t)c->page_stride * e};
  const cuuint32_t width = (cuuint32_t)(d * e < 128 ? d : 128 / e);
  const cuuint32_t box[4] = {width, std::min((cuuint32_t)ps, (cuuint32_t)most), 1, 1}, ones[4] = {1, 1, 1, 1};
  const EncodeTiledFn fn = encode_tiled();
  return fn && fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, data, dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, width * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttnWs {
  size_t cuts, lost, ml, o, total;
};
AttnWs attn_ws(int grid, int D) {
  AttnWs w;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  w.cuts = 256;
  w.lost = w.cuts + up((size_t)grid * sizeof(Cut));
  w.ml = w.lost + up((size_t)grid * 4);
  w.o = w.ml + up((size_t)grid * 2 * kTileRows * 8);
  w.total = w.o + up((size_t)grid * 2 * kTileRows * D * 4);
  return w;
}

template <typename T, bool kE4M3, int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  using S = Shape<T, kE4M3, D>;
  cudaError_t e;
  if (few_rows(p, D * S::kBytes, grid)) {
    e = launch_few_rows(p, std::is_same<T, __nv_bfloat16>::value, kE4M3, D, km, vm, grid, dev, s);
    if (e != cudaSuccess) return e;
  } else {
    e = allow_shared_memory<tree_attention_kernel<T, kE4M3, D>>(dev);
    if (e != cudaSuccess) return e;
    tree_attention_kernel<T, kE4M3, D><<<grid, S::kThreads, S::kSmem, s>>>(p, km, vm);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (grid == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(grid - 1), (unsigned)std::min((std::min(p.max_new * p.group, kTileRows) + 3) / 4, 8));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D>, p);
}
template <typename T, bool kE4M3>
cudaError_t launch(const AttnParams& p, int D, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  return D == 64 ? launch<T, kE4M3, 64>(p, km, vm, grid, dev, s) : launch<T, kE4M3, 128>(p, km, vm, grid, dev, s);
}

bool sizes_ok(const mdw_kv_cache* c, int32_t B, int32_t T, int32_t q_heads, int32_t max_new) {
  return B >= 1 && B <= MDW_MAX_REQUESTS && T >= 1 && max_new >= 1 && max_new <= MDW_MAX_TREE && q_heads >= 1 &&
         q_heads % c->kv_heads == 0 && q_heads / c->kv_heads <= MDW_MAX_GROUP;
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" size_t mdw_tree_attention_workspace_bytes(const mdw_kv_cache* cache, int32_t B, int32_t T,
                                                     int32_t q_heads, int32_t max_new) {
  if (check_kv_cache(cache) != MDW_OK || !sizes_ok(cache, B, T, q_heads, max_new)) return 0;
  const int grid = sm_count(current_device());
  if (grid <= 0) return 0;
  return attn_ws(grid, cache->head_dim).total;
}

extern "C" mdw_status mdw_tree_attention(const mdw_kv_cache* cache, int32_t B, int32_t T, int32_t q_heads,
                                         int32_t max_new, const void* q, int64_t ldq, int32_t q_dtype, void* out,
                                         int64_t ldo, float* lse, const int32_t* block_table, int32_t max_pages,
                                         const int32_t* ctx_len, const int32_t* row_start,
                                         const uint64_t* tree_mask, float scale, uint32_t* status, void* ws,
                                         size_t ws_bytes, mdw_stream_t stream) {
  const mdw_status st = check_kv_cache(cache);
  if (st != MDW_OK) return st;
  if (q_dtype != MDW_DT_BF16 && q_dtype != MDW_DT_F16) return MDW_ERR_FORMAT_MISMATCH;
  const bool fp8 = cache->dtype == MDW_DT_E4M3;
  if (!fp8 && q_dtype != cache->dtype) return MDW_ERR_FORMAT_MISMATCH;
  if (!sizes_ok(cache, B, T, q_heads, max_new)) return MDW_ERR_INVALID_ARG;
  if (max_pages < 1 || (int64_t)max_pages * cache->page_size > 0x7fff0000LL) return MDW_ERR_UNSUPPORTED_SHAPE;   // (keys of a tile past the last are int32)
  const int64_t width = (int64_t)q_heads * cache->head_dim;
  if (!aligned_to(q, 16) || !row_stride_ok(ldq, width) || !aligned_to(out, 16) || !row_stride_ok(ldo, width) ||
      !null_or_aligned(lse, 4) || !aligned_to(block_table, 4) || !aligned_to(ctx_len, 4) ||
      !aligned_to(row_start, 4) || !null_or_aligned(tree_mask, 8) || !null_or_aligned(status, 4) || !aligned_to(ws, 16))
    return MDW_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MDW_ERR_INVALID_ARG;
  const int dev = current_device(), grid = sm_count(dev);
  const AttnWs lay = attn_ws(std::max(grid, 1), cache->head_dim);
  if (ws_bytes < lay.total) return MDW_ERR_WORKSPACE_TOO_SMALL;
  if (grid <= 0) return MDW_ERR_CUDA;
  uint8_t* base = static_cast<uint8_t*>(ws);
  AttnParams p{cache->v, cache->page_stride, cache->k_scale, cache->v_scale, q, out, lse, ldq, ldo, block_table, ctx_len, row_start, tree_mask, status,
                     mdw_spin_budget(), scale, B, T, q_heads, cache->kv_heads, q_heads / cache->kv_heads, max_new, max_pages,
                     cache->num_pages, log2_of(cache->page_size), kItemCost, reinterpret_cast<int32_t*>(base),
                     reinterpret_cast<Cut*>(base + lay.cuts), reinterpret_cast<int32_t*>(base + lay.lost), reinterpret_cast<float2*>(base + lay.ml),
                     reinterpret_cast<float*>(base + lay.o)};
  CUtensorMap km, vm;
  const int D = cache->head_dim, key_bytes = D * (fp8 ? 1 : 2);
  const bool few = few_rows(p, key_bytes, grid);
  const int most = few ? kFewBytes / key_bytes : kTileKeys;
  if (few) p.item_cost = p.max_new * p.group <= 16 ? kItemCost16 : kItemCost32;
  if (!encode_cache(&km, cache, cache->k, most) || !encode_cache(&vm, cache, cache->v, most)) return MDW_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (q_dtype == MDW_DT_BF16)
    e = fp8 ? launch<__nv_bfloat16, true>(p, D, km, vm, grid, dev, s) : launch<__nv_bfloat16, false>(p, D, km, vm, grid, dev, s);
  else
    e = fp8 ? launch<__half, true>(p, D, km, vm, grid, dev, s) : launch<__half, false>(p, D, km, vm, grid, dev, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
