// mdw_tree_attention: attention of trees of drafted tokens over the paged key/value cache.
//
// Mathematics. For a row and the keys it sees, with z_j = q . k_j and c = scale * log2(e):
//   o = sum_j 2^(c z_j - c m) v_j / sum_j 2^(c z_j - c m),   lse = ln2 (c m + log2 sum_j 2^(c z_j - c m)),
// for any m; a running maximum keeps the exponents below 0. Partial results (c m, sum, weighted
// values) over disjoint key sets join by rescaling to the larger c m, so the keys of a row can be
// split over warps and blocks and joined in a fixed order.
//
// Split. The query heads of one kv head and the nodes of one tree are the rows of one tile (node major,
// up to 64 rows), so a key is read from memory once for all of them. The work is the list of
// (request, kv head, row block, 128-key tile), cut into equal contiguous shares, one per block, one block
// per SM: ragged lengths balance, and only the first and last item of a share are partial. Their sums
// go to the workspace and a second, dependent launch joins them.
//
// A block is eight warps, which share no barrier inside an item: each takes 16 rows and a slice of the
// tile's keys (16 keys each of one row tile, or 32 or 64 of one of two or four row tiles) and keeps
// its own maximum, sum and output in registers. The pages of a tile come by TMA (one box of 128 or 64
// bytes per key and head half, swizzled, so that ldmatrix reads it without bank conflicts) into a
// ring of stages that warp 0 keeps filled; a warp of its own for that would leave the others 168
// registers, and they spill.
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mdw_attn.cuh"
#include "mdw_device.cuh"
#include "mdw_internal.h"

namespace mdw {
namespace {

constexpr int kTileKeys = 128;        // keys of a tile (one pipeline stage)
constexpr int kTileRows = 64;         // rows of a row block
constexpr int kConsumers = 8;         // warps, the first of which also requests the tiles
constexpr int kAttnThreads = 32 * kConsumers;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnParams {
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
  int B, T, Hq, Hkv, group, max_new, max_pages, num_pages, page_shift;
  // workspace
  int32_t* total;          // [2] tiles of the whole call, blocks with a share
  struct Cut* cuts;        // [grid] the item that a block's share starts inside of
  float2* part_ml;         // [2 * grid][64] (c m, sum) of partial items
  float* part_o;           // [2 * grid][64][D] their unnormalised outputs
};

// An item that a share boundary cuts; rows = 0: the share starts with a whole item.
struct Cut {
  int row0, rows, first, h;        // request's first row, rows of the block (of rows x heads), its first one, kv head
  int start, tiles;                // first tile of the item, its tiles
};

// ------------------------------------------------------------------ requests and shares

struct Request {
  int row0, rows, ctx, keys;       // first row, rows, cached tokens, keys; rows < 0: not valid
  __device__ __forceinline__ int blocks(const AttnParams& p) const { return (rows * p.group + kTileRows - 1) / kTileRows; }
  __device__ __forceinline__ int tiles() const { return (keys + kTileKeys - 1) / kTileKeys; }
  __device__ __forceinline__ int64_t work(const AttnParams& p) const {
    return rows <= 0 ? 0 : (int64_t)p.Hkv * blocks(p) * tiles();
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

// Equal contiguous shares of `total` tiles: block c has tiles [start(c), start(c + 1)). No share is empty, so every
// partial slot that a join reads was written.
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
  int left;                        // tiles left in the share

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
    left = 0;
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
    left = shares.start(blockIdx.x + 1) - at;
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
    const int in = at - before, item = in / tiles;
    tile = in - item * tiles;
    h = item / r.blocks(p);
    rb = item - h * r.blocks(p);
    if (threadIdx.x == 0) {
      Cut cut{};
      if (tile > 0) cut = Cut{r.row0, min(r.rows * p.group - rb * kTileRows, kTileRows), rb * kTileRows, h, at - tile, tiles};
      p.cuts[blockIdx.x] = cut;
    }
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

// ------------------------------------------------------------------ copies and matrix steps

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int row, int head, int page) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
               :: "r"(dst), "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Types of the two matrix products: the query's own, f16 over an E4M3 cache (exact for its values).
template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
  static constexpr uint32_t kExponent = 0x7F807F80u;
  static constexpr float kShift = 0.f;
  static __device__ __forceinline__ void step(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <> struct Mma<__half> {
  static constexpr uint32_t kExponent = 0x7C007C00u;
  // f16 probabilities are kept times 2^15, so that those below 2^-14 of the largest do not lose bits
  static constexpr float kShift = 15.f;
  static __device__ __forceinline__ void step(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// ------------------------------------------------------------------ the kernel

template <typename T, bool kE4M3, int D>
struct Shape {
  using C = typename std::conditional<kE4M3, __half, T>::type;     // type of the products
  static constexpr int kBytes = kE4M3 ? 1 : 2;
  static constexpr int kRowBytes = D * kBytes < 128 ? D * kBytes : 128;   // one key's row in shared memory
  static constexpr int kHalves = D * kBytes / kRowBytes;                  // rows of a key (128-byte boxes)
  static constexpr int kTileBytes = kTileKeys * D * kBytes;
  static constexpr int kStages = kTileBytes == 32768 ? 3 : (kTileBytes == 16384 ? 5 : 8);
  static constexpr int kMergeBytes = 4 * 16 * D * 4;                      // four warps' outputs
  static constexpr int kSmem = 1024 + kStages * 2 * kTileBytes + kMergeBytes + 4 * 16 * 8 + 256;
  // Address of the 16-byte piece `piece` of a key's row in its tile, as the TMA swizzle places it.
  static __device__ __forceinline__ uint32_t piece(uint32_t tile, int key, int piece_) {
    if constexpr (kRowBytes == 128)
      return tile + (piece_ >> 3) * (kTileKeys * 128) + key * 128 + (((piece_ & 7) ^ (key & 7)) << 4);
    else
      return tile + key * 64 + ((piece_ ^ ((key >> 1) & 3)) << 4);
  }
};

// One warp's state over an item: 16 rows, of which a lane (g, q) holds rows g and g + 8.
template <int D>
struct Rows {
  uint32_t q[D / 16][4];
  float o[D / 8][4];
  float mc[2], l[2], c[2];         // c m, sum, c of the two rows
  uint64_t bits[2];                // nodes they see
};

__device__ __forceinline__ bool sees(const uint64_t bits, int key, int ctx) {
  return key < ctx || (key - ctx < 64 && (bits >> (key - ctx) & 1));
}

// kKeys keys of a tile, from key0 on: scores, softmax step, weighted values. kTail: the tile holds keys that
// not every row sees; values of keys a row does not see must not reach it, whatever they hold, so
// non-finite values enter the product as zeros and are added afterwards where they are seen.
template <typename T, bool kE4M3, int D, int kKeys, bool kTail>
__device__ __forceinline__ void attend(Rows<D>& w, uint32_t kt, uint32_t vt, int key0, int tile_key, const Request& r,
                                       uint32_t bad_pages, int page_shift, int lane) {
  using S = Shape<T, kE4M3, D>;
  using M = Mma<typename S::C>;
  constexpr int kSteps = D / 16;
  const int q = lane & 3, mat = lane >> 3, in8 = lane & 7;
  float s[kKeys / 8][4];
#pragma unroll
  for (int j = 0; j < kKeys / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
  for (int j = 0; j < kKeys / 16; ++j) {
    const int key = key0 + 16 * j + (mat >> 1) * 8 + in8;
    if constexpr (!kE4M3) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        uint32_t f[4];
        ldsm4(f, S::piece(kt, key, 2 * t + (mat & 1)));
        M::step(s[2 * j], w.q[t], f[0], f[1]);
        M::step(s[2 * j + 1], w.q[t], f[2], f[3]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < kSteps; t += 2) {
        uint32_t f[4];
        ldsm4(f, S::piece(kt, key, t + (mat & 1)));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          M::step(s[2 * j + (i >> 1)], w.q[t + (i & 1)], e4m3x2_to_f16x2(f[i] & 0xffffu), e4m3x2_to_f16x2(f[i] >> 16));
      }
    }
  }
  if constexpr (kTail) {
#pragma unroll
    for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int in_tile = key0 + 8 * j + 2 * q + (e & 1);
        const bool on_page = !(bad_pages >> (in_tile >> page_shift) & 1);
        if (!on_page || !sees(w.bits[e >> 1], tile_key + in_tile, r.ctx)) s[j][e] = -INFINITY;
      }
  }
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[j][e]);
  float base[2], keep[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
    top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    const float mc = top[i] == -INFINITY ? -INFINITY : fmaf(top[i], w.c[i], -M::kShift);
    const float now = fmaxf(w.mc[i], mc);
    base[i] = now == -INFINITY ? 0.f : now;
    keep[i] = exp2_fast(w.mc[i] - base[i]);
    w.mc[i] = now;
    w.l[i] *= keep[i];
  }
#pragma unroll
  for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[j][e] = exp2_fast(fmaf(s[j][e], w.c[e >> 1], -base[e >> 1]));
      w.l[e >> 1] += s[j][e];
    }
  if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) w.o[j][e] *= keep[e >> 1];
  }
  uint32_t odd = 0;
#pragma unroll
  for (int j = 0; j < kKeys / 16; ++j) {
    const uint32_t a[4] = {M::pack(s[2 * j][0], s[2 * j][1]), M::pack(s[2 * j][2], s[2 * j][3]),
                           M::pack(s[2 * j + 1][0], s[2 * j + 1][1]), M::pack(s[2 * j + 1][2], s[2 * j + 1][3])};
    const int key = key0 + 16 * j + (mat & 1) * 8 + in8;
    // the lane's values in a step: keys key0 + 16 j + {0, 8} + 2 q + {0, 1}
    auto clean = [&](uint32_t v, int half) {
      if constexpr (kTail) {
        const uint32_t non = __vcmpeq2(v & M::kExponent, M::kExponent);
        const int k = tile_key + key0 + 16 * j + 8 * half + 2 * q;
        odd |= non & ((k < r.keys ? 0xffffu : 0u) | (k + 1 < r.keys ? 0xffff0000u : 0u));
        return v & ~non;
      } else {
        return v;
      }
    };
    if constexpr (!kE4M3) {
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        uint32_t f[4];
        ldsm4_t(f, S::piece(vt, key, n + (mat >> 1)));
        M::step(w.o[n], a, clean(f[0], 0), clean(f[1], 1));
        M::step(w.o[n + 1], a, clean(f[2], 0), clean(f[3], 1));
      }
    } else {
#pragma unroll
      for (int n = 0; n < D / 16; n += 2) {
        uint32_t f[4];
        ldsm4_t(f, S::piece(vt, key, n + (mat >> 1)));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a0 = e4m3x2_to_f16x2(f[2 * i] & 0xffffu), a1 = e4m3x2_to_f16x2(f[2 * i] >> 16);
          const uint32_t b0 = e4m3x2_to_f16x2(f[2 * i + 1] & 0xffffu), b1 = e4m3x2_to_f16x2(f[2 * i + 1] >> 16);
          M::step(w.o[2 * (n + i)], a, clean(__byte_perm(a0, a1, 0x5410), 0), clean(__byte_perm(b0, b1, 0x5410), 1));
          M::step(w.o[2 * (n + i) + 1], a, clean(__byte_perm(a0, a1, 0x7632), 0), clean(__byte_perm(b0, b1, 0x7632), 1));
        }
      }
    }
  }
  if constexpr (kTail) {
    if (__any_sync(0xffffffffu, odd != 0)) {
      // rare: some visible value is NaN or infinite; add such values key by key
#pragma unroll 1
      for (int k = 0; k < kKeys; ++k) {
        const int in_tile = key0 + k, from = (lane & ~3) | (k >> 1 & 3);
        float mine0 = 0.f, mine1 = 0.f;
#pragma unroll
        for (int j = 0; j < kKeys / 8; ++j)
          if (k >> 3 == j) {
            mine0 = k & 1 ? s[j][1] : s[j][0];
            mine1 = k & 1 ? s[j][3] : s[j][2];
          }
        const float p0 = __shfl_sync(0xffffffffu, mine0, from), p1 = __shfl_sync(0xffffffffu, mine1, from);
        if (tile_key + in_tile >= r.keys || (bad_pages >> (in_tile >> page_shift) & 1)) continue;
        const bool see0 = sees(w.bits[0], tile_key + in_tile, r.ctx), see1 = sees(w.bits[1], tile_key + in_tile, r.ctx);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the lane's output columns: 8 n + 2 q + e, or interleaved by fours over an E4M3 cache
            const int d = kE4M3 ? 16 * (n >> 1) + 4 * q + 2 * e + (n & 1) : 8 * n + 2 * q + e;
            const uint32_t at = S::piece(vt, in_tile, d * S::kBytes / 16) + (d * S::kBytes & 15);
            float v;
            if constexpr (kE4M3) {
              uint32_t raw;
              asm volatile("ld.shared.u8 %0, [%1];" : "=r"(raw) : "r"(at));
              v = __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(raw)));
            } else {
              unsigned short raw;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(raw) : "r"(at));
              T t;
              memcpy(&t, &raw, 2);
              v = Elem<T>::to_float(t);
            }
            if (!isfinite(v)) {
              if (see0) w.o[n][e] += p0 * v;
              if (see1) w.o[n][2 + e] += p1 * v;
            }
          }
      }
    }
  }
}

template <typename T, bool kE4M3, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
tree_attention_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<T, kE4M3, D>;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* base = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  const uint32_t stages = smem_u32(base);
  float* merge_o = reinterpret_cast<float*>(base + S::kStages * 2 * S::kTileBytes);
  float2* merge_ml = reinterpret_cast<float2*>(merge_o + 4 * 16 * D);
  uint8_t* tail = reinterpret_cast<uint8_t*>(merge_ml + 4 * 16);
  const uint32_t full = smem_u32(tail), empty = full + 8 * S::kStages;
  uint32_t* bad_pages = reinterpret_cast<uint32_t*>(tail + 16 * S::kStages);
  volatile int* dead = reinterpret_cast<volatile int*>(bad_pages + S::kStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, kConsumers);
    }
    *dead = 0;
    mbar_init_fence();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Walk walk;
  walk.begin(p, lane);
  __syncthreads();
  if (walk.left == 0) return;

  // Warp 0 requests the tiles, kStages ahead at first, then one for each that every warp has left: it
  // asks for the stage of the tile before the one it has just done itself, so it seldom waits. Lane i
  // serves a tile's i-th page; the page's number is loaded one tile ahead.
  Walk ask = walk;
  int asked = 0, ask_stage = 0;
  uint32_t ask_phase = 0;
  const int box_rows = min(1 << p.page_shift, kTileKeys), pages = kTileKeys / box_rows;
  int page = -1;
  bool wanted = false;
  auto look = [&]() {
    const int key = ask.tile * kTileKeys + lane * box_rows;
    wanted = ask.left > 0 && lane < pages && key < ask.r.keys;
    if (wanted) page = p.block_table[(size_t)ask.b * p.max_pages + (key >> p.page_shift)];
  };
  auto request = [&]() {
    if (ask.left == 0) return;
    if (asked >= S::kStages) mbar_wait(empty + 8 * ask_stage, ask_phase ^ 1, p.spin_budget, p.status, dead);
    if (__any_sync(0xffffffffu, *dead)) return;
    const bool ok = wanted && page >= 0 && page < p.num_pages;
    const unsigned good = __ballot_sync(0xffffffffu, ok), bad = __ballot_sync(0xffffffffu, wanted && !ok);
    const uint32_t bar = full + 8 * ask_stage, kt = stages + ask_stage * 2 * S::kTileBytes, vt = kt + S::kTileBytes;
    const uint32_t page_bytes = (uint32_t)box_rows * D * S::kBytes;
    if (lane == 0) {
      bad_pages[ask_stage] = bad;
      if (bad) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
      mbar_arrive_tx(bar, 2 * page_bytes * __popc(good));
    }
    __syncwarp();
    if (ok) {
      const int row = (ask.tile * kTileKeys + lane * box_rows) & ((1 << p.page_shift) - 1);
#pragma unroll
      for (int i = 0; i < S::kHalves; ++i) {
        const uint32_t off = i * (kTileKeys * S::kRowBytes) + lane * box_rows * S::kRowBytes;
        tma_load(kt + off, &kmap, bar, i * (S::kRowBytes / S::kBytes), row, ask.h, page);
      }
#pragma unroll
      for (int i = 0; i < S::kHalves; ++i) {
        const uint32_t off = i * (kTileKeys * S::kRowBytes) + lane * box_rows * S::kRowBytes;
        tma_load(vt + off, &vmap, bar, i * (S::kRowBytes / S::kBytes), row, ask.h, page);
      }
    }
    ++asked;
    if (++ask_stage == S::kStages) { ask_stage = 0; ask_phase ^= 1; }
    if (--ask.left > 0 && ++ask.tile == ask.tiles) ask.next_item(p, lane);
    look();
  };
  if (warp == 0) {
    look();
    for (int i = 0; i < S::kStages; ++i) request();
  }

  int stage = 0;
  uint32_t phase = 0;
  bool behind = false;             // whether a tile has been done
  const int g = lane >> 2, q = lane & 3;
  while (walk.left > 0) {
    // one item: rows [first, first + rows) of the request, tiles [tile, tile + count)
    const Request r = walk.r;
    const int first = walk.rb * kTileRows, rows = min(r.rows * p.group - first, kTileRows);
    const int row_warps = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4), slices = kConsumers / row_warps;
    const int wr = warp % row_warps, slice = warp / row_warps, h = walk.h;
    const int tile0 = walk.tile, count = min(walk.tiles - tile0, walk.left);
    const bool whole = count == walk.tiles;

    Rows<D> w;
    const bool live = wr * 16 < rows;
    const float c = p.scale * kLog2e * (kE4M3 ? p.k_scale[h] : 1.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = wr * 16 + g + 8 * i, flat = first + row;
      const bool in = row < rows;
      const int node = in ? flat / p.group : 0, head = h * p.group + (in ? flat - node * p.group : 0);
      const T* src = static_cast<const T*>(p.q) + (int64_t)(r.row0 + node) * p.ldq + (int64_t)head * D;
      w.bits[i] = 0;
      if (in) {
        w.bits[i] = p.tree_mask ? p.tree_mask[r.row0 + node] : ~0ull >> (63 - node);
        if (r.rows < 64) w.bits[i] &= (1ull << r.rows) - 1;
      }
      w.c[i] = c;
      w.mc[i] = -INFINITY;
      w.l[i] = 0.f;
      if constexpr (!kE4M3) {
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            w.q[t][i + 2 * e] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * t + 8 * e + 2 * q) : 0u;
      } else {
        // E4M3 keys give a lane four consecutive elements; the order of a product's k is free
        uint2 v[D / 16];
        float top = 0.f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          v[t] = in ? *reinterpret_cast<const uint2*>(src + 16 * t + 4 * q) : make_uint2(0u, 0u);
          T x[4];
          memcpy(x, &v[t], 8);
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(Elem<T>::to_float(x[e])));
        }
        float f = 1.f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          // bf16 rows enter f16 times a power of two that puts their largest element in [1, 4)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int ex = top > 0.f && isfinite(top) ? min((int)(__float_as_uint(top) >> 23) - 127, 126) : 0;
          f = __uint_as_float((uint32_t)(127 - ex) << 23);
          w.c[i] = c * (ex >= -126 ? __uint_as_float((uint32_t)(127 + ex) << 23) : 5.877471754111438e-39f);
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          T x[4];
          memcpy(x, &v[t], 8);
          for (int e = 0; e < 2; ++e)
            w.q[t][i + 2 * e] = Mma<__half>::pack(Elem<T>::to_float(x[2 * e]) * f, Elem<T>::to_float(x[2 * e + 1]) * f);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n) w.o[n][0] = w.o[n][1] = w.o[n][2] = w.o[n][3] = 0.f;

    for (int i = 0; i < count; ++i) {
      mbar_wait(full + 8 * stage, phase, p.spin_budget, p.status, dead);
      __syncwarp();
      if (live) {
        const uint32_t kt = stages + stage * 2 * S::kTileBytes, vt = kt + S::kTileBytes, bad = bad_pages[stage];
        const int tile_key = (tile0 + i) * kTileKeys;
        const bool all = tile_key + kTileKeys <= r.ctx && bad == 0;
        const int keys = 16 * row_warps, key0 = slice * keys;
        if (!all)
          for (int k = 0; k < keys; k += 16) attend<T, kE4M3, D, 16, true>(w, kt, vt, key0 + k, tile_key, r, bad, p.page_shift, lane);
        else if (row_warps == 1)
          attend<T, kE4M3, D, 16, false>(w, kt, vt, key0, tile_key, r, bad, p.page_shift, lane);
        else
          for (int k = 0; k < keys; k += 32) attend<T, kE4M3, D, 32, false>(w, kt, vt, key0 + k, tile_key, r, bad, p.page_shift, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * stage);
      if (++stage == S::kStages) { stage = 0; phase ^= 1; }
      if (warp == 0) {
        if (behind) request();
        behind = true;
      }
    }

    // join the slices of each row tile: halves, in a fixed order
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], 1);
      w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], 2);
    }
    for (int off = slices / 2; off > 0; off >>= 1) {
      if (slice >= off && slice < 2 * off) {
        const int at = (slice - off) * row_warps + wr;
        float* o = merge_o + at * 16 * D + lane;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[32 * (4 * n + e)] = w.o[n][e];
        if (q == 0) {
          merge_ml[at * 16 + g] = make_float2(w.mc[0], w.l[0]);
          merge_ml[at * 16 + g + 8] = make_float2(w.mc[1], w.l[1]);
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (slice < off) {
        const int at = slice * row_warps + wr;
        const float* o = merge_o + at * 16 * D + lane;
        float mine[2], other[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 ml = merge_ml[at * 16 + g + 8 * i];
          const float top = fmaxf(w.mc[i], ml.x), safe = top == -INFINITY ? 0.f : top;
          mine[i] = exp2_fast(w.mc[i] - safe);
          other[i] = exp2_fast(ml.x - safe);
          w.mc[i] = top;
          w.l[i] = w.l[i] * mine[i] + ml.y * other[i];
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) w.o[n][e] = w.o[n][e] * mine[e >> 1] + o[32 * (4 * n + e)] * other[e >> 1];
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (slice == 0 && live && !*dead) {
      const int slot = 2 * blockIdx.x + (tile0 > 0 ? 0 : 1);
      const float vs = kE4M3 ? p.v_scale[h] : 1.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = wr * 16 + g + 8 * i, flat = first + row;
        if (row >= rows) continue;
        if (whole) {
          const int node = flat / p.group, head = h * p.group + flat - node * p.group;
          T* dst = static_cast<T*>(p.out) + (int64_t)(r.row0 + node) * p.ldo + (int64_t)head * D;
          const float f = w.l[i] == 0.f ? 0.f : vs / w.l[i];
          if constexpr (!kE4M3) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<uint32_t*>(dst + 8 * n + 2 * q) =
                  Mma<T>::pack(w.l[i] == 0.f ? 0.f : w.o[n][2 * i] * f, w.l[i] == 0.f ? 0.f : w.o[n][2 * i + 1] * f);
          } else {
#pragma unroll
            for (int n = 0; n < D / 8; n += 2)
              *reinterpret_cast<uint2*>(dst + 8 * n + 4 * q) =
                  w.l[i] == 0.f ? make_uint2(0u, 0u)
                                : make_uint2(Mma<T>::pack(w.o[n][2 * i] * f, w.o[n + 1][2 * i] * f),
                                             Mma<T>::pack(w.o[n][2 * i + 1] * f, w.o[n + 1][2 * i + 1] * f));
          }
          if (p.lse && q == 0)
            p.lse[(int64_t)(r.row0 + node) * p.Hq + head] = w.l[i] == 0.f ? -INFINITY : (w.mc[i] + log2f(w.l[i])) * kLn2;
        } else {
          float* o = p.part_o + ((size_t)slot * kTileRows + row) * D;
          if constexpr (!kE4M3) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<float2*>(o + 8 * n + 2 * q) = make_float2(w.o[n][2 * i], w.o[n][2 * i + 1]);
          } else {
#pragma unroll
            for (int n = 0; n < D / 8; n += 2)
              *reinterpret_cast<float4*>(o + 8 * n + 4 * q) =
                  make_float4(w.o[n][2 * i], w.o[n + 1][2 * i], w.o[n][2 * i + 1], w.o[n + 1][2 * i + 1]);
          }
          if (q == 0) p.part_ml[(size_t)slot * kTileRows + row] = make_float2(w.mc[i], w.l[i]);
        }
      }
    }
    walk.left -= count;
    if (walk.left > 0) walk.next_item(p, lane);
  }
  if (warp == 0 && __any_sync(0xffffffffu, *dead))
    for (int i = 0; i < S::kStages && i < asked; ++i) mbar_drain(full + 8 * i, ((asked - i + S::kStages - 1) / S::kStages - 1) & 1);
}

// Joins the partial items: block x belongs to the boundary before share x + 1, and works if it is the first one
// inside its item. One warp per row, a lane D / 32 columns, the shares' sums in order.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(const AttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPer = D / 32;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int total = p.total[0], blocks = p.total[1];
  if ((int)blockIdx.x + 1 >= blocks) return;
  const Cut cut = p.cuts[blockIdx.x + 1];
  if (row >= cut.rows) return;
  const Shares shares(total, blocks);
  if (shares.start(blockIdx.x) > cut.start) return;             // an earlier boundary is inside too
  const int c0 = blockIdx.x, parts = shares.owner(cut.start + cut.tiles - 1) - c0 + 1;
  // the item's first part is the last of its block's share, the others are the first of theirs
  auto slot = [&](int i) { return (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * kTileRows + row; };
  float mc = -INFINITY;
  for (int i = lane; i < parts; i += 32) mc = fmaxf(mc, p.part_ml[slot(i)].x);
  mc = warp_max(mc);
  const float base = mc == -INFINITY ? 0.f : mc;
  float o[kPer], l = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float f = 0.f;
    if (i0 + lane < parts) {
      const float2 ml = p.part_ml[slot(i0 + lane)];
      f = exp2_fast(ml.x - base);
      l = fmaf(ml.y, f, l);
    }
    const int n = min(parts - i0, 32);
    for (int i = 0; i < n; i += 8) {
      float v[8][kPer];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* src = p.part_o + slot(i0 + min(i + u, n - 1)) * D + lane * kPer;
        if constexpr (kPer == 4) *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(src);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float g = __shfl_sync(0xffffffffu, f, min(i + u, 31));
        if (i + u < n)
#pragma unroll
          for (int j = 0; j < kPer; ++j) o[j] = fmaf(v[u][j], g, o[j]);
      }
    }
  }
  l = warp_sum(l);
  const int flat = cut.first + row, node = flat / p.group, head = cut.h * p.group + flat - node * p.group;
  const float f = l == 0.f ? 0.f : (p.v_scale ? p.v_scale[cut.h] : 1.f) / l;
  T* dst = static_cast<T*>(p.out) + (int64_t)(cut.row0 + node) * p.ldo + (int64_t)head * D + lane * kPer;
  uint32_t packed[kPer / 2];
#pragma unroll
  for (int j = 0; j < kPer; j += 2) packed[j / 2] = l == 0.f ? 0u : Mma<T>::pack(o[j] * f, o[j + 1] * f);
  if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
  else *reinterpret_cast<uint32_t*>(dst) = packed[0];
  if (p.lse && lane == 0) p.lse[(int64_t)(cut.row0 + node) * p.Hq + head] = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
}

// ------------------------------------------------------------------ host

// The cache as [pages][heads][page size][head dim]; a box is up to 128 rows of one page and head, 128 bytes (or
// a whole 64-byte row) wide.
bool encode_cache(CUtensorMap* map, const mdw_kv_cache* c, void* data) {
  const bool fp8 = c->dtype == MDW_DT_E4M3;
  const cuuint64_t e = fp8 ? 1 : 2, d = c->head_dim, ps = c->page_size;
  const cuuint64_t dims[4] = {d, ps, (cuuint64_t)c->kv_heads, (cuuint64_t)c->num_pages};
  const cuuint64_t strides[3] = {d * e, d * ps * e, (cuuint64_t)c->page_stride * e};
  const cuuint32_t width = (cuuint32_t)(d * e < 128 ? d : 128 / e);
  const cuuint32_t box[4] = {width, (cuuint32_t)(ps < kTileKeys ? ps : kTileKeys), 1, 1}, ones[4] = {1, 1, 1, 1};
  const EncodeTiledFn fn = encode_tiled();
  return fn && fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, data, dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, width * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttnWs {
  size_t cuts, ml, o, total;
};
AttnWs attn_ws(int grid, int D) {
  AttnWs w;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  w.cuts = 256;
  w.ml = w.cuts + up((size_t)grid * sizeof(Cut));
  w.o = w.ml + up((size_t)grid * 2 * kTileRows * 8);
  w.total = w.o + up((size_t)grid * 2 * kTileRows * D * 4);
  return w;
}

template <typename T, bool kE4M3, int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  using S = Shape<T, kE4M3, D>;
  cudaError_t e = allow_shared_memory<tree_attention_kernel<T, kE4M3, D>>(dev);
  if (e != cudaSuccess) return e;
  tree_attention_kernel<T, kE4M3, D><<<grid, kAttnThreads, S::kSmem, s>>>(p, km, vm);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (grid == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(grid - 1), (unsigned)((std::min(p.max_new * p.group, kTileRows) + 3) / 4));
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
  if (max_pages < 1 || (int64_t)max_pages * cache->page_size > 0x7fffffffLL) return MDW_ERR_UNSUPPORTED_SHAPE;
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
  const AttnParams p{cache->k_scale, cache->v_scale, q, out, lse, ldq, ldo, block_table, ctx_len, row_start, tree_mask, status,
                     mdw_spin_budget(), scale, B, T, q_heads, cache->kv_heads, q_heads / cache->kv_heads, max_new, max_pages,
                     cache->num_pages, log2_of(cache->page_size), reinterpret_cast<int32_t*>(base),
                     reinterpret_cast<Cut*>(base + lay.cuts), reinterpret_cast<float2*>(base + lay.ml),
                     reinterpret_cast<float*>(base + lay.o)};
  CUtensorMap km, vm;
  if (!encode_cache(&km, cache, cache->k) || !encode_cache(&vm, cache, cache->v)) return MDW_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int D = cache->head_dim;
  cudaError_t e;
  if (q_dtype == MDW_DT_BF16)
    e = fp8 ? launch<__nv_bfloat16, true>(p, D, km, vm, grid, dev, s) : launch<__nv_bfloat16, false>(p, D, km, vm, grid, dev, s);
  else
    e = fp8 ? launch<__half, true>(p, D, km, vm, grid, dev, s) : launch<__half, false>(p, D, km, vm, grid, dev, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
