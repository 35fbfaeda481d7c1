// mdw_tree_attention for up to 32 rows a request and kv head: single tokens and short windows.
//
// Mathematics as in tree_attention.cu. With so few rows the tensor-memory form wastes its products (128 lanes a
// tile, whatever the rows: 2,700 cycles for a tile's two products against the 1,400 that its E4M3 keys and
// values take to arrive), and E4M3 tiles would be converted in shared memory. Here a warp does
// everything for 16 rows and its keys: it forms scores and outputs with m16n8k16 (16 rows x 8 keys x
// 16 elements), converts E4M3 codes in registers on the way into the products, and keeps maximum, sum and output
// of its own. Up to 16 rows every warp has a ring of copies to itself, up to 32 two warps share one, 16 rows each.
// The rings take the item's stages (4 KB of keys and of values, 192 KB in flight per SM) in turn, each
// at its own pace, and the warps join once per item: there is no barrier of the block in the loop. A
// warp of its own makes the copies (made by the warps of the products, between two stages, they cost 4 to 9 % over
// E4M3 caches). All lanes' page ids are loaded one stage early and looked at when they are used.
//
// Measured: one token over 131k E4M3 keys of 8 kv heads 51 us (5.2 TB/s; the stream alone 38, then begin 4, end 2
// and join 3), 16-bit keys 90 us (5.9 TB/s), the 20 rows of a 4-token window over 1,500 keys 11.5 us, of which
// launch, first copies, end and join are all but 2. What bounds it is the keys' stream; over E4M3 with more than
// 16 rows the conversion, which every 16 rows repeat (5.2 -> 3.2 TB/s).
//
// Order of elements and keys. A contraction may take its index in any order if both operands do: lane (g, q) of a
// product (g = 0..7, q = 0..3) has keys q and q + 4 of eight as its two columns, and 16 bytes in a row of a key as
// its elements, so that every load of keys or values is 16 bytes wide and without bank conflicts in the
// swizzled tiles (of 128-byte rows).
#include <type_traits>

#include "mdw_internal.h"
#include "tree_attention.cuh"

namespace mdw {
namespace {

// Warps of the products; a third warpgroup, of which one warp works, makes the copies. The groups share the registers
// that the launch gives each thread (168) as 40 + 2 x 232.
constexpr int kWarps = 8, kThreads = 32 * kWarps + 128;

// kBlocks warps share the copies of a ring and have 16 rows each.
template <typename T, bool kE4M3, int D, int kBlocks>
struct Few {
  using C = typename std::conditional<kE4M3, __half, T>::type;     // type of the products
  static constexpr int kBytes = kE4M3 ? 1 : 2;
  static constexpr int kKeys = kFewBytes / (D * kBytes);           // keys of a stage
  static constexpr int kRowBytes = D * kBytes < 128 ? D * kBytes : 128, kHalves = D * kBytes / kRowBytes;
  static constexpr int kStageBytes = 2 * kFewBytes;                // keys, then values
  static constexpr int kRings = kWarps / kBlocks, kStages = 3 * kBlocks, kRows = 16 * kBlocks;
  static constexpr int kPitch = D + 4;                             // floats of a joined row
  static constexpr int kJoinAt = kRings * kStages * kStageBytes, kSmall = kJoinAt + kWarps / 2 * 16 * kPitch * 4;
  static constexpr int kBarsAt = kSmall + kWarps * 16 * 8, kBadAt = kBarsAt + 2 * kRings * kStages * 8;
  static constexpr int kSmem = kBadAt + kRings * kStages * 4 + 16;

  static __device__ __forceinline__ uint32_t piece(uint32_t tile, int key, int i) {   // 16 bytes of a key's row
    if constexpr (kRowBytes == 128) return tile + (i >> 3) * (kKeys * 128) + key * 128 + (((i & 7) ^ (key & 7)) << 4);
    else return tile + key * 64 + ((i ^ ((key >> 1) & 3)) << 4);
  }
  // Element that output column g of tile t holds; the lanes of a pair of columns are far apart for the loads' sake.
  static __device__ __forceinline__ int element(int t, int g) {
    if constexpr (kE4M3) return (D / 8) * ((g & 1) << 2 | g >> 1) + t;
    else return 8 * t + g;
  }
};

template <typename C>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<C, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void load_transposed(uint32_t (&v)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Stages of the walk's current item that lie in the block's share.
template <int kKeys>
__device__ __forceinline__ int stages(const Walk& w) {
  const int keys = min(w.r.keys, (w.tile + w.count()) * kTileKeys) - w.tile * kTileKeys;
  return (keys + kKeys - 1) / kKeys;
}

template <typename T, bool kE4M3, int D, int kBlocks>
__global__ void __launch_bounds__(kThreads, 1)
few_rows_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = Few<T, kE4M3, D, kBlocks>;
  using C = typename S::C;
  using M = Mma<C>;
  constexpr int kOctets = S::kKeys / 8, kOut = D / 8, kSteps = D / 16, kStages = S::kStages, kRings = S::kRings;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  float2* ml = reinterpret_cast<float2*>(smem + S::kSmall);     // [warp][16] (c m, sum)
  // barriers of ring x, slot i at 8 (kStages x + i); pages of its stage outside the cache
  const uint32_t full = base + S::kBarsAt, empty = full + kRings * kStages * 8;
  volatile uint32_t* bads = reinterpret_cast<volatile uint32_t*>(smem + S::kBadAt);
  volatile int* dead = reinterpret_cast<volatile int*>(smem + S::kBadAt + kRings * kStages * 4);
  if (base & 1023) {                                            // the swizzled tiles need the alignment asked for above
    if (threadIdx.x == 0) raise_status(p.status, MDW_ERR_UNSUPPORTED_SHAPE);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.total[0] = p.total[1] = 0;
    return;
  }
  if (threadIdx.x == 0) {
    *dead = 0;
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  if (threadIdx.x < kRings * kStages) {
    mbar_init(full + 8 * threadIdx.x, 1);
    mbar_init(empty + 8 * threadIdx.x, kBlocks);
    mbar_init_fence();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Walk walk;
  walk.begin(p, lane);
  if (!walk.more()) return;                                     // the whole block
  __syncthreads();                                              // barriers, *dead

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp > kWarps) return;
    // ---- copies. Stages go to the rings in turn, across items; a lane has one page of one ring's next stage. Within an
    // item the rings advance on their own, each as its slots become free.
    const int box_rows = min(1 << p.page_shift, S::kKeys), pages = S::kKeys / box_rows;
    const uint32_t page_bytes = (uint32_t)box_rows * D * S::kBytes, of_stage = (1u << pages) - 1u;
    const int x = lane / pages, sub = lane - x * pages, low = x * pages;   // ring, page of the stage, ring's first lane
    int before = 0, asked = 0;                                  // stages before the item; copies of this lane's ring
    while (walk.more() && !__any_sync(0xffffffffu, *dead)) {
      const Request r = walk.r;
      const int n = stages<S::kKeys>(walk), first = walk.tile * kTileKeys + sub * box_rows, h = walk.h;
      const int32_t* table = p.block_table + (size_t)walk.b * p.max_pages;
      int i = x < kRings ? (x - before) & (kRings - 1) : n;     // the ring's next stage of the item
      auto wanted = [&](int i) { return i < n && first + i * S::kKeys < r.keys; };
      // the lane's page of it, not looked at before its copy: the load is on its way meanwhile
      auto look = [&](int i) { return wanted(i) ? table[(first + i * S::kKeys) >> p.page_shift] : 0; };
      int id = look(i), next_id = look(i + kRings);
      long long t0 = clock64();
      while (__any_sync(0xffffffffu, i < n)) {
        if (__any_sync(0xffffffffu, *dead)) break;
        const int slot = x * kStages + asked % kStages;
        const unsigned free = __ballot_sync(0xffffffffu, i < n && mbar_test(empty + 8 * slot, (asked / kStages & 1) ^ 1));
        const bool go = i < n && (free >> low & of_stage) == of_stage;
        const bool want = go && wanted(i), there = want && id >= 0 && id < p.num_pages;
        const unsigned good = __ballot_sync(0xffffffffu, there), bad = __ballot_sync(0xffffffffu, want && !there);
        if (!__any_sync(0xffffffffu, go)) {
          if (clock64() - t0 > p.spin_budget) {
            *dead = 1;
            raise_status(p.status, MDW_ERR_TIMEOUT);
          }
          __nanosleep(40);
          continue;
        }
        const uint32_t bar = full + 8 * slot, to = base + slot * S::kStageBytes + sub * box_rows * S::kRowBytes;
        if (go && sub == 0) {
          bads[slot] = bad >> low & of_stage;
          if (bad >> low & of_stage) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
          mbar_arrive_tx(bar, 2 * page_bytes * __popc(good >> low & of_stage));
        }
        __syncwarp();
        if (go) {
          if (there) {
            const int row = (first + i * S::kKeys) & ((1 << p.page_shift) - 1);
#pragma unroll
            for (int k = 0; k < S::kHalves; ++k) {
              tma_load(to + k * (S::kKeys * S::kRowBytes), &kmap, bar, k * (S::kRowBytes / S::kBytes), row, h, id);
              tma_load(to + k * (S::kKeys * S::kRowBytes) + kFewBytes, &vmap, bar, k * (S::kRowBytes / S::kBytes), row, h, id);
            }
          }
          ++asked;
          i += kRings;
          id = next_id;
          next_id = look(i + kRings);
        }
        __syncwarp();
        t0 = clock64();
      }
      before += n;
      walk.done(p, lane);
    }
    // Every copy arrives before the block ends, also where a wait runs out after the last one was requested: the block is not
    // over before this warp has waited for each ring's last ones.
    if (x < kRings && sub == 0)
      for (int i = max(asked - kStages, 0); i < asked; ++i) mbar_drain_inline(full + 8 * (x * kStages + i % kStages), i / kStages & 1);
    return;
  }

  auto join_barrier = [] { asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory"); };
  asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
  const int mine = warp / kBlocks, row0 = warp % kBlocks * 16;  // the warp's ring; first of its rows
  const uint32_t ring = base + mine * kStages * S::kStageBytes, full0 = full + 8 * mine * kStages, empty0 = empty + 8 * mine * kStages;
  int slot = 0, before = 0;
  uint32_t phase = 0;
  while (walk.more()) {
    const Request r = walk.r;
    const int rows = r.rows * p.group, tile0 = walk.tile, count = walk.count(), h = walk.h;
    const bool whole = count == walk.tiles;
    const bool active = kBlocks == 1 || row0 < rows;
    // ---- rows g and g + 8 of the warp, four elements of each per step; the nodes they see; c
    uint32_t qf[kSteps][4];
    uint64_t bits[2];
    float c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row0 + g + 8 * i, node = row / p.group;
      const bool valid = row < rows;
      bits[i] = 0;
      if (valid) {
        bits[i] = (p.tree_mask ? p.tree_mask[r.row0 + node] : ~0ull >> (63 - node)) & ((1ull << r.rows) - 1);
      }
      c[i] = p.scale * kLog2e * (kE4M3 ? p.k_scale[h] : 1.f);
      const T* src = static_cast<const T*>(p.q) + (valid ? (int64_t)(r.row0 + node) * p.ldq + (int64_t)(h * p.group + row - node * p.group) * D : 0);
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int d = kE4M3 ? 16 * (q + 4 * (st >> 2)) + 4 * (st & 3) : 64 * (st >> 2) + 8 * (q + 4 * (st >> 1 & 1)) + 4 * (st & 1);
        const uint2 v = valid ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0u, 0u);
        qf[st][i] = v.x;
        qf[st][2 + i] = v.y;
      }
      if constexpr (kE4M3 && std::is_same<T, __nv_bfloat16>::value) {
        // bf16 rows enter f16, the type of the converted keys, times a power of two that puts their largest element in [1, 4):
        // elements below 2^-17 of it are off by up to 2^-25 of it, far below the fp32 sums' own error
        auto low = [](uint32_t v) { return __uint_as_float(v << 16); };
        auto high = [](uint32_t v) { return __uint_as_float(v & 0xffff0000u); };
        float top = 0.f;
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int j = i; j < 4; j += 2) top = fmaxf(top, fmaxf(fabsf(low(qf[st][j])), fabsf(high(qf[st][j]))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = top > 0.f && isfinite(top) ? min((int)(__float_as_uint(top) >> 23) - 127, 126) : 0;
        const float f = __uint_as_float((uint32_t)(127 - ex) << 23);
        c[i] *= ex >= -126 ? __uint_as_float((uint32_t)(127 + ex) << 23) : 5.877471754111438e-39f;
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
#pragma unroll
          for (int j = i; j < 4; j += 2) qf[st][j] = M::pack(low(qf[st][j]) * f, high(qf[st][j]) * f);
      }
      if constexpr (kE4M3) c[i] = positive(c[i]);
    }
    float o[kOut][4], mc[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < kOut; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

    auto stage = [&](const int key0) {
      const uint32_t bad = bads[mine * kStages + slot], keys = ring + slot * S::kStageBytes, values = keys + kFewBytes;
      const int box_rows = min(1 << p.page_shift, S::kKeys);
      const bool all = key0 + S::kKeys <= r.ctx && bad == 0;    // every row sees every key
      // ---- scores; columns 2 q and 2 q + 1 of octet n: keys 8 n + q and 8 n + q + 4
      float s[kOctets][4];
#pragma unroll
      for (int n = 0; n < kOctets; ++n) {
        const int key = 8 * n + ((g & 1) << 2 | g >> 1);
        float part[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};   // two chains, shorter than one
        if constexpr (kE4M3) {
#pragma unroll
          for (int j = 0; j < kSteps / 4; ++j) {
            const uint4 v = lds16(S::piece(keys, key, q + 4 * j));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) mma16<C>(part[i & 1], qf[4 * j + i], e4m3x2_to_f16x2(w[i] & 0xffffu), e4m3x2_to_f16x2(w[i] >> 16));
          }
        } else {
#pragma unroll
          for (int j = 0; j < kSteps / 2; ++j) {
            const uint4 v = lds16(S::piece(keys, key, 8 * (j >> 1) + q + 4 * (j & 1)));
            mma16<C>(part[0], qf[2 * j], v.x, v.y);
            mma16<C>(part[1], qf[2 * j + 1], v.z, v.w);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = part[0][e] + part[1][e];
      }
      uint32_t see[2][(S::kKeys + 31) / 32], there[(S::kKeys + 31) / 32];   // keys that the rows see; that exist
      if (!all) {
#pragma unroll
        for (int j = 0; j < (S::kKeys + 31) / 32; ++j) {
          uint32_t on = 0;                                      // keys on pages of the cache
#pragma unroll
          for (int k = 0; k < 32 && k < S::kKeys; k += 16)
            if (!(bad >> (32 * j + k) / box_rows & 1)) on |= 0xffffu << k;
          there[j] = on & visible32((1ull << r.rows) - 1, key0 + 32 * j, r.ctx);
#pragma unroll
          for (int i = 0; i < 2; ++i) see[i][j] = on & visible32(bits[i], key0 + 32 * j, r.ctx);
        }
#pragma unroll
        for (int n = 0; n < kOctets; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(see[e >> 1][n / 4] >> (8 * (n & 3) + q + 4 * (e & 1)) & 1)) s[n][e] = -INFINITY;
      }
      // ---- exponentials; the base of a row's exponents moves only when its maximum has grown by more than kSlack
      float now[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kOctets; ++n) top = fmaxf(top, fmaxf(s[n][2 * i], s[n][2 * i + 1]));
        now[i] = top == -INFINITY ? -INFINITY : fmaf(top, c[i], -M::kShift);
      }
      if (__any_sync(0xffffffffu, now[0] > mc[0] + kSlack || now[1] > mc[1] + kSlack)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          now[i] = fmaxf(now[i], __shfl_xor_sync(0xffffffffu, now[i], 1));
          now[i] = fmaxf(now[i], __shfl_xor_sync(0xffffffffu, now[i], 2));
          const bool grown = now[i] > mc[i] + kSlack;           // also from -inf
          const float f = grown ? (mc[i] == -INFINITY ? 0.f : exp2_fast(mc[i] - now[i])) : 1.f;
          if (grown) mc[i] = now[i];
          l[i] *= f;
#pragma unroll
          for (int t = 0; t < kOut; ++t) {
            o[t][2 * i] *= f;
            o[t][2 * i + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float from = mc[i] == -INFINITY ? 0.f : mc[i];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < kOctets; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[n][2 * i + e] = exp2_fast(fmaf(s[n][2 * i + e], c[i], -from));
            sum[e] += s[n][2 * i + e];
          }
        l[i] += sum[0] + sum[1];
      }
      // ---- outputs, 16 keys at a time. The probabilities are rounded to the products' type (m16n8k16 has both operands of one)
#pragma unroll
      for (int k = 0; k < kOctets / 2; ++k) {
        const uint32_t pf[4] = {M::pack(s[2 * k][0], s[2 * k][1]), M::pack(s[2 * k][2], s[2 * k][3]),
                                M::pack(s[2 * k + 1][0], s[2 * k + 1][1]), M::pack(s[2 * k + 1][2], s[2 * k + 1][3])};
        uint32_t odd = 0;                                       // keys (of the 16) with values that are not finite, where not every row sees all
        if constexpr (kE4M3) {
          constexpr int kWords = D / 32;
          uint32_t v[4][kWords];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = 16 * k + 4 * j + q, unit = (g & 1) << 2 | g >> 1;
            if constexpr (D == 128) {
              const uint4 x = lds16(S::piece(values, key, unit));
              v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
            } else {
              const uint2 x = lds8(S::piece(values, key, unit >> 1) + (unit & 1) * 8);
              v[j][0] = x.x, v[j][1] = x.y;
            }
            if (!all)
#pragma unroll
              for (int w = 0; w < kWords; ++w) {
                const uint32_t non = __vcmpeq4(v[j][w] & 0x7f7f7f7fu, 0x7f7f7f7fu);   // the only non-finite code is S.1111.111
                v[j][w] &= ~non;
                if (non) odd |= 1u << (4 * j + q);
              }
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int b = 0; b < 4; b += 2) {
              const uint32_t x = __byte_perm(v[0][w], v[1][w], b == 0 ? 0x5140 : 0x7362), y = __byte_perm(v[2][w], v[3][w], b == 0 ? 0x5140 : 0x7362);
              mma16<C>(o[4 * w + b], pf, e4m3x2_to_f16x2(x & 0xffffu), e4m3x2_to_f16x2(y & 0xffffu));
              mma16<C>(o[4 * w + b + 1], pf, e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(y >> 16));
            }
        } else {
          const int key = 16 * k + (lane & 8) + ((lane & 7) >> 1) + 4 * (lane & 1);
#pragma unroll
          for (int t = 0; t < kOut; t += 2) {
            uint32_t v[4];
            load_transposed(v, S::piece(values, key, t + (lane >> 4)));
            if (!all)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t non = __vcmpeq2(v[j] & M::kExponent, M::kExponent);
                v[j] &= ~non;
                if (non & 0xffffu) odd |= 1u << (8 * (j & 1) + q);
                if (non >> 16) odd |= 1u << (8 * (j & 1) + q + 4);
              }
            mma16<C>(o[t], pf, v[0], v[1]);
            mma16<C>(o[t + 1], pf, v[2], v[3]);
          }
        }
        if (!all) {
          odd = __reduce_or_sync(0xffffffffu, odd) & there[k / 2] >> (16 * (k & 1));
          // rare: the rows that see such a key add what was taken out
          for (; odd; odd &= odd - 1) {
            const int x = __ffs(odd) - 1, from = (lane & ~3) | (x & 3);
            const float up = x & 8 ? (x & 4 ? s[2 * k + 1][1] : s[2 * k + 1][0]) : (x & 4 ? s[2 * k][1] : s[2 * k][0]);
            const float down = x & 8 ? (x & 4 ? s[2 * k + 1][3] : s[2 * k + 1][2]) : (x & 4 ? s[2 * k][3] : s[2 * k][2]);
            const float pk[2] = {__shfl_sync(0xffffffffu, up, from), __shfl_sync(0xffffffffu, down, from)};
#pragma unroll
            for (int t = 0; t < kOut; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int d = S::element(t, 2 * q + e), key = 16 * k + x;
                const uint32_t a = S::piece(values, key, d * S::kBytes / 16) + d * S::kBytes % 16;
                float f;
                if constexpr (kE4M3) {
                  uint32_t code;
                  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(a) : "memory");
                  f = __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(code)));
                } else {
                  T y;
                  unsigned short code;
                  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(code) : "r"(a) : "memory");
                  memcpy(&y, &code, 2);
                  f = Elem<T>::to_float(y);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (!isfinite(f) && (see[i][k / 2] >> (16 * (k & 1) + x) & 1)) o[t][2 * i + e] += pk[i] * f;
              }
          }
        }
      }
    };
    const int n = stages<S::kKeys>(walk);
    for (int i = (mine - before) & (kRings - 1); i < n; i += kRings) {
      mbar_wait(full0 + 8 * slot, phase, p.spin_budget, p.status, dead);
      __syncwarp();
      if (active) stage(tile0 * kTileKeys + i * S::kKeys);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * slot);
      if (++slot == kStages) { slot = 0; phase ^= 1; }
    }
    before += n;

    // ---- the item's result: the warps' outputs on one base, four at a time added up in shared memory
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (q == 0) ml[warp * 16 + g + 8 * i] = make_float2(mc[i], l[i]);
    }
    join_barrier();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kRings; ++w) m = fmaxf(m, ml[(w * kBlocks + warp % kBlocks) * 16 + g + 8 * i].x);
      const float f = exp2_fast(mc[i] - (m == -INFINITY ? 0.f : m));
#pragma unroll
      for (int t = 0; t < kOut; ++t) {
        o[t][2 * i] *= f;
        o[t][2 * i + 1] *= f;
      }
    }
    float* place = reinterpret_cast<float*>(smem + S::kJoinAt) + (warp & 3) * (16 * S::kPitch);
    auto each = [&](auto&& f) {                                 // the lane's outputs and their place
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < kOut; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) f(o[t][2 * i + e], place[(g + 8 * i) * S::kPitch + S::element(t, 2 * q + e)]);
    };
    if (warp >= 4) each([](float& mine, float& there) { there = mine; });
    join_barrier();
    if (warp < 4) each([](float& mine, float& there) { there += mine; });
    join_barrier();
    {
      constexpr int kCols = D * kBlocks / 16, kPer = D / kCols;  // columns of a thread, threads of a row
      const int row = threadIdx.x / kPer, d = threadIdx.x % kPer * kCols, node = row / p.group;
      const float2* of_row = ml + row;                          // [ring][kRows]: a block's warps are those of its rows
      float m = -INFINITY, sum = 0.f, v[kCols];
#pragma unroll
      for (int w = 0; w < kRings; ++w) m = fmaxf(m, of_row[w * S::kRows].x);
      const float from = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < kRings; ++w) sum += of_row[w * S::kRows].y * exp2_fast(of_row[w * S::kRows].x - from);
      const float* joined = reinterpret_cast<const float*>(smem + S::kJoinAt) + row * S::kPitch + d;
#pragma unroll
      for (int j = 0; j < kCols; j += 4) {
        float4 x = *reinterpret_cast<const float4*>(joined + j);
#pragma unroll
        for (int w = kBlocks; w < 4; w += kBlocks) {
          const float4 y = *reinterpret_cast<const float4*>(joined + w * 16 * S::kPitch + j);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        v[j] = x.x, v[j + 1] = x.y, v[j + 2] = x.z, v[j + 3] = x.w;
      }
      const bool stored = row < rows && !*dead;
      if (stored) {
        if (whole) {
          const float f = sum == 0.f ? 0.f : (kE4M3 ? p.v_scale[h] : 1.f) / sum;
          const int head = h * p.group + row - node * p.group;
          T* dst = static_cast<T*>(p.out) + (int64_t)(r.row0 + node) * p.ldo + (int64_t)head * D + d;
          uint32_t packed[kCols / 2];
#pragma unroll
          for (int j = 0; j < kCols; j += 2) packed[j / 2] = sum == 0.f ? 0u : Mma<T>::pack(v[j] * f, v[j + 1] * f);
          if constexpr (kCols == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
          else
#pragma unroll
            for (int j = 0; j < kCols / 2; j += 4) *reinterpret_cast<uint4*>(dst + 2 * j) = make_uint4(packed[j], packed[j + 1], packed[j + 2], packed[j + 3]);
          if (p.lse && d == 0) p.lse[(int64_t)(r.row0 + node) * p.Hq + head] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        } else {
          const size_t part = (size_t)(2 * blockIdx.x + (tile0 > 0 ? 0 : 1)) * kTileRows + row;
#pragma unroll
          for (int j = 0; j < kCols; j += 4) *reinterpret_cast<float4*>(p.part_o + part * D + d + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          if (d == 0) p.part_ml[part] = make_float2(m, sum);
        }
      }
      if constexpr (kE4M3) {
        join_barrier();
      } else {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < kCols; ++j) odd |= isnan(v[j]);
        odd &= stored && isfinite(sum);
        __syncwarp();
        if (join_barrier_or(odd)) {
          T* out = whole ? static_cast<T*>(p.out) + (int64_t)(r.row0 + node) * p.ldo + (int64_t)(h * p.group + row - node * p.group) * D + d : nullptr;
          uint64_t sees = 0;
          if (odd) sees = (p.tree_mask ? p.tree_mask[r.row0 + node] : ~0ull >> (63 - node)) & ((1ull << r.rows) - 1);
          mend_item<T, D>(p, walk, reinterpret_cast<uint32_t*>(smem + S::kJoinAt), threadIdx.x, odd, out,
                          p.part_o + ((size_t)(2 * blockIdx.x + (tile0 > 0 ? 0 : 1)) * kTileRows + row) * D + d, d, kCols, sees);
        }
      }
    }
    walk.done(p, lane);                                         // sums and outputs are read; the next item may write
  }
  if (threadIdx.x == 0 && *dead) p.lost[blockIdx.x] = 1;
}

template <typename T, bool kE4M3, int D, int kBlocks>
cudaError_t launch(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  const cudaError_t e = allow_shared_memory<few_rows_kernel<T, kE4M3, D, kBlocks>>(dev);
  if (e != cudaSuccess) return e;
  few_rows_kernel<T, kE4M3, D, kBlocks><<<grid, kThreads, Few<T, kE4M3, D, kBlocks>::kSmem, s>>>(p, km, vm);
  return cudaGetLastError();
}
template <typename T, bool kE4M3, int D>
cudaError_t launch(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  return p.max_new * p.group <= 16 ? launch<T, kE4M3, D, 1>(p, km, vm, grid, dev, s) : launch<T, kE4M3, D, 2>(p, km, vm, grid, dev, s);
}
template <typename T>
cudaError_t launch(const AttnParams& p, bool e4m3, int D, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  if (D == 64) return e4m3 ? launch<T, true, 64>(p, km, vm, grid, dev, s) : launch<T, false, 64>(p, km, vm, grid, dev, s);
  return e4m3 ? launch<T, true, 128>(p, km, vm, grid, dev, s) : launch<T, false, 128>(p, km, vm, grid, dev, s);
}

}  // namespace

cudaError_t launch_few_rows(const AttnParams& p, bool bf16, bool e4m3, int D, const CUtensorMap& km, const CUtensorMap& vm, int grid, int dev, cudaStream_t s) {
  return bf16 ? launch<__nv_bfloat16>(p, e4m3, D, km, vm, grid, dev, s) : launch<__half>(p, e4m3, D, km, vm, grid, dev, s);
}

}  // namespace mdw
