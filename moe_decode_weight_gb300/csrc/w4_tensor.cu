// w4_linear for wide windows of many features: the products on tcgen05.
//
// Mathematics as in w4_linear.cu. 128 features are the lanes of tensor memory, the tokens (16 or 32, the missing ones
// zeros) the columns of a result. A group's codes - zero enter tensor memory as the first operand (128 lanes x
// half of the group's elements, two to a column), the tokens lie in shared memory as the second one, and a
// group has a result of its own: the scales are not rounded into the operands, they multiply the fp32
// results. A block walks over tiles of 128 features; per unit of 256 codes of each,
//   warp 0        requests the codes and the tokens' elements by TMA
//   warps 4-11    expand the codes into tensor memory, a thread a feature, four warps every other unit
//   warps 1, 2    issue the products, each those of every other unit (one warp alone took as long as the expansion)
//   warps 12-15   add scale times result to the thread's feature, all tokens in registers, and store them
// Warp 3 only completes the first group of four.
//
// Expansion. The tokens stay in their own order, so two neighbouring codes have to come out as the halves of a word: a
// byte goes into both halves, a mask leaves the first code in the low one and 16 times the second in the high one,
// and a fused multiply-add, exact in both halves, takes 16 and the zero out, as in Int4. 12 operations for eight
// codes of a feature, done once for all tokens.
//
// Measured, 157184 features x 2560 in groups of 128: 9 tokens 51.5 us, 32 tokens 60 us (3.8 TB/s; m16n8k16 products fed from
// shared memory took 63 and 104). What bounds it is the way of a half unit through its stages, expansion, products and
// sums, of which each takes 600 to 900 cycles and waits for the others' barriers, not one of them alone: without
// the expansion it is 15 % faster, without the products 8 %, from L2 2 %.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "mdw_internal.h"
#include "mdw_tcgen05.cuh"
#include "w4_linear.cuh"

namespace mdw {
namespace {

constexpr int kThreads = 512, kCodeBytes = kTensorRows * kUnit / 2, kHalf = kUnit / 2;
constexpr int kOperands = 4;                   // halves of a unit in tensor memory, expanded, 64 columns each

// Results pass from the products to the sums in halves of a unit, through up to eight of them in 256 columns.
template <int kGroup, int kTokens>
struct WideSmem {
  static constexpr int kHalfColumns = kHalf / kGroup * kTokens, kResults = 256 / kHalfColumns < 8 ? 256 / kHalfColumns : 8;
  static constexpr int kIssuers = kResults > 2 ? 2 : 1, kRing = kResults / kIssuers;   // warps that issue products, each with a ring of its own
  // Place of a half of unit n, and the parity of its round.
  static __device__ __forceinline__ int place(int n, int half) { return n % kIssuers * kRing + (2 * (n / kIssuers) + half) % kRing; }
  static __device__ __forceinline__ int round(int n, int half) { return (2 * (n / kIssuers) + half) / kRing & 1; }
  // Sums of a tile that other blocks continue (which = 1), or that this one continues (0).
  static __device__ __forceinline__ int part(int which, int t, int row) { return kJoin + ((which * kTokens + t) * kTensorRows + row) * 4; }
  static constexpr int kXBlock = kTokens * 128, kStageBytes = kCodeBytes + 4 * kXBlock;   // 64 elements of the tokens; codes and tokens of a unit
  static constexpr int kStages = 192 * 1024 / kStageBytes, kJoin = kStages * kStageBytes, kBars = kJoin + 2 * kTokens * kTensorRows * 4;
  static constexpr int kFull = kBars, kEmpty = kFull + 8 * kStages, kOperand = kEmpty + 8 * kStages, kOperandFree = kOperand + 8 * kOperands;
  static constexpr int kResult = kOperandFree + 8 * kOperands, kResultFree = kResult + 8 * kResults, kEnd = kResultFree + 8 * kResults;
  static constexpr int kDead = kEnd + 8, kTmem = kDead + 4, kTotal = kTmem + 4 + 1024;   // (and the alignment of the swizzled tiles)
};

// Eight codes, neighbours in the halves of a word.
template <typename T> struct Neighbours;
template <> struct Neighbours<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t zero(uint32_t z) { return Int4<__nv_bfloat16>::zero2(z); }
  static __device__ __forceinline__ uint32_t expand(uint32_t two, uint32_t z) { return Int4<__nv_bfloat16>::fma2(two & 0x00f0000fu, 0x7d007f00u, z); }
};
template <> struct Neighbours<__half> {
  // -(64 + z), -(1024 + z): (960, 0) - (1024 + z), exactly
  static __device__ __forceinline__ uint32_t zero(uint32_t z) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(0x63800000u), "r"(0x64006400u + z * 0x00010001u));
    return r;
  }
  static __device__ __forceinline__ uint32_t expand(uint32_t two, uint32_t z) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(and_or(two, 0x00f0000fu, 0x64006400u)), "r"(0x2c003c00u), "r"(z));
    return r;
  }
};

// Position in the block's share of the sequence of (tile, unit), over which every role walks.
struct Units {
  int tile, unit, units, left;     // units of a tile; units left in the share
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next() {
    --left;
    if (++unit == units) {
      unit = 0;
      ++tile;
    }
  }
};

// The tiles are divided among the clusters, and the (tile, unit) sequence of a cluster into equal contiguous shares of its
// blocks: a tile cut between blocks is finished from their sums, in order, when all are done.
struct Share {
  int t0, units, per, rest;        // cluster's first tile, units of a tile; of a block of it (the first `rest` blocks have one more)
  __device__ __forceinline__ Share(const W4Params& p, int blocks) {
    const int tiles = (p.N + kTensorRows - 1) / kTensorRows, clusters = (unsigned)gridDim.x / (unsigned)blocks, c = (unsigned)blockIdx.x / (unsigned)blocks;
    const int some = (unsigned)tiles / (unsigned)clusters, more = tiles - some * clusters;
    units = (p.K + kUnit - 1) / kUnit;
    t0 = c * some + min(c, more);
    const int all = (some + (c < more)) * units;
    per = (unsigned)all / (unsigned)blocks;
    rest = all - per * blocks;
  }
  __device__ __forceinline__ int start(int rank) const { return rank * per + min(rank, rest); }
};

// Scales or zeros of one unit (256 / kGroup of them) for one feature.
template <int kGroup>
struct UnitScales {
  static constexpr int kGroups = kUnit / kGroup;
  uint32_t w[kGroups / 2];
  __device__ __forceinline__ void load(const W4Params& p, const Units& at, int row) {
    const int groups = p.K / kGroup, first = at.unit * kGroups;
    const uint16_t* src = static_cast<const uint16_t*>(p.scale) + (size_t)min(at.tile * kTensorRows + row, p.N - 1) * groups + first;
    if (p.K % kUnit == 0) {
      if constexpr (kGroups == 2) w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
      if constexpr (kGroups == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        w[0] = v.x, w[1] = v.y;
      }
      if constexpr (kGroups == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kGroups; j += 2)                      // those behind the row's end are zeros
        w[j / 2] = (first + j < groups ? (uint32_t)__ldg(src + j) : 0u) | (first + j + 1 < groups ? (uint32_t)__ldg(src + j + 1) << 16 : 0u);
    }
  }
  template <typename T> __device__ __forceinline__ float get(int j) const {
    const unsigned short v = (unsigned short)(w[j / 2] >> (16 * (j & 1)));
    T t;
    memcpy(&t, &v, 2);
    return Elem<T>::to_float(t);
  }
};
template <int kGroup>
struct UnitZeros {
  static constexpr int kGroups = kUnit / kGroup;
  uint32_t w[(kGroups + 3) / 4];
  __device__ __forceinline__ void load(const W4Params& p, const Units& at, int row) {
#pragma unroll
    for (int j = 0; j < (kGroups + 3) / 4; ++j) w[j] = 0x08080808u;
    if (!p.zero) return;
    const int groups = p.K / kGroup, first = at.unit * kGroups;
    const uint8_t* src = p.zero + (size_t)min(at.tile * kTensorRows + row, p.N - 1) * groups + first;
    if (p.K % kUnit == 0) {
      if constexpr (kGroups == 2) w[0] = __ldg(reinterpret_cast<const uint16_t*>(src));
      if constexpr (kGroups == 4) w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
      if constexpr (kGroups == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        w[0] = v.x, w[1] = v.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kGroups; ++j)
        if (first + j < groups) w[j / 4] = (w[j / 4] & ~(0xffu << 8 * (j % 4))) | (uint32_t)__ldg(src + j) << 8 * (j % 4);
    }
  }
  __device__ __forceinline__ uint32_t get(int j) const { return w[j / 4] >> (8 * (j % 4)) & 0xffu; }
};

// A unit's scales and zeros, kFar units ahead: under load memory answers later than one unit takes.
constexpr int kFar = 4;
template <int kGroup>
__device__ __forceinline__ void prefetch_scales(const W4Params& p, const Units& at, int row) {
  const size_t first = (size_t)min(at.tile * kTensorRows + row, p.N - 1) * (p.K / kGroup) + at.unit * (kUnit / kGroup);
  asm volatile("prefetch.global.L2 [%0];" :: "l"(static_cast<const uint16_t*>(p.scale) + first));
  if (p.zero) asm volatile("prefetch.global.L2 [%0];" :: "l"(p.zero + first));
}

// One rounding of a token's feature, after bias and residual.
template <typename T>
__device__ __forceinline__ void store(const W4Params& p, int t, int feature, float v) {
  if (p.bias) v += Elem<T>::to_float(static_cast<const T*>(p.bias)[feature]);
  if (p.residual) v += Elem<T>::to_float(static_cast<const T*>(p.residual)[t * p.ldr + feature]);
  if (p.y_f32) static_cast<float*>(p.y)[t * p.ldy + feature] = v;
  else static_cast<T*>(p.y)[t * p.ldy + feature] = Elem<T>::from_float(v);
}

template <typename T, int kGroup, int kTokens>
__global__ void __launch_bounds__(kThreads, 1)
w4_tensor_kernel(const W4Params p, const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap tokens, int blocks) {
  using L = WideSmem<kGroup, kTokens>;
  extern __shared__ uint8_t raw_smem[];
  const uint32_t base = (smem_u32(raw_smem) + 1023) & ~1023u;
  uint8_t* smem = raw_smem + (base - smem_u32(raw_smem));
  volatile int* dead = reinterpret_cast<volatile int*>(smem + L::kDead);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int at, int i) { return base + at + 8 * i; };
  auto wait = [&](uint32_t b, uint32_t parity) { mbar_wait(b, parity, p.spin_budget, p.status, dead); };
  if (threadIdx.x == 0) {
    prefetch_map(&codes);
    prefetch_map(&tokens);
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar(L::kFull, i), 1);
      mbar_init(bar(L::kEmpty, i), 5);                          // four warps that expand; the products
    }
    for (int i = 0; i < kOperands; ++i) {
      mbar_init(bar(L::kOperand, i), 4);
      mbar_init(bar(L::kOperandFree, i), 1);
    }
    for (int i = 0; i < L::kResults; ++i) {
      mbar_init(bar(L::kResult, i), 1);
      mbar_init(bar(L::kResultFree, i), 4);
    }
    mbar_init(bar(L::kEnd, 0), L::kIssuers);
    *dead = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(base + L::kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + L::kTmem), 0);
  const Share share(p, blocks);
  const int rank = blockIdx.x % blocks, units = share.units, u0 = share.start(rank), u1 = share.start(rank + 1);
  Units at{share.t0 + u0 / units, u0 % units, units, u1 - u0};

  if (warp == 0) {
    // ---- copies
    if (lane == 0) {
      int n = 0;
      for (; at.more(); at.next(), ++n) {
        const int stage = n % L::kStages;
        const uint32_t full = bar(L::kFull, stage), to = base + stage * L::kStageBytes;
        wait(bar(L::kEmpty, stage), (n / L::kStages & 1) ^ 1);
        if (*dead) break;
        mbar_arrive_tx(full, L::kStageBytes);
        tma_codes(to, &codes, full, at.unit * (kUnit / 2), at.tile * kTensorRows);
#pragma unroll
        for (int i = 0; i < kUnit / 64; ++i) tma_codes(to + kCodeBytes + i * L::kXBlock, &tokens, full, at.unit * kUnit + 64 * i, 0);
      }
      // what was requested arrives before the block ends, also where a wait runs out after the last request
      for (int i = n > L::kStages ? n - L::kStages : 0; i < n; ++i) mbar_drain(bar(L::kFull, i % L::kStages), i / L::kStages & 1);
    }
    __syncwarp();
  } else if (warp <= L::kIssuers) {
    // ---- products
    if (warp == 2) at.next();
    for (int n = warp - 1; at.more(); n += L::kIssuers) {
      const int stage = n % L::kStages;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int from = (2 * n + half) % kOperands, to = L::place(n, half);
        const uint32_t a = tmem + from * 64, d = tmem + kOperands * 64 + to * L::kHalfColumns;
        const uint32_t x = operand_low(base + stage * L::kStageBytes + kCodeBytes + half * 2 * L::kXBlock, 16);
        wait(bar(L::kResultFree, to), L::round(n, half) ^ 1);
        // the codes are expanded, so the unit's copies, the tokens among them, are there as well
        wait(bar(L::kOperand, from), n / 2 & 1);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < kHalf / 16; ++t)
            tc_mma_tmem(d + t * 16 / kGroup * kTokens, a + 8 * t, x + ((t / 4 * L::kXBlock + t % 4 * 32) >> 4),
                        mma_shape(std::is_same<T, __nv_bfloat16>::value, false, kTokens), t * 16 % kGroup != 0);
          tc_commit(bar(L::kResult, to));
          tc_commit(bar(L::kOperandFree, from));
          if (half == 1) tc_commit(bar(L::kEmpty, stage));
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < L::kIssuers; ++i)
        if (at.more()) at.next();
    }
    if (lane == 0) tc_commit(bar(L::kEnd, 0));
    __syncwarp();
    mbar_drain(bar(L::kEnd, 0), 0);                             // nothing is in flight when the columns are given back
  } else if (warp >= 4 && warp < 12) {
    // ---- expansion: thread = feature, every other unit
    const int set = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
    UnitZeros<kGroup> now, next;
    if (set == 1) at.next();
    if (at.more()) next.load(p, at, row);
    for (int n = set; at.more(); n += 2) {
      now = next;
      at.next();
      if (at.more()) at.next();
      if (at.more()) next.load(p, at, row);
      const int stage = n % L::kStages;
      wait(bar(L::kFull, stage), n / L::kStages & 1);
      __syncwarp();
      const uint32_t src = base + stage * L::kStageBytes + row * 128;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int h = 2 * n + half, to = h % kOperands;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lds128(src + ((4 * half + i) ^ (row & 7)) * 16);
        wait(bar(L::kOperandFree, to), (h / kOperands & 1) ^ 1);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          const uint32_t z = Neighbours<T>::zero(now.get((kHalf * half + 32 * i) / kGroup));
          uint32_t e[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) e[j] = Neighbours<T>::expand(__byte_perm(w[j / 4], 0u, 0x4040u + 0x0101u * (j % 4)), z);
          tc_st16(tmem + lanes + to * 64 + 16 * i, e);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::kOperand, to));
          if (half == 1) mbar_arrive(bar(L::kEmpty, stage));
        }
      }
    }
  } else if (warp >= 12) {
    // ---- sums: thread = feature
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
    UnitScales<kGroup> now, next;
    next.load(p, at, row);
    Units far = at;                                             // scales and zeros come into L2 before they are loaded
    for (int i = 0; i < kFar && far.more(); ++i) {
      prefetch_scales<kGroup>(p, far, row);
      far.next();
    }
    float acc[kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) acc[t] = 0.f;
    bool from_start = at.unit == 0;                             // of the tile
    for (int n = 0; at.more(); ++n) {
      const int feature = at.tile * kTensorRows + row, unit = at.unit;
      now = next;
      at.next();
      if (at.more()) next.load(p, at, row);
      if (far.more()) {
        prefetch_scales<kGroup>(p, far, row);
        far.next();
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int from = L::place(n, half);
        wait(bar(L::kResult, from), L::round(n, half));
        __syncwarp();
        tc_fence_after();
        constexpr int kGroups = kHalf / kGroup, kAtOnce = kGroups * kTokens <= 64 ? kGroups : 64 / kTokens;
#pragma unroll
        for (int j0 = 0; j0 < kGroups; j0 += kAtOnce) {
          float d[kAtOnce][kTokens];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const uint32_t src = tmem + lanes + kOperands * 64 + from * L::kHalfColumns + (j0 + j) * kTokens;
            if constexpr (kTokens == 32) tc_ld32(d[j], src);
            else tc_ld16(d[j], src);
          }
          tc_wait_ld();
          if (j0 + kAtOnce == kGroups) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kResultFree, from));
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const float s = Int4<T>::kFactor * now.template get<T>(half * kGroups + j0 + j);
#pragma unroll
            for (int t = 0; t < kTokens; ++t) acc[t] = fmaf(s, d[j][t], acc[t]);
          }
        }
      }
      if (unit + 1 < units && at.more()) continue;
      if (unit + 1 == units && from_start) {
        if (feature < p.N && !*dead) {
#pragma unroll
          for (int t = 0; t < kTokens; ++t)
            if (t < p.M) store<T>(p, t, feature, acc[t]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < kTokens; ++t)
          asm volatile("st.shared.f32 [%0], %1;" :: "r"(base + L::part(from_start, t, row)), "f"(acc[t]) : "memory");
      }
      from_start = true;
#pragma unroll
      for (int t = 0; t < kTokens; ++t) acc[t] = 0.f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
  }
  if (blocks == 1) return;
  sync_cluster();
  bool lost = false;                                            // a dead block anywhere in the cluster
  for (int r = 0; r < blocks; ++r) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_block(base + L::kDead, r)) : "memory");
    lost |= v != 0;
  }
  // Tiles that this share starts inside of or ends inside of. Of up to three blocks with parts of one the second adds
  // them up; of more each adds up some of the tokens.
  const int row = (warp & 3) * 32 + lane;
  auto part = [&](int rank, int which, int t) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(in_block(base + L::part(which, t, row), rank)) : "memory");
    return v;
  };
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int u = which ? u1 : u0, tile = u / units, begin = tile * units, feature = (share.t0 + tile) * kTensorRows + row;
    if (u == begin || (which == 1 && u0 > begin)) continue;
    int first = rank, end = rank;                               // blocks with a part of it
    while (share.start(first) > begin) --first;
    while (share.start(end + 1) < begin + units) ++end;
    const int n = end - first + 1;
    if (n <= 3) {
      if (rank != first + 1) continue;
      float v[3][kTokens / 4];                                  // requested together: each takes some 250 cycles
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int j = 0; j < kTokens / 4; ++j) v[i][j] = i < n ? part(first + i, i == 0, (warp >> 2) + 4 * j) : 0.f;
#pragma unroll
      for (int j = 0; j < kTokens / 4; ++j)
        if (feature < p.N && (warp >> 2) + 4 * j < p.M && !lost) store<T>(p, (warp >> 2) + 4 * j, feature, v[0][j] + v[1][j] + v[2][j]);
    } else {
      for (int t = rank - first + n * (warp >> 2); t < p.M; t += 4 * n) {
        float v[kMostCluster], sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMostCluster; ++i) v[i] = i < n ? part(first + i, i == 0, t) : 0.f;
#pragma unroll
        for (int i = 0; i < kMostCluster; ++i) sum += v[i];
        if (feature < p.N && !lost) store<T>(p, t, feature, sum);
      }
    }
  }
  sync_cluster();                                               // no block ends while another reads its sums
}

// The tokens as [M][K] elements; a box is 64 elements of all of them, those that are missing zeros.
bool encode_tokens(CUtensorMap* map, const W4Params& p, int tokens) {
  const cuuint64_t dims[2] = {(cuuint64_t)p.K, (cuuint64_t)p.M}, strides[1] = {(cuuint64_t)p.ldx * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)tokens}, ones[2] = {1, 1};
  const EncodeTiledFn fn = encode_tiled();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(p.x), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kJoinUnits = 4;

template <typename T, int kGroup, int kTokens>
cudaError_t launch(const W4Params& p, const CUtensorMap& codes, int dev, cudaStream_t s) {
  constexpr auto kKernel = w4_tensor_kernel<T, kGroup, kTokens>;
  const cudaError_t e = allow_shared_memory<kKernel>(dev);
  if (e != cudaSuccess) return e;
  CUtensorMap tokens;
  if (!encode_tokens(&tokens, p, kTokens)) return cudaErrorInvalidValue;
  const int tiles = (p.N + kTensorRows - 1) / kTensorRows, units = (p.K + kUnit - 1) / kUnit;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = WideSmem<kGroup, kTokens>::kTotal;
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  // Blocks to a cluster: the fewest units in a block's share, a join counted as kJoinUnits of them.
  int blocks = 1, many = std::min(sm_count(dev), tiles), best = (tiles + many - 1) / many * units;
  for (int n = 2; n <= kMostCluster && n <= units; ++n) {
    a.val.clusterDim.x = n;
    cfg.gridDim = dim3((unsigned)n);
    const int fit = std::min(clusters<kKernel>(cfg, n, dev), tiles);
    if (fit < 1) continue;
    const int cost = ((tiles + fit - 1) / fit * units + n - 1) / n + kJoinUnits;
    if (cost < best) {
      best = cost;
      blocks = n;
      many = fit;
    }
  }
  a.val.clusterDim.x = blocks;
  cfg.gridDim = dim3((unsigned)(blocks * many));
  return cudaLaunchKernelEx(&cfg, kKernel, p, codes, tokens, blocks);
}
template <typename T, int kGroup>
cudaError_t launch(const W4Params& p, const CUtensorMap& codes, int dev, cudaStream_t s) {
  return p.M <= 16 ? launch<T, kGroup, 16>(p, codes, dev, s) : launch<T, kGroup, 32>(p, codes, dev, s);
}
template <typename T>
cudaError_t launch(const W4Params& p, const CUtensorMap& codes, int group, int dev, cudaStream_t s) {
  return group == 32 ? launch<T, 32>(p, codes, dev, s) : (group == 64 ? launch<T, 64>(p, codes, dev, s) : launch<T, 128>(p, codes, dev, s));
}

}  // namespace

cudaError_t launch_w4_tensor(const W4Params& p, const CUtensorMap& codes, bool bf16, int group, int dev, cudaStream_t s) {
  return bf16 ? launch<__nv_bfloat16>(p, codes, group, dev, s) : launch<__half>(p, codes, group, dev, s);
}

}  // namespace mdw
