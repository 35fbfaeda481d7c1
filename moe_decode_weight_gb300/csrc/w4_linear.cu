// w4_linear: y = x . W^T (+ bias) (+ residual) with W in int4 codes and group scales, for windows of
// up to MDW_MAX_M tokens.
//
// Mathematics. y[t][n] = sum over groups s[n][j] * sum over the group's k of (code - zero) x[t][k]: the inner sum on
// the tensor cores (integers up to 15 times 16-bit elements, exact products, fp32 sums), the outer
// one in fp32. m16n8k16 with 16 features as the rows and 8 tokens as the columns.
//
// Codes. A lane (g, q) of a product holds two features and a quarter of a group's codes (8, 16 or 32 of them, one
// load), so the four lanes of a product always share a group. Masking a word by 0x000f000f leaves codes
// j and j + 4 in its halves, by 0x00f000f0 codes j + 1 and j + 5, times 16. Under the exponent of 1024 that is a
// f16 number, and as it is a bf16 one (see Int4); one more operation, exact, leaves code - zero. The
// token's elements are put in the same order once, when they enter shared memory. This expansion takes
// 9 operations for eight codes of a feature, whatever the number of tokens, of which 5 on the integer pipe. 157184
// features x 2560, one token: 43.3 us, 4.8 TB/s, issuing in 62 % of the cycles with the memory at 58 % of its rate: neither is
// full, and a warp has two units of 4 KB on their way.
#include <type_traits>

#include "mdw_internal.h"
#include "w4_linear.cuh"

namespace mdw {
namespace {

template <int kWords> __device__ __forceinline__ void lds_words(uint32_t (&w)[kWords], uint32_t a) {
  if constexpr (kWords == 1) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
  if constexpr (kWords == 2) asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  if constexpr (kWords == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
}
// Where a lane's two features' scales and zeros lie.
template <typename T>
struct ScaleRows {
  const uint16_t* s[2];
  const uint8_t* z[2];
  __device__ __forceinline__ void begin(const W4Params& p, int n, int groups) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const size_t at = (size_t)min(n + 8 * i, p.N - 1) * groups;
      s[i] = static_cast<const uint16_t*>(p.scale) + at;
      z[i] = p.zero + at;                       // not read without zeros
    }
  }
};

// Scales and zeros of one unit for those features, requested one unit ahead: the sectors come
// from memory, and a load at the point of use would stall every unit.
template <typename T, int kGroup>
struct Scales {
  static constexpr int kGroups = kUnit / kGroup;
  uint32_t s[2][kGroups / 2], z[2][(kGroups + 3) / 4];

  // Rows of whole units start on the boundary of a unit's scales, so one load serves a row.
  __device__ __forceinline__ void load(const W4Params& p, const ScaleRows<T>& rows, int unit) {
    if (p.K % kUnit != 0) {
      Scales part;
      part.load_single(p, rows, unit);
      *this = part;
      return;
    }
    const int first = unit * kGroups;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint16_t* src = rows.s[i] + first;
      if constexpr (kGroups == 2) {
        s[i][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
      } else if constexpr (kGroups == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        s[i][0] = v.x;
        s[i][1] = v.y;
      } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
        s[i][0] = v.x;
        s[i][1] = v.y;
        s[i][2] = v.z;
        s[i][3] = v.w;
      }
    }
    if (p.zero) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* zero = rows.z[i] + first;
        if constexpr (kGroups == 2) {
          z[i][0] = __ldg(reinterpret_cast<const uint16_t*>(zero));
        } else if constexpr (kGroups == 4) {
          z[i][0] = __ldg(reinterpret_cast<const uint32_t*>(zero));
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(zero));
          z[i][0] = u.x;
          z[i][1] = u.y;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < (kGroups + 3) / 4; ++j) z[0][j] = z[1][j] = 0x08080808u;
    }
  }
  // Otherwise the scales are read one by one, and those behind the row's end not at all.
  __device__ __noinline__ void load_single(const W4Params& p, const ScaleRows<T>& rows, int unit) {
    const int first = unit * kGroups, left = p.K / kGroup - first;
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < (kGroups + 3) / 4; ++j) z[i][j] = 0x08080808u;
      for (int j = 0; j < kGroups / 2; ++j) s[i][j] = 0u;
      for (int j = 0; j < kGroups && j < left; ++j) {
        s[i][j / 2] |= (uint32_t)__ldg(rows.s[i] + first + j) << (16 * (j & 1));
        if (p.zero) z[i][j / 4] = (z[i][j / 4] & ~(0xffu << (8 * (j & 3)))) | (uint32_t)__ldg(rows.z[i] + first + j) << (8 * (j & 3));
      }
    }
  }
  __device__ __forceinline__ float scale(int i, int j) const {
    const unsigned short v = (unsigned short)(s[i][j / 2] >> (16 * (j & 1)));
    T t;
    memcpy(&t, &v, 2);
    return Int4<T>::kFactor * Elem<T>::to_float(t);
  }
  __device__ __forceinline__ uint32_t zero2(int i, int j) const {
    return Int4<T>::zero2((z[i][j / 4] >> (8 * (j & 3))) & 0xffu);
  }
};

// A lane's part of a line and of a token. Feature of product row g: bit-reversed g, so that the rows that one
// phase of a 4-, 8- or 16-byte load touches lie in different banks of the swizzled lines.
template <int kGroup>
struct Lane {
  static constexpr int kWords = kGroup / 32;                    // words of a group per lane
  static __device__ __forceinline__ int feature(int lane) { return lane >> 4 | (lane >> 2 & 2) | (lane & 4); }
  // Offset of group 0 in the line of `feature`; group s lies at this ^ (s * kGroup / 2).
  static __device__ __forceinline__ uint32_t code(int lane) {
    const int f = feature(lane), q = lane & 3;
    return f * 128 + (((kWords == 4 ? q : kWords == 2 ? q >> 1 : 0) << 4) ^ (f << 4)) + (kWords == 2 ? (q & 1) * 8 : kWords == 1 ? q * 4 : 0);
  }
  // Where elements k .. k + 7 of a token go: word w of lane q of a group at 64 w + 16 q.
  static __device__ __forceinline__ int element(int k) {
    const int c = k % kGroup / 8;
    return k / kGroup * (2 * kGroup) + c % kWords * 64 + c / kWords * 16;
  }
};

// 16 features x kUnit codes x 8 tokens: acc += scale * (codes - zero) . x. `code`: the lane's words of group 0 (its
// second feature lies 1,024 bytes further). x: the lane's elements of its token; a column without a token
// repeats the last one's, its sums are not stored. Codes and elements behind K are zeros.
template <typename T, int kGroup>
__device__ __forceinline__ void multiply(uint32_t code, uint32_t x, const Scales<T, kGroup>& sc, float (&acc)[4]) {
  constexpr int kWords = Lane<kGroup>::kWords;
  constexpr float kNone[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < kUnit / kGroup; ++s) {
    const uint32_t z0 = sc.zero2(0, s), z1 = sc.zero2(1, s);
    // two chains of products, so that one need not wait for the other's result
    constexpr int kChains = kWords > 1 ? 2 : 1;
    float d[kChains][4];
    uint32_t w0[kWords], w1[kWords];
    lds_words<kWords>(w0, code ^ (s * kGroup / 2));
    lds_words<kWords>(w1, (code ^ (s * kGroup / 2)) + 1024);
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      uint32_t lo[4], hi[4];
      Int4<T>::expand(w0[w], z0, lo);
      Int4<T>::expand(w1[w], z1, hi);
      float (&sum)[4] = d[w % kChains];
      const uint4 v = lds128(x + s * (2 * kGroup) + 64 * w);
      if (w < kChains) Int4<T>::mma(sum, kNone, lo[0], hi[0], lo[1], hi[1], v.x, v.y);
      else Int4<T>::mma(sum, sum, lo[0], hi[0], lo[1], hi[1], v.x, v.y);
      Int4<T>::mma(sum, sum, lo[2], hi[2], lo[3], hi[3], v.z, v.w);
    }
    const float s0 = sc.scale(0, s), s1 = sc.scale(1, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float sum = d[0][e];
      if constexpr (kChains == 2) sum += d[1][e];
      acc[e] = fmaf(e < 2 ? s0 : s1, sum, acc[e]);
    }
  }
}

// The lane's two features of the 16 from n0 on, tokens 2 q + {0, 1}: bias, residual, one rounding.
template <typename T>
__device__ __forceinline__ void store(const W4Params& p, int n0, int lane, const float (&acc)[4]) {
  const int f = Lane<32>::feature(lane), q = lane & 3;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int n = n0 + f + 8 * (e >> 1), t = 2 * q + (e & 1);
    if (n >= p.N || t >= p.M) continue;
    float v = acc[e];
    if (p.bias) v += Elem<T>::to_float(static_cast<const T*>(p.bias)[n]);
    if (p.residual) v += Elem<T>::to_float(static_cast<const T*>(p.residual)[t * p.ldr + n]);
    if (p.y_f32) static_cast<float*>(p.y)[t * p.ldy + n] = v;
    else static_cast<T*>(p.y)[t * p.ldy + n] = Elem<T>::from_float(v);
  }
}

// ------------------------------------------------------------------ windows of up to 8 tokens
//
// A cluster of blocks (most often of one) owns a contiguous range of 16-feature tiles and cuts its (tile, unit) sequence into
// equal contiguous shares, one per warp; each warp streams its share through a ring of its own (two TMA boxes of
// 16 x 128 bytes a unit), with no barrier between the first and the last. A tile cut between warps is
// finished from their partial sums, in order. x stays in each block's shared memory as a whole.
constexpr int kRowWarps = 8, kRowStages = 2, kLineBytes = 16 * kUnit / 2, kRowUnit = 2 * kUnit, kRowBytes = 2 * kLineBytes;
constexpr int kRowJoin = 10;
constexpr int kRowMaxX = 36 * 1024;            // bytes of x that leave room for two blocks on an SM

// Bytes of a token in shared memory, whole units; 64 more put two tokens' loads on different banks.
__host__ __device__ constexpr int x_pitch(int K) { return (K + kRowUnit - 1) / kRowUnit * kRowUnit * 2 + 64; }

template <typename T, int kGroup>
__global__ void __launch_bounds__(32 * kRowWarps, 2)
w4_rows_kernel(const W4Params p, const __grid_constant__ CUtensorMap codes, int tiles, int blocks) {
  extern __shared__ uint8_t raw_smem[];
  __shared__ float part[kRowWarps][2][4][32];
  __shared__ __align__(8) uint64_t bars[kRowWarps][kRowStages];
  __shared__ int dead_flag;
  volatile int* dead = &dead_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, f = Lane<kGroup>::feature(lane);
  const uint32_t base = (smem_u32(raw_smem) + 1023) & ~1023u;
  const uint32_t ring = base + warp * kRowStages * kRowBytes, xs = base + kRowWarps * kRowStages * kRowBytes;
  const uint32_t bar = smem_u32(&bars[warp][0]);
  const int units = (p.K + kRowUnit - 1) / kRowUnit, pitch = x_pitch(p.K);
  // (32-bit divisions, and few: a warp that starts with 64-bit ones starts a microsecond later)
  const unsigned clusters = blocks == 1 ? gridDim.x : gridDim.x / (unsigned)blocks, cluster = blocks == 1 ? blockIdx.x : blockIdx.x / (unsigned)blocks;
  const int all_warps = kRowWarps * blocks, mine = ((int)blockIdx.x - (int)cluster * blocks) * kRowWarps + warp;   // the warp's place in the cluster
  const int some = (unsigned)tiles / clusters, more = tiles - some * (int)clusters;
  const int t0 = (int)cluster * some + min((int)cluster, more), n_tiles = some + ((int)cluster < more);
  const int all = n_tiles * units;                              // the cluster's units (the host bounds them)
  const int per = (unsigned)all / (unsigned)all_warps, rest = all - per * all_warps;
  auto share = [&](int w) { return w * per + min(w, rest); };
  const int u0 = share(mine), u1 = share(mine + 1);

  int tile = u0 / units, unit = u0 - tile * units;
  int ask = u0, ask_tile = tile, ask_unit = unit;
  auto request = [&](int stage) {                               // lane 0
    mbar_arrive_tx(bar + 8 * stage, kRowBytes);
    tma_codes(ring + stage * kRowBytes, &codes, bar + 8 * stage, ask_unit * (kRowUnit / 2), (t0 + ask_tile) * 16);
    tma_codes(ring + stage * kRowBytes + kLineBytes, &codes, bar + 8 * stage, ask_unit * (kRowUnit / 2) + kUnit / 2, (t0 + ask_tile) * 16);
    ++ask;
    if (++ask_unit == units) { ask_unit = 0; ++ask_tile; }
  };
  if (threadIdx.x == 0) *dead = 0;
  if (lane == 0) {
    for (int i = 0; i < kRowStages; ++i) mbar_init(bar + 8 * i, 1);
    mbar_init_fence();
    for (int i = 0; i < kRowStages && ask < u1; ++i) request(i);
  }
  Scales<T, kGroup> now[2], next[2];
  ScaleRows<T> rows;
  int s_tile = tile, s_unit = unit, s_at = u0;
  rows.begin(p, (t0 + tile) * 16 + f, p.K / kGroup);
  auto scales = [&](Scales<T, kGroup> (&s)[2]) {
    if (s_at >= u1) return;
    s[0].load(p, rows, 2 * s_unit);
    if (s_unit * kRowUnit + kUnit < p.K) s[1].load(p, rows, 2 * s_unit + 1);
    ++s_at;
    if (++s_unit == units) {
      s_unit = 0;
      ++s_tile;
      rows.begin(p, (t0 + s_tile) * 16 + f, p.K / kGroup);
    }
  };
  scales(now);
  const int pieces = units * (kRowUnit / 8), all_pieces = p.M * pieces;
  for (int i = threadIdx.x; i < all_pieces; i += 4 * 32 * kRowWarps) {
    uint4 v[4];
    uint32_t to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = i + j * 32 * kRowWarps, t = at / pieces, k = (at - t * pieces) * 8;
      to[j] = xs + t * pitch + Lane<kGroup>::element(k);
      v[j] = at < all_pieces && k < p.K ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + t * p.ldx + k) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * 32 * kRowWarps < all_pieces) sts_paired(to[j], v[j]);
  }
  __syncthreads();

  bool from_start = unit == 0;
  int stage = 0;
  uint32_t phase = 0;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const uint32_t code = ring + Lane<kGroup>::code(lane), x = xs + min(lane >> 2, p.M - 1) * pitch + 16 * (lane & 3);
  for (int u = u0; u < u1; ++u) {
    scales(next);
    mbar_wait(bar + 8 * stage, phase, p.spin_budget, p.status, dead);
    __syncwarp();
    const uint32_t at = code + stage * kRowBytes, x0 = x + unit * (2 * kRowUnit);
    multiply<T, kGroup>(at, x0, now[0], acc);
    if (unit * kRowUnit + kUnit < p.K) multiply<T, kGroup>(at + kLineBytes, x0 + 2 * kUnit, now[1], acc);
    __syncwarp();
    if (lane == 0 && ask < u1 && !*dead) request(stage);
    now[0] = next[0];
    now[1] = next[1];
    if (++stage == kRowStages) { stage = 0; phase ^= 1; }
    if (++unit == units || u + 1 == u1) {
      if (from_start && unit == units) {
        if (!*dead) store<T>(p, (t0 + tile) * 16, lane, acc);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][from_start ? 1 : 0][e][lane] = acc[e];
      }
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      from_start = true;
      if (unit == units) { unit = 0; ++tile; }
    }
  }
  if (*dead && lane == 0)
    // what this warp requested has arrived or arrives now: its i-th copy into a stage ends phase i
    for (int i = 0; i < kRowStages; ++i) {
      const int n = (ask - u0 - i + kRowStages - 1) / kRowStages;
      if (ask - u0 > i) mbar_drain(bar + 8 * i, (n - 1) & 1);
    }
  __syncwarp();
  bool lost;                                                    // a dead block anywhere in the cluster
  if (blocks == 1) {
    __syncthreads();
    lost = *dead;
  } else {
    sync_cluster();
    lost = false;
    for (int r = 0; r < blocks; ++r) {
      uint32_t v;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_block(smem_u32(&dead_flag), r)) : "memory");
      lost |= v != 0;
    }
  }
  auto partial = [&](int w, int which, int e) {                 // of warp w of the cluster
    if (blocks == 1) return part[w][which][e][lane];
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(in_block(smem_u32(&part[w % kRowWarps][which][e][lane]), w / kRowWarps)) : "memory");
    return v;
  };
  auto finish = [&]() {
    // the first warp whose share starts inside a tile finishes that tile
    if (lost || u1 == u0 || u0 % units == 0) return;
    const int cut = u0 / units, begin = cut * units;
    int w = mine - 1;
    for (; share(w) > begin; --w)
      if (share(w + 1) > share(w)) return;                      // an earlier warp does
    while (share(w + 1) <= begin) ++w;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = partial(w, 1, e);
    for (++w; w < all_warps && share(w) < begin + units; ++w) {
      if (share(w + 1) == share(w)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += partial(w, 0, e);
    }
    store<T>(p, (t0 + cut) * 16, lane, acc);
  };
  finish();
  if (blocks > 1) {
    __syncwarp();
    sync_cluster();                                             // no block ends while another reads its sums
  }
}

// ------------------------------------------------------------------ launches

// The codes as [N][K / 2] bytes; a box is `rows` features x one unit, lines swizzled over 128 bytes.
bool encode_codes(CUtensorMap* map, const W4Params& p, int rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)p.K / 2, (cuuint64_t)p.N}, strides[1] = {(cuuint64_t)p.K / 2};
  const cuuint32_t box[2] = {kUnit / 2, (cuuint32_t)rows}, ones[2] = {1, 1};
  const EncodeTiledFn fn = encode_tiled();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.q), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kGroup>
cudaError_t launch_rows(const W4Params& p, int dev, cudaStream_t s) {
  const cudaError_t e = allow_shared_memory<w4_rows_kernel<T, kGroup>>(dev);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  if (!encode_codes(&map, p, 16)) return cudaErrorInvalidValue;
  const int smem = 1024 + kRowWarps * kRowStages * kRowBytes + p.M * x_pitch(p.K);
  const int tiles = (p.N + 15) / 16, most = 2 * sm_count(dev), units = (p.K + kRowUnit - 1) / kRowUnit;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  cfg.attrs = &a;
  // Blocks to a cluster: the fewest units in a block's share, a join of a cluster counted as kRowJoin of them (one token, 10007
  // features: 16384 elements 32.9 us in clusters, 41.6 without; 5120 elements 13.0 and 12.0). Only where there are more tiles than
  // blocks: with fewer, each tile's block brings in the token for itself, which more blocks repeat (1000 features x 16384: 12.8 us in
  // clusters, 9.2 without; x 5120 5.6 and 5.7; 2560 x 16384 13.9 and 13.3).
  // (How many clusters fit is asked once: registers and shared memory leave two blocks an SM for every window of this kernel.)
  int blocks = 1, many = tiles < most ? tiles : most, best = (tiles + many - 1) / many * units;
  for (int n = 2; n <= kMostCluster && tiles > most; n *= 2) {
    a.val.clusterDim.x = n;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)n);
    const int fit = clusters<w4_rows_kernel<T, kGroup>>(cfg, n, dev);
    if (fit < 1) continue;
    const int cost = ((tiles + fit - 1) / fit * units + n - 1) / n + kRowJoin;
    if (cost < best) {
      best = cost;
      blocks = n;
      many = fit;
    }
  }
  a.val.clusterDim.x = blocks;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)(blocks * many));
  return cudaLaunchKernelEx(&cfg, w4_rows_kernel<T, kGroup>, p, map, tiles, blocks);
}

// Up to 8 tokens whose elements leave two blocks a SM's shared memory: the rows' kernel (157184 features x 2560, one token: 43 us, on
// tcgen05 51; 8 tokens x 2048: 38 and 43; 4000 features x 4096, 4 tokens: 7.8 and 7.9). 8 tokens x 2560 elements do not fit.
constexpr bool fits_rows(int M, int64_t K) { return M <= 8 && K <= kRowMaxX / 2 && M * x_pitch((int)K) <= kRowMaxX; }
// (a K that is compared as it is: tokens of 2^28 elements and more pass 32 bits in bytes)
static_assert(fits_rows(1, 17920) && !fits_rows(1, 17952) && fits_rows(8, 2048) && !fits_rows(8, 2560));
static_assert(!fits_rows(8, 1 << 28) && !fits_rows(4, 1 << 29) && !fits_rows(1, 1 << 30) && !fits_rows(2, 1 << 30) && !fits_rows(1, 0x7fffff00));

template <typename T, int kGroup>
cudaError_t launch(const W4Params& p, int dev, cudaStream_t s) {
  if (fits_rows(p.M, p.K)) return launch_rows<T, kGroup>(p, dev, s);
  CUtensorMap map;
  if (!encode_codes(&map, p, kTensorRows)) return cudaErrorInvalidValue;
  return launch_w4_tensor(p, map, std::is_same<T, __nv_bfloat16>::value, kGroup, dev, s);
}
template <typename T>
cudaError_t launch(const W4Params& p, int group, int dev, cudaStream_t s) {
  return group == 32 ? launch<T, 32>(p, dev, s) : (group == 64 ? launch<T, 64>(p, dev, s) : launch<T, 128>(p, dev, s));
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" mdw_status w4_linear(const mdw_w4_weights* w, int32_t M, const void* x, int64_t ldx, void* y,
                                int64_t ldy, int32_t y_dtype, const void* bias, const void* residual,
                                int64_t ldr, uint32_t* status, mdw_stream_t stream) {
  if (!w) return MDW_ERR_INVALID_ARG;
  if (w->magic != MDW_MAGIC || w->fmt != MDW_FMT_INT4_GROUP) return MDW_ERR_FORMAT_MISMATCH;
  if (w->dtype != MDW_DT_BF16 && w->dtype != MDW_DT_F16) return MDW_ERR_FORMAT_MISMATCH;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MDW_ERR_UNSUPPORTED_SHAPE;
  // (rows of a tile past n are int32, and so are elements of a unit past k)
  if (w->n < 1 || w->n > 0x7fffff00 || w->k < w->group || w->k > 0x7fffff00 || w->k % w->group != 0) return MDW_ERR_UNSUPPORTED_SHAPE;
  if (M < 1 || M > MDW_MAX_M) return MDW_ERR_INVALID_ARG;
  if (!aligned_to(w->q, 16) || !aligned_to(w->scale, 16) || !null_or_aligned(w->zero, 16) || !aligned_to(x, 16) || !row_stride_ok(ldx, w->k))
    return MDW_ERR_INVALID_ARG;
  if (y_dtype != w->dtype && y_dtype != MDW_DT_F32) return MDW_ERR_FORMAT_MISMATCH;
  if (!aligned_to(y, y_dtype == MDW_DT_F32 ? 4 : 2) || ldy < w->n || !null_or_aligned(bias, 2) ||
      !null_or_aligned(residual, 2) || (residual && ldr < w->n) || !null_or_aligned(status, 4))
    return MDW_ERR_INVALID_ARG;
  const int dev = current_device(), sms = sm_count(dev);
  if (sms <= 0) return MDW_ERR_CUDA;
  // units of one block's share of the tiles stay far below 2^31
  if ((int64_t)((w->n + 15) / 16 / sms + 1) * (w->k / kRowUnit + 1) > 1 << 28) return MDW_ERR_UNSUPPORTED_SHAPE;
  const W4Params p{static_cast<const uint8_t*>(w->q), w->scale, static_cast<const uint8_t*>(w->zero), x, y, bias,
                   residual, ldx, ldy, ldr, status, mdw_spin_budget(), M, w->n, w->k, y_dtype == MDW_DT_F32};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = w->dtype == MDW_DT_BF16 ? launch<__nv_bfloat16>(p, w->group, dev, s) : launch<__half>(p, w->group, dev, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
