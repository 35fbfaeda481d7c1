// w4_linear: y = x . W^T (+ bias) (+ residual) with W in int4 codes and group scales, for windows of
// up to MDW_MAX_M tokens.
#include <cstring>

#include "mdw_attn.cuh"
#include "mdw_internal.h"

namespace mdw {
namespace {

struct W4Params {
  const uint8_t* q;
  const void* scale;
  const uint8_t* zero;
  const void* x;
  void* y;
  const void* bias;
  const void* residual;
  int64_t ldx, ldy, ldr;
  int M, N, K, y_f32, sms;
};

// ------------------------------------------------------------------ the matrix step
//
// y = W x^T on m16n8k16: 16 features are the rows, 8 tokens the columns. A lane (g, q) holds the codes of
// features g and g + 8; of every 32-code block it takes word q (8 codes, k = 8 q .. 8 q + 7), so all four
// lanes of a product stay inside one group. Masking a word by 0x000f000f leaves the codes j and
// j + 4 of it in the two halves, under the exponent of 128 (bf16) or 1024 (f16) that is code + 128 or
// + 1024 exactly; subtracting 128 + zero leaves code - zero, exact. The token's elements are
// paired the same way. Groups are summed apart in fp32 and enter the result times their scale.

template <typename T> struct Int4;
template <> struct Int4<__nv_bfloat16> {
  // z2: 128 + zero in both halves
  static __device__ __forceinline__ uint32_t zero2(uint32_t z) { return (0x4300u + z) * 0x00010001u; }
  static __device__ __forceinline__ uint32_t sub(uint32_t v, uint32_t z2) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(z2));
    return r;
  }
  static __device__ __forceinline__ void expand(uint32_t w, uint32_t z2, uint32_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = sub(((w >> (4 * i)) & 0x000f000fu) | 0x43004300u, z2);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
template <> struct Int4<__half> {
  // low half: 1024 + zero; the odd codes stay in their upper nibble as 1024 + 16 code and are brought
  // down by one exact multiply-add: (1024 + 16 code) / 16 - (64 + zero)
  static __device__ __forceinline__ uint32_t zero2(uint32_t z) { return (0x6400u + z) * 0x00010001u; }
  static __device__ __forceinline__ void expand(uint32_t w, uint32_t z2, uint32_t (&p)[4]) {
    // -(64 + zero) in f16: 0xd400 is -64, whose unit in the last place is 1 / 16
    const uint32_t nz = 0xd400d400u + ((z2 & 0x000f000fu) << 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w >> (8 * i), lo = (v & 0x000f000fu) | 0x64006400u, hi = (v & 0x00f000f0u) | 0x64006400u;
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * i]) : "r"(lo), "r"(z2));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[2 * i + 1]) : "r"(hi), "r"(0x2c002c00u), "r"(nz));
    }
  }
  static __device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
template <typename T>
__device__ __forceinline__ float lds_elem(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  T t;
  memcpy(&t, &v, 2);
  return Elem<T>::to_float(t);
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// A stage of 16 features x kU codes: code rows of kU / 2 bytes, 16 bytes apart more so that the eight
// features of a load fall on different banks; the scales and zeros as the 4-byte words that cover
// them (a row of an odd number of groups starts inside a word).
template <int kU, int kGroup>
struct Unit {
  static constexpr int kGroups = kU / kGroup;
  static constexpr int kCodePitch = kU / 2 + 16;
  static constexpr int kScaleWords = kGroups / 2 + 1, kZeroWords = (kGroups + 6) / 4;
  static constexpr int kXPitch = 2 * kU + 64;                   // two tokens of a 16-byte load on different banks
  static __host__ __device__ constexpr int scales(int rows) { return rows * kCodePitch; }
  static __host__ __device__ constexpr int zeros(int rows) { return scales(rows) + rows * kScaleWords * 4; }
  static __host__ __device__ constexpr int tokens(int rows) { return (zeros(rows) + rows * kZeroWords * 4 + 15) / 16 * 16; }
  static __host__ __device__ constexpr int bytes(int rows, int m) { return tokens(rows) + m * kXPitch; }
};

// Word window of `count` bytes from byte `at` on: word i starts at (at & ~3) + 4 i; src bytes are cut at `total`.
__device__ __forceinline__ void cp_window(uint32_t dst, const uint8_t* base, int64_t at, int64_t total, int i) {
  const int64_t pos = (at & ~int64_t{3}) + 4 * i;
  const int64_t left = total - pos;
  cp4(dst, base + (left > 0 ? pos : 0), left >= 4 ? 4 : (left > 0 ? (int)left : 0));
}

// Requests rows [n0, n0 + kRows) x codes [k0, k0 + kU) and the tokens' elements there; `id` of `threads`
// takes part. Codes and elements behind K arrive as zeros, rows behind N repeat the last one.
template <typename T, int kU, int kGroup, int kRows>
__device__ __forceinline__ void request(const W4Params& p, uint32_t stage, int n0, int k0, int id, int threads) {
  using U = Unit<kU, kGroup>;
  const int groups = p.K / kGroup;
  constexpr int kPieces = kU / 32;
#pragma unroll
  for (int i = 0; i < kRows * kPieces; i += threads) {
    const int at = i + id;
    if (kRows * kPieces % threads != 0 && at >= kRows * kPieces) break;
    const int row = at / kPieces, piece = at % kPieces, k = k0 + 32 * piece;
    const int n = min(n0 + row, p.N - 1);
    const bool on = k < p.K;
    cp16(stage + row * U::kCodePitch + 16 * piece, p.q + (size_t)n * (p.K / 2) + (on ? k / 2 : 0), on);
  }
  const int64_t group0 = k0 / kGroup;
  for (int at = id; at < kRows * U::kScaleWords; at += threads) {
    const int row = at / U::kScaleWords, i = at - row * U::kScaleWords;
    const int n = min(n0 + row, p.N - 1);
    cp_window(stage + U::scales(kRows) + 4 * at, static_cast<const uint8_t*>(p.scale), ((int64_t)n * groups + group0) * 2,
              (int64_t)p.N * groups * 2, i);
  }
  if (p.zero)
    for (int at = id; at < kRows * U::kZeroWords; at += threads) {
      const int row = at / U::kZeroWords, i = at - row * U::kZeroWords;
      const int n = min(n0 + row, p.N - 1);
      cp_window(stage + U::zeros(kRows) + 4 * at, p.zero, (int64_t)n * groups + group0, (int64_t)p.N * groups, i);
    }
  for (int at = id; at < p.M * (kU / 8); at += threads) {
    const int t = at / (kU / 8), piece = at % (kU / 8), k = k0 + 8 * piece;
    const bool on = k < p.K;
    cp16(stage + U::tokens(kRows) + t * U::kXPitch + 16 * piece, static_cast<const T*>(p.x) + t * p.ldx + (on ? k : 0), on);
  }
}

// The 16 features of a stage from row `row0` on, times kTiles x 8 tokens: acc += scale * (codes - zero) . x.
template <typename T, int kU, int kGroup, int kRows, int kTiles>
__device__ __forceinline__ void multiply(const W4Params& p, uint32_t stage, int n0, int row0, int k0, int lane, float (&acc)[kTiles][4]) {
  using U = Unit<kU, kGroup>;
  const int g = lane >> 2, q = lane & 3, groups = p.K / kGroup, group0 = k0 / kGroup;
  const uint32_t code = stage + (row0 + g) * U::kCodePitch + 4 * q;
  // byte offsets of the two features' first scale and zero in their windows
  uint32_t scale[2], zero[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = row0 + g + 8 * i;
    const uint32_t at = (uint32_t)min(n0 + row, p.N - 1) * (uint32_t)groups + (uint32_t)group0;
    scale[i] = stage + U::scales(kRows) + row * U::kScaleWords * 4 + (at * 2 & 3);
    zero[i] = stage + U::zeros(kRows) + row * U::kZeroWords * 4 + (at & 3);
  }
#pragma unroll
  for (int s = 0; s < U::kGroups; ++s) {
    if (group0 + s >= groups) break;
    const uint32_t z0 = Int4<T>::zero2(p.zero ? lds8(zero[0] + s) : 8u), z1 = Int4<T>::zero2(p.zero ? lds8(zero[1] + s) : 8u);
    float d[kTiles][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) d[t][0] = d[t][1] = d[t][2] = d[t][3] = 0.f;
#pragma unroll
    for (int b = s * (kGroup / 32); b < (s + 1) * (kGroup / 32); ++b) {
      uint32_t lo[4], hi[4];
      Int4<T>::expand(lds32(code + 16 * b), z0, lo);
      Int4<T>::expand(lds32(code + 8 * U::kCodePitch + 16 * b), z1, hi);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (8 * t + g < p.M) x = lds128(stage + U::tokens(kRows) + (8 * t + g) * U::kXPitch + 64 * b + 16 * q);
        Int4<T>::mma(d[t], lo[0], hi[0], lo[1], hi[1], __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
        Int4<T>::mma(d[t], lo[2], hi[2], lo[3], hi[3], __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
      }
    }
    const float s0 = lds_elem<T>(scale[0] + 2 * s), s1 = lds_elem<T>(scale[1] + 2 * s);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      acc[t][0] = fmaf(s0, d[t][0], acc[t][0]);
      acc[t][1] = fmaf(s0, d[t][1], acc[t][1]);
      acc[t][2] = fmaf(s1, d[t][2], acc[t][2]);
      acc[t][3] = fmaf(s1, d[t][3], acc[t][3]);
    }
  }
}

// Features n0 + {g, g + 8}, tokens t0 + 2 q + {0, 1}: bias, residual, one rounding.
template <typename T>
__device__ __forceinline__ void store(const W4Params& p, int n0, int t0, int lane, const float (&acc)[4]) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int n = n0 + g + 8 * (e >> 1), t = t0 + 2 * q + (e & 1);
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
// Bound by the codes' stream. A block owns a contiguous range of 16-feature tiles and cuts its
// (tile, unit of kU codes) sequence into eight equal contiguous shares, one per warp; each warp
// streams its share through a ring of its own, with no barrier until the end. A tile cut between
// warps is finished from their partial sums, in order.
constexpr int kRowWarps = 8;

template <typename T, int kU, int kGroup, int kStages>
__global__ void __launch_bounds__(32 * kRowWarps) w4_rows_kernel(const W4Params p, int tiles) {
  using U = Unit<kU, kGroup>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float part[kRowWarps][2][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = (p.K + kU - 1) / kU;
  const int t0 = (int)((int64_t)tiles * blockIdx.x / gridDim.x), t1 = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  const int all = (t1 - t0) * units;                            // this block's units (the host bounds them)
  const int u0 = (int)((int64_t)all * warp / kRowWarps), u1 = (int)((int64_t)all * (warp + 1) / kRowWarps);
  const int bytes = U::bytes(16, p.M);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kStages * bytes;

  int ask = u0, ask_tile = u0 / units, ask_unit = u0 - ask_tile * units;
  uint32_t to = ring;
  auto next = [&]() {
    if (ask < u1) {
      request<T, kU, kGroup, 16>(p, to, (t0 + ask_tile) * 16, ask_unit * kU, lane, 32);
      ++ask;
      if (++ask_unit == units) { ask_unit = 0; ++ask_tile; }
      to = to + bytes == ring + kStages * bytes ? ring : to + bytes;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kStages - 1; ++i) next();

  int tile = u0 / units, unit = u0 - tile * units;
  bool from_start = unit == 0;
  uint32_t at = ring;
  float acc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
  for (int u = u0; u < u1; ++u) {
    asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 2) : "memory");
    __syncwarp();                                               // all lanes' copies are here, and the oldest stage is read
    next();
    multiply<T, kU, kGroup, 16, 1>(p, at, (t0 + tile) * 16, 0, unit * kU, lane, acc);
    at = at + bytes == ring + kStages * bytes ? ring : at + bytes;
    if (++unit == units || u + 1 == u1) {
      if (from_start && unit == units) {
        store<T>(p, (t0 + tile) * 16, 0, lane, acc[0]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) part[warp][from_start ? 1 : 0][e][lane] = acc[0][e];
      }
      acc[0][0] = acc[0][1] = acc[0][2] = acc[0][3] = 0.f;
      from_start = true;
      if (unit == units) { unit = 0; ++tile; }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // the first warp whose share starts inside a tile finishes that tile
  if (u1 == u0 || u0 % units == 0) return;
  const int cut = u0 / units, begin = cut * units;
  int w = warp - 1;
  while ((int64_t)all * w / kRowWarps > begin) {
    if ((int)((int64_t)all * (w + 1) / kRowWarps) > (int)((int64_t)all * w / kRowWarps)) return;   // an earlier warp does
    --w;
  }
  while ((int)((int64_t)all * (w + 1) / kRowWarps) <= begin) ++w;
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[0][e] = part[w][1][e][lane];
  for (++w; w < kRowWarps; ++w) {
    const int s0 = (int)((int64_t)all * w / kRowWarps), s1 = (int)((int64_t)all * (w + 1) / kRowWarps);
    if (s0 >= begin + units) break;
    if (s1 == s0) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[0][e] += part[w][0][e][lane];
  }
  store<T>(p, (t0 + cut) * 16, 0, lane, acc[0]);
}

// ------------------------------------------------------------------ wider windows
//
// With 9 to 32 tokens the elements of x outweigh the codes of 16 features, so eight warps (128
// features) share them: one stage holds 128 features x 128 codes and the tokens' elements there.
// Where there are few blocks of features, a cluster of blocks splits K and joins the sums
// over distributed shared memory, in rank order.
constexpr int kWideRows = 128, kWideUnit = 128, kWideStages = 4;

template <typename T, int kGroup, int kTiles>
__global__ void __launch_bounds__(256) w4_wide_kernel(const W4Params p, int split) {
  using U = Unit<kWideUnit, kGroup>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split, n0 = blockIdx.x / split * kWideRows;
  const int units = (p.K + kWideUnit - 1) / kWideUnit;
  const int u0 = units * rank / split, u1 = units * (rank + 1) / split;
  const int bytes = U::bytes(kWideRows, p.M);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem);
  float acc[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
  auto ask = [&](int u) {
    if (u < u1) request<T, kWideUnit, kGroup, kWideRows>(p, ring + (u - u0) % kWideStages * bytes, n0, u * kWideUnit, threadIdx.x, 256);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kWideStages - 1; ++i) ask(u0 + i);
  for (int u = u0; u < u1; ++u) {
    asm volatile("cp.async.wait_group %0;" :: "n"(kWideStages - 2) : "memory");
    __syncthreads();
    ask(u + kWideStages - 1);
    multiply<T, kWideUnit, kGroup, kWideRows, kTiles>(p, ring + (u - u0) % kWideStages * bytes, n0, warp * 16, u * kWideUnit, lane, acc);
  }
  if (split == 1) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) store<T>(p, n0 + warp * 16, 8 * t, lane, acc[t]);
    return;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float4* sums = reinterpret_cast<float4*>(smem);
#pragma unroll
  for (int t = 0; t < kTiles; ++t) sums[(warp * kTiles + t) * 32 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int i = rank * 8 + warp; i < 8 * kTiles; i += 8 * split) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < split; ++r) {
      uint32_t a;
      float4 v;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(ring + (i * 32 + lane) * 16), "r"(r));
      asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
      sum[0] += v.x;
      sum[1] += v.y;
      sum[2] += v.z;
      sum[3] += v.w;
    }
    store<T>(p, n0 + i / kTiles * 16, i % kTiles * 8, lane, sum);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ launches

template <typename K>
cudaError_t allow_smem(K kernel, int bytes) {
  return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) : cudaSuccess;
}

template <typename T, int kU, int kGroup, int kStages>
cudaError_t launch_rows(const W4Params& p, cudaStream_t s) {
  const int tiles = (p.N + 15) / 16, smem = kRowWarps * kStages * Unit<kU, kGroup>::bytes(16, p.M);
  const cudaError_t e = allow_smem(w4_rows_kernel<T, kU, kGroup, kStages>, smem);
  if (e != cudaSuccess) return e;
  const int grid = tiles < 2 * p.sms ? tiles : 2 * p.sms;
  w4_rows_kernel<T, kU, kGroup, kStages><<<grid, 32 * kRowWarps, smem, s>>>(p, tiles);
  return cudaGetLastError();
}

template <typename T, int kGroup, int kTiles>
cudaError_t launch_wide(const W4Params& p, cudaStream_t s) {
  const int blocks = (p.N + kWideRows - 1) / kWideRows, units = (p.K + kWideUnit - 1) / kWideUnit;
  int split = 1;
  while (split < 8 && blocks * split < p.sms && units >= 4 * split) split *= 2;
  const int ring = kWideStages * Unit<kWideUnit, kGroup>::bytes(kWideRows, p.M), sums = 8 * kTiles * 32 * 16;
  const int smem = ring > sums ? ring : sums;
  cudaError_t e = allow_smem(w4_wide_kernel<T, kGroup, kTiles>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * split));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = split;
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4_wide_kernel<T, kGroup, kTiles>, p, split);
}

template <typename T, int kGroup>
cudaError_t launch(const W4Params& p, cudaStream_t s) {
  if (p.M == 1) return launch_rows<T, 256, kGroup, 4>(p, s);
  if (p.M == 2) return launch_rows<T, 256, kGroup, 3>(p, s);
  if (p.M <= 4) return launch_rows<T, 128, kGroup, 4>(p, s);
  if (p.M <= 8) return launch_rows<T, 128, kGroup, 3>(p, s);
  return p.M <= 16 ? launch_wide<T, kGroup, 2>(p, s) : launch_wide<T, kGroup, 4>(p, s);
}
template <typename T>
cudaError_t launch(const W4Params& p, int group, cudaStream_t s) {
  return group == 32 ? launch<T, 32>(p, s) : (group == 64 ? launch<T, 64>(p, s) : launch<T, 128>(p, s));
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" mdw_status w4_linear(const mdw_w4_weights* w, int32_t M, const void* x, int64_t ldx, void* y,
                                int64_t ldy, int32_t y_dtype, const void* bias, const void* residual,
                                int64_t ldr, mdw_stream_t stream) {
  if (!w) return MDW_ERR_INVALID_ARG;
  if (w->magic != MDW_MAGIC || w->fmt != MDW_FMT_INT4_GROUP) return MDW_ERR_FORMAT_MISMATCH;
  if (w->dtype != MDW_DT_BF16 && w->dtype != MDW_DT_F16) return MDW_ERR_FORMAT_MISMATCH;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MDW_ERR_UNSUPPORTED_SHAPE;
  if (w->n < 1 || w->k < w->group || w->k % w->group != 0) return MDW_ERR_UNSUPPORTED_SHAPE;
  if (M < 1 || M > MDW_MAX_M) return MDW_ERR_INVALID_ARG;
  if (!aligned_to(w->q, 16) || !aligned_to(w->scale, 16) || !null_or_aligned(w->zero, 16) || !aligned_to(x, 16) || !row_stride_ok(ldx, w->k))
    return MDW_ERR_INVALID_ARG;
  if (y_dtype != w->dtype && y_dtype != MDW_DT_F32) return MDW_ERR_FORMAT_MISMATCH;
  if (!aligned_to(y, y_dtype == MDW_DT_F32 ? 4 : 2) || ldy < w->n || !null_or_aligned(bias, 2) ||
      !null_or_aligned(residual, 2) || (residual && ldr < w->n))
    return MDW_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return MDW_ERR_CUDA;
  // units of one block's share of the tiles stay far below 2^31
  if ((int64_t)((w->n + 15) / 16 / sms + 1) * (w->k / 128 + 1) > 1 << 28) return MDW_ERR_UNSUPPORTED_SHAPE;
  const W4Params p{static_cast<const uint8_t*>(w->q), w->scale, static_cast<const uint8_t*>(w->zero), x, y, bias,
                   residual, ldx, ldy, ldr, M, w->n, w->k, y_dtype == MDW_DT_F32, sms};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = w->dtype == MDW_DT_BF16 ? launch<__nv_bfloat16>(p, w->group, s) : launch<__half>(p, w->group, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
