// mdw_block_norm: what stands between two sub-layers, one pass over the rows.
//
// Mathematics. z = y / sqrt(mean(y^2) + eps) * post_w, gated; sum = residual_scale * residual + branch_scale * z; x = sum / sqrt(mean
// (sum^2) + eps) * pre_w of the sum as it is stored. Everything is fp32 between the loads and the stores.
//
// What bounds it is memory for many rows and the two chains load - sum - exchange for few. A row lies in the
// registers of its threads, eight neighbouring elements (16 or 32 bytes of a load) at a time, so it is read once; the norms are
// sums over the row's warps. Rows that are not on 16-byte boundaries are read by the aligned pieces around them and shifted in registers.
// Measured: 16,381 rows of 2,560 elements with an fp32 residual 76 us (6.6 TB/s), gated norms of 4,099 rows of 32 heads 23 us (4.4
// TB/s: there the conversions and sigmoids take 70 % of the issue slots).
#include <cmath>
#include <type_traits>

#include "mdw_attn.cuh"

namespace mdw {
namespace {

static_assert(MDW_MAX_NORM_WIDTH <= 2 * 8 * 1024, "");

struct NormParams {
  const void *y, *post_w, *gate, *residual, *pre_w;
  void *sum, *x;
  int64_t ldy, ldg, ldr, lds, ldx;
  float branch_scale, residual_scale, eps, inv_group, inv_width;
  int T, width, group, gate_kind, threads;                      // threads of a row
};

__device__ __forceinline__ void load16_if(uint4& v, const void* src, bool wanted) {
  asm volatile("{ .reg .pred p; setp.ne.b32 p, %5, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0; @p ld.global.v4.b32 {%0,%1,%2,%3}, [%4]; }"
               : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(src), "r"((int)wanted));
}
// Words moved towards the first one, by `halves` half words (below 16).
template <int kWords> __device__ __forceinline__ void shift_words(uint32_t (&w)[kWords], int halves) {
#pragma unroll
  for (int n = 4; n >= 1; n >>= 1)
    if (halves & 2 * n)
#pragma unroll
      for (int i = 0; i + n < kWords; ++i) w[i] = w[i + n];
  if (halves & 1)
#pragma unroll
    for (int i = 0; i + 1 < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
}

// Eight elements of a row, element `at` (a multiple of 8) and on, as they lie in memory; zeros where there are none. Rows that do not lie on
// 16-byte boundaries are read by the 16-byte pieces around the elements, which may reach into the rows beside them, and shifted. Only the
// ends of the whole array (`total` elements) are read by elements: waiting for those of every row took three times as long.
template <typename T, bool kAligned> struct Raw {
  static constexpr int kLoads = sizeof(T) / 2 + (kAligned ? 0 : 1), kPer = 16 / sizeof(T);
  uint4 v[kLoads];
  int off, left;                                                // elements before the first one, and of the row from it on
  __device__ __forceinline__ void ask(const void* p, int64_t base, int at, int width, int64_t total, bool wanted) {
    const T* src = static_cast<const T*>(p) + base + at;
    off = 0;
    if constexpr (kAligned) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load16_if(v[i], src + i * kPer, wanted);
    } else {
      if (wanted) off = (int)(reinterpret_cast<uintptr_t>(src) & 15) / (int)sizeof(T);
      const int reach = off ? kLoads * kPer - off : 8;
      const bool inside = wanted && base + at >= off && base + at + reach <= total;
      left = wanted ? width - at : 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) load16_if(v[i], src - off + i * kPer, inside && (i + 1 < kLoads || off));
      if (wanted && !inside) {
        T e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = at + j < width ? src[j] : T(0.f);
        memcpy(v, e, sizeof e);
        off = 0;
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    uint32_t w[4 * kLoads];
    memcpy(w, v, sizeof w);
    if constexpr (!kAligned)
      if (off) shift_words(w, off * (int)sizeof(T) / 2);
    T e[8];
    memcpy(e, w, sizeof e);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = Elem<T>::to_float(e[i]);
    if constexpr (!kAligned)
      if (left < 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < left ? f[i] : 0.f;
  }
};

// Stores the row's elements at .. at + 7 (those below width) of every lane of a warp; neighbouring lanes have neighbouring ones. Rows that do not
// lie on 16-byte boundaries: a lane takes over the last elements of the lane before it and writes whole 16-byte pieces; what no lane
// takes over is written by elements.
template <typename T, bool kAligned> __device__ __forceinline__ void store_row(void* p, int64_t base, int at, int width, bool wanted, const float (&f)[8]) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = Elem<T>::from_float(f[i]);
  T* dst = static_cast<T*>(p) + base + at;
  constexpr int kPer = 16 / sizeof(T), kPiecesOf8 = 8 / kPer, kWords = 2 * sizeof(T);
  if constexpr (kAligned) {
    uint4 x[kPiecesOf8];
    memcpy(x, e, sizeof e);
    if (wanted)
#pragma unroll
      for (int i = 0; i < kPiecesOf8; ++i) reinterpret_cast<uint4*>(dst)[i] = x[i];
  } else {
    const int off = (int)(reinterpret_cast<uintptr_t>(dst) & 15) / (int)sizeof(T), lane = threadIdx.x & 31, count = wanted ? min(width - at, 8) : 0;
    uint32_t w[4 + kWords];                                     // the last 16 bytes of the lane before, then the lane's own
    memcpy(w + 4, e, sizeof e);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[kWords + i], 1);
    shift_words(w, (kPer - off) * (int)sizeof(T) / 2);          // (off = 0: by 16 bytes, so that only the lane's own are left)
#pragma unroll
    for (int i = 0; i < kPiecesOf8; ++i) {
      // elements i kPer - off .. + kPer - 1 of the lane's
      const bool whole = count >= (i + 1) * kPer - off && (i > 0 || off == 0 || (lane > 0 && at > 0));
      if (whole) reinterpret_cast<uint4*>(dst - off)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < count && j >= i * kPer - off && j < (i + 1) * kPer - off) dst[j] = e[j];
    }
    // the last ones, if the next lane does not take them over
    if (off != 0 && !(lane < 31 && width - at - 8 >= kPer - off))
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < count && j >= 8 - off) dst[j] = e[j];
  }
}

// 0 below 2^-126. The exponential and the reciprocal take one instruction each (with the library's the gated norm of 4,099 rows of 32
// heads took 39 us) and are off by 2^-22 and 2^-23; the rounding of x log2(e) adds |x| 2^-25, 2^-18.5 at -80, to what is stored in 16 bits. Sums
// in fp32 (kFine) take what it left along: e^(-x) = 2^h e^(rest), rest below 2^-17.
template <bool kFine> __device__ __forceinline__ float sigmoid(float x) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLn2 = 0.6931471805599453f;   // log2(e) = this + 1.9259629...e-8
  float e, r;
  if (kFine) {                                                  // (so that the exponential is finite; the sigmoid is 0 or 1 there; NaN stays)
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(-88.f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(88.f));
  }
  const float h = x * -kLog2e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h));
  if (kFine) e = fmaf(e, fmaf(fmaf(x, -kLog2e, -h), kLn2, x * (-1.92596303339e-8f * kLn2)), e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// Pieces of a thread: two above 256 elements, as more rows are on their way then (16,381 rows of 2,560 elements: 69 us, one piece 83; 256
// elements: 18 and 16). Rows off 16-byte boundaries take more registers a piece and are spread over more threads, up to 8,192 elements one
// piece each (16,381 rows of 2,563 elements: two pieces 195 us, one 144).
constexpr int kMaxThreads = 1024;
// Registers: 64, or 56 for one piece off 16-byte boundaries, so that one more block fits an SM (fp32 y, f16 residual: 4,617 rows of 4,374 elements 105
// and 75 us, 16,381 of 2,563 204 and 173, 7,000 of 6,001 214 and 222; with 48: 77, 179, 235). 56 spill 60 bytes a thread where y and the sum are
// fp32, and two pieces off boundaries, above 8,192 elements, spill 340 to 720.
constexpr int registers_of(bool vector, int pieces) { return vector || pieces == 2 ? 64 : 56; }

// T: the 16-bit type; Y, S: types of y and of residual and sum. kPieces of eight elements a thread. kVector: all rows on 16-byte
// boundaries, and whole pieces.
template <typename T, typename Y, typename S, int kPieces, bool kVector>
__global__ void __maxnreg__(registers_of(kVector, kPieces)) norm_kernel(const NormParams p) {
  __shared__ float part[2][32];
  const int row = blockIdx.x * (blockDim.x / p.threads) + threadIdx.x / p.threads, tid = threadIdx.x % p.threads;
  const bool live = row < p.T;                                  // (rows share a block only where a row is a warp's)
  auto place = [&](int i) { return (i * p.threads + tid) * 8; };   // first element of piece i
  auto has = [&](int i) { return live && place(i) < p.width; };
  // sum over the threads of a row
  auto over_row = [&](float v, int which) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (p.threads > 32) {
      if ((threadIdx.x & 31) == 0) part[which][threadIdx.x >> 5] = v;
      __syncthreads();
      const int warps = p.threads >> 5;
      v = (threadIdx.x & 31) < warps ? part[which][threadIdx.x & 31] : 0.f;
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    }
    return v;
  };

  // Everything a row needs is asked for at once, by loads under a predicate (a branch around some of them would wait for the others), and
  // unpacked when it is used.
  float z[kPieces][8];
  Raw<Y, kVector> y[kPieces];
  Raw<S, kVector> r[kPieces];
  Raw<T, kVector> gate[kPieces], weight[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = place(i);
    const bool in = has(i);
    y[i].ask(p.y, row * p.ldy, at, p.width, (p.T - 1) * p.ldy + p.width, in);
    r[i].ask(p.residual, row * p.ldr, at, p.width, (p.T - 1) * p.ldr + p.width, in && p.residual != nullptr);
    gate[i].ask(p.gate, row * p.ldg, at, p.width, (p.T - 1) * p.ldg + p.width, in && p.gate != nullptr);
    if (p.group == p.width) weight[i].ask(p.post_w, 0, at, p.width, p.width, in && p.post_w != nullptr);
    else weight[i].ask(p.post_w, 0, at & (p.group - 1), p.group, p.group, in && p.post_w != nullptr);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) y[i].get(z[i]);
  if (p.post_w) {
    float f[kPieces];
    if (p.group == p.width) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(z[i][j], z[i][j], ss);
      const float all = rsqrtf(over_row(ss, 0) * p.inv_group + p.eps);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) f[i] = all;
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {                       // 8 or 16 neighbouring lanes hold a group
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(z[i][j], z[i][j], ss);
        for (int m = 1; m < p.group / 8; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        f[i] = rsqrtf(ss * p.inv_group + p.eps);
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float w[8];
      weight[i].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] *= f[i] * w[j];
    }
  }
  if (p.gate_kind != MDW_GATE_NONE)
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float g[8];
      gate[i].get(g);
      if (p.gate_kind != MDW_GATE_MUL)                          // (first: times the gate alone could overflow)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] *= sigmoid<sizeof(S) == 4>(g[j]);
      if (p.gate_kind != MDW_GATE_SIGMOID)
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] *= g[j];
    }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[i][j] *= p.branch_scale;
    if (p.residual) {
      float old[8];
      r[i].get(old);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = fmaf(p.residual_scale, old[j], z[i][j]);
    }
    if (p.x)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[i][j] = Elem<S>::to_float(Elem<S>::from_float(z[i][j]));
        ss = fmaf(z[i][j], z[i][j], ss);
      }
    if (p.sum) store_row<S, kVector>(p.sum, row * p.lds, place(i), p.width, has(i), z[i]);
  }
  if (!p.x) return;
  Raw<T, kVector> pre[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) pre[i].ask(p.pre_w, 0, place(i), p.width, p.width, has(i));
  const float f = rsqrtf(over_row(ss, 1) * p.inv_width + p.eps);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    float w[8];
    pre[i].get(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= z[i][j] * f;
    store_row<T, kVector>(p.x, row * p.ldx, place(i), p.width, has(i), w);
  }
}

template <typename T, typename Y, typename S, bool kVector>
cudaError_t launch(const NormParams& p0, cudaStream_t s) {
  NormParams p = p0;
  const int vectors = (p.width + 7) / 8;
  const int pieces = vectors <= (kVector ? 32 : kMaxThreads) ? 1 : 2;
  p.threads = ((vectors + pieces - 1) / pieces + 31) / 32 * 32;
  const int rows = p.threads == 32 ? 4 : 1;
  const unsigned blocks = ((unsigned)p.T + rows - 1) / rows;
  const int threads = p.threads * rows;
  if (pieces == 1) norm_kernel<T, Y, S, 1, kVector><<<blocks, threads, 0, s>>>(p);
  else norm_kernel<T, Y, S, 2, kVector><<<blocks, threads, 0, s>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch(const NormParams& p, bool y32, bool s32, bool vector, cudaStream_t s) {
  if (vector) {
    if (y32) return s32 ? launch<T, float, float, true>(p, s) : launch<T, float, T, true>(p, s);
    return s32 ? launch<T, T, float, true>(p, s) : launch<T, T, T, true>(p, s);
  }
  if (y32) return s32 ? launch<T, float, float, false>(p, s) : launch<T, float, T, false>(p, s);
  return s32 ? launch<T, T, float, false>(p, s) : launch<T, T, T, false>(p, s);
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" mdw_status mdw_block_norm(int32_t T, int32_t width, int32_t dtype, const void* y, int64_t ldy, int32_t y_dtype,
                                     const void* post_w, int32_t group, const void* gate, int64_t ldg, int32_t gate_kind,
                                     float branch_scale, const void* residual, int64_t ldr, float residual_scale,
                                     void* sum, int64_t lds, int32_t sum_dtype, const void* pre_w, void* x, int64_t ldx,
                                     float eps, mdw_stream_t stream) {
  if (dtype != MDW_DT_BF16 && dtype != MDW_DT_F16) return MDW_ERR_FORMAT_MISMATCH;
  if ((y_dtype != dtype && y_dtype != MDW_DT_F32) || (sum_dtype != dtype && sum_dtype != MDW_DT_F32)) return MDW_ERR_FORMAT_MISMATCH;
  if (T < 1 || width < 1) return MDW_ERR_INVALID_ARG;
  if (width > MDW_MAX_NORM_WIDTH) return MDW_ERR_UNSUPPORTED_SHAPE;
  if (group != width && ((group != 64 && group != 128) || width % group != 0)) return MDW_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t ye = y_dtype == MDW_DT_F32 ? 4 : 2, se = sum_dtype == MDW_DT_F32 ? 4 : 2;
  if (!aligned_to(y, ye) || ldy < width || !null_or_aligned(post_w, 2) || !null_or_aligned(gate, 2) || (gate && ldg != 0 && ldg < width) ||
      gate_kind < MDW_GATE_NONE || gate_kind > MDW_GATE_SILU || (gate == nullptr) != (gate_kind == MDW_GATE_NONE) ||
      !null_or_aligned(residual, se) || (residual && ldr < width) || !null_or_aligned(sum, se) || (sum && lds < width) ||
      !null_or_aligned(pre_w, 2) || !null_or_aligned(x, 2) || (x && ldx < width) || (pre_w == nullptr) != (x == nullptr) || (!sum && !x))
    return MDW_ERR_INVALID_ARG;
  if (!std::isfinite(branch_scale) || !std::isfinite(residual_scale) || !(eps > 0.f) || !std::isfinite(eps)) return MDW_ERR_INVALID_ARG;
  auto row_ok = [](const void* q, int64_t ld, uintptr_t e) { return q == nullptr || (aligned_to(q, 16) && ld * e % 16 == 0); };
  const bool vector = width % 8 == 0 && row_ok(y, ldy, ye) && row_ok(post_w, 0, 2) && row_ok(gate, ldg, 2) && row_ok(residual, ldr, se) &&
                      row_ok(sum, lds, se) && row_ok(pre_w, 0, 2) && row_ok(x, ldx, 2);
  const NormParams p{y, post_w, gate, residual, pre_w, sum, x, ldy, ldg, ldr, lds, ldx, branch_scale, residual_scale, eps, 1.f / (float)group,
               1.f / (float)width, T, width, group, gate_kind, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MDW_DT_BF16 ? launch<__nv_bfloat16>(p, y_dtype == MDW_DT_F32, sum_dtype == MDW_DT_F32, vector, s)
                                             : launch<__half>(p, y_dtype == MDW_DT_F32, sum_dtype == MDW_DT_F32, vector, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
