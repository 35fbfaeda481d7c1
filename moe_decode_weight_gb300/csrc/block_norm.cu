// mdw_block_norm: what stands between two sub-layers, one pass over the rows.
//
// Mathematics. z = y / sqrt(mean(y^2) + eps) * post_w, gated; sum = residual_scale * residual + branch_scale * z; x = sum / sqrt(mean
// (sum^2) + eps) * pre_w of the sum as it is stored. Everything is fp32 between the loads and the stores.
//
// What bounds it is memory for many rows and the two chains load - sum - exchange for few. A row lies in the
// registers of its threads, eight neighbouring elements (16 or 32 bytes of a load) at a time, so it is read once; the norms are
// sums over the row's warps. Rows that are not on 16-byte boundaries are read and written by elements, neighbouring threads at
// neighbouring ones.
#include <cmath>
#include <type_traits>

#include "mdw_attn.cuh"

namespace mdw {
namespace {

struct NormParams {
  const void *y, *post_w, *gate, *residual, *pre_w;
  void *sum, *x;
  int64_t ldy, ldg, ldr, lds, ldx;
  float branch_scale, residual_scale, eps, inv_group, inv_width;
  int T, width, group, gate_kind, threads;                      // threads of a row
  int scattered;                                                // by elements, neighbouring threads at neighbouring ones
};

// Eight elements as they lie in memory, zeros where they are not asked for.
template <typename T> struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void ask(const void* p, int64_t at, bool wanted) {
    const T* src = static_cast<const T*>(p) + at;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      asm volatile("{ .reg .pred p; setp.ne.b32 p, %5, 0; mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0; @p ld.global.v4.b32 {%0,%1,%2,%3}, [%4]; }"
                   : "=&r"(v[i].x), "=&r"(v[i].y), "=&r"(v[i].z), "=&r"(v[i].w) : "l"(reinterpret_cast<const uint4*>(src) + i), "r"((int)wanted));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    T e[8];
    memcpy(e, v, sizeof e);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = Elem<T>::to_float(e[i]);
  }
};
template <typename T> __device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  const T* src = static_cast<const T*>(p) + at;
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    T e[8];
    memcpy(e, &x, 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::to_float(e[i]);
  }
}
template <typename T> __device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  T* dst = static_cast<T*>(p) + at;
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = Elem<T>::from_float(v[i]);
    uint4 x;
    memcpy(&x, e, 16);
    *reinterpret_cast<uint4*>(dst) = x;
  }
}

// Off by a few 2^-22: the exponential and the reciprocal take one instruction each (with the exact ones the gated norm of 4,099
// rows of 32 heads took 39 us).
__device__ __forceinline__ float sigmoid(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

constexpr int kMaxThreads = 512;

// T: the 16-bit type; Y, S: types of y and of residual and sum. kPieces of eight elements a thread. kVector: by 16 bytes.
template <typename T, typename Y, typename S, int kPieces, bool kVector>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p) {
  __shared__ float part[2][32];
  const int row = blockIdx.x * (blockDim.x / p.threads) + threadIdx.x / p.threads, tid = threadIdx.x % p.threads;
  const bool live = row < p.T;                                  // (rows share a block only where a row is a warp's)
  auto place = [&](int i, int j) {                              // of element j of piece i
    return kVector || !p.scattered ? (i * p.threads + tid) * 8 + j : (i * 8 + j) * p.threads + tid;
  };
  auto has = [&](int i, int j) { return live && (kVector ? (i * p.threads + tid) * 8 < p.width : place(i, j) < p.width); };
  auto get = [&](auto type, const void* src, int64_t base, int i, float (&v)[8]) {
    using E = decltype(type);
    if constexpr (kVector) {
      if (has(i, 0)) load8<E>(src, base + place(i, 0), v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(i, j)) v[j] = Elem<E>::to_float(static_cast<const E*>(src)[base + place(i, j)]);
    }
  };
  auto put = [&](auto type, void* dst, int64_t base, int i, const float (&v)[8]) {
    using E = decltype(type);
    if constexpr (kVector) {
      if (has(i, 0)) store8<E>(dst, base + place(i, 0), v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(i, j)) static_cast<E*>(dst)[base + place(i, j)] = Elem<E>::from_float(v[j]);
    }
  };
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
  Raw<Y> y_raw[kVector ? kPieces : 1];
  Raw<S> r_raw[kVector ? kPieces : 1];
  Raw<T> gate[kVector ? kPieces : 1], weight[kVector ? kPieces : 1];
  if constexpr (kVector) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = place(i, 0);
      const bool in = has(i, 0);
      y_raw[i].ask(p.y, row * p.ldy + at, in);
      r_raw[i].ask(p.residual, row * p.ldr + at, in && p.residual);
      gate[i].ask(p.gate, row * p.ldg + at, in && p.gate);
      weight[i].ask(p.post_w, p.group == p.width ? at : at & (p.group - 1), in && p.post_w);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) y_raw[i].get(z[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
      get(Y(), p.y, row * p.ldy, i, z[i]);
    }
  }
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
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0.f;
      if constexpr (kVector) {
        weight[i].get(w);
      } else if (p.group == p.width) {
        get(T(), p.post_w, 0, i, w);
      } else if (has(i, 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = Elem<T>::to_float(static_cast<const T*>(p.post_w)[(place(i, 0) & (p.group - 1)) + j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] *= f[i] * w[j];
    }
  }
  if (p.gate_kind != MDW_GATE_NONE)
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.f;
      if constexpr (kVector) gate[i].get(g);
      else get(T(), p.gate, row * p.ldg, i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float act = p.gate_kind == MDW_GATE_MUL ? 1.f : sigmoid(g[j]);
        z[i][j] *= p.gate_kind == MDW_GATE_SIGMOID ? act : g[j] * act;
      }
    }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = 0.f;
    if constexpr (kVector) r_raw[i].get(r);
    else if (p.residual) get(S(), p.residual, row * p.ldr, i, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float s = p.branch_scale * z[i][j];
      if (p.residual) s = fmaf(p.residual_scale, r[j], s);
      z[i][j] = p.x ? Elem<S>::to_float(Elem<S>::from_float(s)) : s;
      ss = fmaf(z[i][j], z[i][j], ss);
    }
    if (p.sum) put(S(), p.sum, row * p.lds, i, z[i]);
  }
  if (!p.x) return;
  const float f = rsqrtf(over_row(ss, 1) * p.inv_width + p.eps);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
    get(T(), p.pre_w, 0, i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= z[i][j] * f;
    put(T(), p.x, row * p.ldx, i, w);
  }
}

template <typename T, typename Y, typename S, bool kVector>
cudaError_t launch(const NormParams& p0, cudaStream_t s) {
  NormParams p = p0;
  const int vectors = (p.width + 7) / 8;
  const int pieces = vectors <= 32 ? 1 : vectors <= 2 * kMaxThreads ? 2 : 4;
  p.threads = ((vectors + pieces - 1) / pieces + 31) / 32 * 32;
  const int rows = p.threads == 32 ? 4 : 1;
  const unsigned blocks = (unsigned)((p.T + rows - 1) / rows);
  const int threads = p.threads * rows;
  if (pieces == 1) norm_kernel<T, Y, S, 1, kVector><<<blocks, threads, 0, s>>>(p);
  else if (pieces == 2) norm_kernel<T, Y, S, 2, kVector><<<blocks, threads, 0, s>>>(p);
  else norm_kernel<T, Y, S, 4, kVector><<<blocks, threads, 0, s>>>(p);
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
  NormParams p{y, post_w, gate, residual, pre_w, sum, x, ldy, ldg, ldr, lds, ldx, branch_scale, residual_scale, eps, 1.f / (float)group,
               1.f / (float)width, T, width, group, gate_kind, 0, group == width || !post_w};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MDW_DT_BF16 ? launch<__nv_bfloat16>(p, y_dtype == MDW_DT_F32, sum_dtype == MDW_DT_F32, vector, s)
                                             : launch<__half>(p, y_dtype == MDW_DT_F32, sum_dtype == MDW_DT_F32, vector, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
