// w4_linear: y = x . W^T (+ bias) (+ residual) with W in int4 codes and group scales, for windows of
// up to MDW_MAX_M tokens.
#include "mdw_attn.cuh"

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
  int M, N, K, group;
};

// One warp per (row, token); each lane takes the 32 codes of one 16-byte block at a time.
template <typename T, typename Y>
__global__ void __launch_bounds__(256) w4_kernel(W4Params p) {
  const int lane = threadIdx.x & 31, n = blockIdx.x * 8 + (threadIdx.x >> 5), t = blockIdx.y;
  if (n >= p.N) return;
  const int groups = p.K / p.group;
  const T* x = static_cast<const T*>(p.x) + t * p.ldx;
  float sum = 0.f;
  for (int b = lane; b < p.K / 32; b += 32) {
    const uint4 v = *reinterpret_cast<const uint4*>(p.q + (size_t)n * (p.K / 2) + 16 * b);
    const int g = b * 32 / p.group;
    const float z = p.zero ? (float)p.zero[(size_t)n * groups + g] : 8.f;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float part = 0.f;
    for (int i = 0; i < 32; ++i)
      part = fmaf(Elem<T>::to_float(x[32 * b + i]), (float)((w[i >> 3] >> (4 * (i & 7))) & 15u) - z, part);
    sum = fmaf(part, Elem<T>::to_float(static_cast<const T*>(p.scale)[(size_t)n * groups + g]), sum);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane != 0) return;
  if (p.bias) sum += Elem<T>::to_float(static_cast<const T*>(p.bias)[n]);
  if (p.residual) sum += Elem<T>::to_float(static_cast<const T*>(p.residual)[t * p.ldr + n]);
  static_cast<Y*>(p.y)[t * p.ldy + n] = Elem<Y>::from_float(sum);
}

template <typename T, typename Y>
cudaError_t launch(const W4Params& p, cudaStream_t s) {
  w4_kernel<T, Y><<<dim3((p.N + 7) / 8, p.M), 256, 0, s>>>(p);
  return cudaGetLastError();
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
  if (!aligned_to(w->q, 16) || !aligned_to(w->scale, 2) || !aligned_to(x, 16) || !row_stride_ok(ldx, w->k))
    return MDW_ERR_INVALID_ARG;
  if (y_dtype != w->dtype && y_dtype != MDW_DT_F32) return MDW_ERR_FORMAT_MISMATCH;
  if (!aligned_to(y, y_dtype == MDW_DT_F32 ? 4 : 2) || ldy < w->n || !null_or_aligned(bias, 2) ||
      !null_or_aligned(residual, 2) || (residual && ldr < w->n))
    return MDW_ERR_INVALID_ARG;
  W4Params p{static_cast<const uint8_t*>(w->q), w->scale, static_cast<const uint8_t*>(w->zero), x, y, bias,
             residual, ldx, ldy, ldr, M, w->n, w->k, w->group};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = y_dtype == MDW_DT_F32;
  cudaError_t e;
  if (w->dtype == MDW_DT_BF16)
    e = f32 ? launch<__nv_bfloat16, float>(p, s) : launch<__nv_bfloat16, __nv_bfloat16>(p, s);
  else
    e = f32 ? launch<__half, float>(p, s) : launch<__half, __half>(p, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
