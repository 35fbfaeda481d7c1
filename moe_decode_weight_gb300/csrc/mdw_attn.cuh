// Shared by the attention sub-layer's kernels (w4_linear, mdw_kv_plan, mdw_kv_write,
// mdw_tree_attention): 16-bit element types, the caller's status word and host-side checks.
#pragma once

#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "moe_decode_weight.h"

namespace mdw {

// The first bad datum a call meets names the error; the word belongs to the caller.
__device__ __forceinline__ void raise_status(uint32_t* status, mdw_status s) {
  if (status) atomicCAS(status, 0u, (uint32_t)s);
}

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr int32_t kDtype = MDW_DT_BF16;
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
  static constexpr int32_t kDtype = MDW_DT_F16;
  static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
  static constexpr int32_t kDtype = MDW_DT_F32;
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
};

inline bool aligned_to(const void* p, uintptr_t a) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool null_or_aligned(const void* p, uintptr_t a) { return p == nullptr || aligned_to(p, a); }
// A row stride in 16-bit elements that keeps every row on a 16-byte boundary.
inline bool row_stride_ok(int64_t ld, int64_t width) { return ld >= width && ld % 8 == 0; }
inline int log2_of(int32_t pow2) { return __builtin_ctz((unsigned)pow2); }

mdw_status check_kv_cache(const mdw_kv_cache* c);

}  // namespace mdw
