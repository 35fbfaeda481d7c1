// Shared by the attention sub-layer's kernels (w4_linear, mdw_kv_plan, mdw_kv_write,
// mdw_tree_attention): 16-bit element types, the caller's status word and host-side checks.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

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

// ------------------------------------------------------------------ asynchronous copies

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
// Makes the initialised barriers visible to the copy engine.
__device__ __forceinline__ void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Brings a copy's descriptor in before the first copy needs it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) { asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory"); }
// A wait that outlasts the budget marks the block dead: it and every later wait then give up at
// once, so the block runs to its end (its results are not stored) and the status says so.
static __device__ __noinline__ void mbar_wait_slow(uint32_t bar, uint32_t parity, long long budget, uint32_t* status, volatile int* dead) {
  const long long t0 = clock64();
  for (;;) {
    if (*dead) return;
    if (clock64() - t0 > budget) {
      *dead = 1;
      raise_status(status, MDW_ERR_TIMEOUT);
      return;
    }
    if (mbar_try(bar, parity)) return;
  }
}
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, long long budget, uint32_t* status, volatile int* dead) {
  if (!mbar_test(bar, parity)) mbar_wait_slow(bar, parity, budget, status, dead);
}
// Waits for a copy's arrival whether or not the block is dead (bounded as well): a block does not end before its copies, which
// would write into the shared memory of the one that follows.
__device__ __forceinline__ void mbar_drain_inline(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity) && clock64() - t0 < (1ll << 28)) {}
}
static __device__ __noinline__ void mbar_drain(uint32_t bar, uint32_t parity) { mbar_drain_inline(bar, parity); }

// ------------------------------------------------------------------ host

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled of the driver (the library does not link against it); null without one.
inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) != cudaSuccess) f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

constexpr int kMaxDevices = 64;
inline int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices ? dev : -1;
}
// SM count of a device, asked once; 0 without one.
inline int sm_count(int dev) {
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}
// Lets a kernel use the whole shared memory of an SM, once per device.
template <auto kKernel>
cudaError_t allow_shared_memory(int dev) {
  static std::atomic<bool> done[kMaxDevices];
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, kKernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - (int)a.sharedSizeBytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline bool null_or_aligned(const void* p, uintptr_t a) { return p == nullptr || aligned_to(p, a); }
// A row stride in 16-bit elements that keeps every row on a 16-byte boundary.
inline bool row_stride_ok(int64_t ld, int64_t width) { return ld >= width && ld % 8 == 0; }
inline int log2_of(int32_t pow2) { return __builtin_ctz((unsigned)pow2); }

mdw_status check_kv_cache(const mdw_kv_cache* c);

}  // namespace mdw
