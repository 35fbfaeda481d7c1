// What the kernels of w4_linear share: the call's parameters, the expansion of the codes, small steps.
#pragma once

#include <atomic>
#include <cstring>

#include "mdw_attn.cuh"

namespace mdw {

struct W4Params {
  const uint8_t* q;
  const void* scale;
  const uint8_t* zero;
  const void* x;
  void* y;
  const void* bias;
  const void* residual;
  int64_t ldx, ldy, ldr;
  uint32_t* status;
  long long spin_budget;
  int M, N, K, y_f32;
};

constexpr int kUnit = 256;                     // codes of a feature in one swizzled line of 128 bytes

__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));   // (v & mask) | bits in one operation
  return r;
}

template <typename T> struct Int4;
template <> struct Int4<__nv_bfloat16> {
  // The numbers up to 255 * 2^-133, subnormal and the first normal ones, are the integers times 2^-133: a code in the low
  // nibble of a half is one, a code in the next nibble 16 times one. A product with 2^127 (2^123), with the zero
  // taken out by the same operation, makes them (code - zero) * 2^-6 exactly; kFactor goes into the scale.
  static constexpr float kFactor = 64.f;
  static __device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
  }
  static __device__ __forceinline__ uint32_t zero2(uint32_t z) { return fma2(z * 0x00010001u, 0xff00ff00u, 0u); }   // -zero * 2^-6
  static __device__ __forceinline__ void expand(uint32_t w, uint32_t z2, uint32_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w >> (8 * i);
      p[2 * i] = fma2(v & 0x000f000fu, 0x7f007f00u, z2);
      p[2 * i + 1] = fma2(v & 0x00f000f0u, 0x7d007d00u, z2);
    }
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  }
};
template <> struct Int4<__half> {
  static constexpr float kFactor = 1.f;
  // low half: 1024 + zero; the odd codes stay in their upper nibble as 1024 + 16 code and are brought
  // down by one exact multiply-add: (1024 + 16 code) / 16 - (64 + zero)
  static __device__ __forceinline__ uint32_t zero2(uint32_t z) { return (0x6400u + z) * 0x00010001u; }
  static __device__ __forceinline__ void expand(uint32_t w, uint32_t z2, uint32_t (&p)[4]) {
    uint32_t nz;                                                // 960 - (1024 + zero) = -(64 + zero), exactly
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(nz) : "r"(0x63806380u), "r"(z2));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w >> (8 * i), lo = and_or(v, 0x000f000fu, 0x64006400u), hi = and_or(v, 0x00f000f0u, 0x64006400u);
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[2 * i]) : "r"(lo), "r"(z2));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[2 * i + 1]) : "r"(hi), "r"(0x2c002c00u), "r"(nz));
    }
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// Eight elements of a token in the order of the expanded codes: pairs (j, j + 4).
__device__ __forceinline__ void sts_paired(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(__byte_perm(v.x, v.z, 0x5410)), "r"(__byte_perm(v.x, v.z, 0x7632)),
               "r"(__byte_perm(v.y, v.w, 0x5410)), "r"(__byte_perm(v.y, v.w, 0x7632)) : "memory");
}
__device__ __forceinline__ void tma_codes(uint32_t dst, const CUtensorMap* map, uint32_t bar, int byte, int row) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               :: "r"(dst), "l"(map), "r"(byte), "r"(row), "r"(bar) : "memory");
}

// ------------------------------------------------------------------ clusters

constexpr int kMostCluster = 8;

// Address of another block's shared memory in the cluster.
__device__ __forceinline__ uint32_t in_block(uint32_t a, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void sync_cluster() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Clusters of `blocks` blocks that a device runs at once, asked once.
template <auto kKernel>
int clusters(const cudaLaunchConfig_t& cfg, int blocks, int dev) {
  static std::atomic<int> known[kMaxDevices][kMostCluster + 1];
  int n = known[dev][blocks].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = -1;
    }
    known[dev][blocks].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Windows of up to 32 tokens on the tensor cores' own memory (w4_tensor.cu); codes: boxes of kTensorRows features x one unit.
constexpr int kTensorRows = 128;
cudaError_t launch_w4_tensor(const W4Params& p, const CUtensorMap& codes, bool bf16, int group, int dev, cudaStream_t s);

}  // namespace mdw
