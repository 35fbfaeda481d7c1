// mdw_linear_tree_attention: the nodes of trees of drafted tokens against a state that stays as it is.
//
// Mathematics. Node i comes after its ancestors j (mask_i, itself among them). With b_i the sum of their log decays,
//   o_i = scale ( e^{b_i} S^T q_i + sum_{j in mask_i} e^{b_i - b_j} (q_i . k_j) v_j ):
// b_i - b_j is the sum over the nodes between the two, taken as such (differences of long sums would lose digits).
//
// What bounds it up to a few nodes is the state's 64 KB (heads of 128) from memory.
#include <cmath>

#include "linear.cuh"

namespace mdw {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kNodes = 8;

template <int D>
__global__ void __launch_bounds__(kThreads) tree_kernel(const LinearParams p) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes, kPer = D / kGroups;
  __shared__ float prob[MDW_MAX_TREE][MDW_MAX_TREE], whole[MDW_MAX_TREE], gs[MDW_MAX_TREE];
  __shared__ uint64_t bits[MDW_MAX_TREE];
  __shared__ __align__(16) float qs[kNodes][D], parts[kNodes][kWarps][D];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  LinearRequest r;
  if (!linear_request(p, b, r) || r.n == 0) return;
  const int c = tid % kLanes * 4, a0 = tid / kLanes * kPer;
  float4 s[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.in >= 0) s[i] = *reinterpret_cast<const float4*>(p.s + r.in * p.slot_stride + ((int64_t)h * D + a0 + i) * D + c);
  }
  const int64_t qk = (int64_t)(h / p.share) * D;
  for (int i = tid; i < r.n; i += kThreads) {
    bits[i] = ((p.bits ? p.bits[r.row0 + i] : ~0ull) & ((1ull << i) - 1)) | 1ull << i;
    gs[i] = log_decay_of(p, r.row0 + i, h);
  }
  __syncthreads();
  for (int at = tid; at < r.n * r.n; at += kThreads) {
    const int i = at / r.n, j = at % r.n;
    float x = 0.f;
    if (bits[i] >> j & 1) {
      float gap = 0.f, dot = 0.f;
      for (int m = j + 1; m <= i; ++m)
        if (bits[i] >> m & 1) gap += gs[m];
      for (int e = 0; e < D; ++e)
        dot = fmaf(__bfloat162float(p.q[(r.row0 + i) * p.ldq + qk + e]), __bfloat162float(p.k[(r.row0 + j) * p.ldk + qk + e]), dot);
      x = dot * expf(gap);
    }
    prob[i][j] = x;
  }
  for (int i = tid; i < r.n; i += kThreads) {
    float sum = 0.f;
    for (int m = 0; m <= i; ++m)
      if (bits[i] >> m & 1) sum += gs[m];
    whole[i] = r.in < 0 ? 0.f : expf(sum);
  }
  for (int first = 0; first < r.n; first += kNodes) {
    const int count = min(r.n - first, kNodes);
    __syncthreads();
    for (int i = tid; i < count * D; i += kThreads) qs[i / D][i % D] = __bfloat162float(p.q[(r.row0 + first + i / D) * p.ldq + qk + i % D]);
    __syncthreads();
    for (int t = 0; t < count; ++t) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float q = qs[t][a0 + i];
        o = make_float4(fmaf(q, s[i].x, o.x), fmaf(q, s[i].y, o.y), fmaf(q, s[i].z, o.z), fmaf(q, s[i].w, o.w));
      }
#pragma unroll
      for (int m = kLanes; m < 32; m <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
      }
      if (lane < kLanes) *reinterpret_cast<float4*>(&parts[t][warp][c]) = o;
    }
    __syncthreads();
    for (int i = tid; i < count * D; i += kThreads) {
      const int t = i / D, at = i % D, node = first + t;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) o += parts[t][w][at];
      o = r.in < 0 ? 0.f : o * whole[node];
      for (int j = 0; j <= node; ++j)
        if (bits[node] >> j & 1) o = fmaf(prob[node][j], __bfloat162float(p.v[(r.row0 + j) * p.ldv + (int64_t)h * D + at]), o);
      p.out[(int64_t)(r.row0 + node) * p.ldo + (int64_t)h * D + at] = __float2bfloat16_rn(o * p.scale);
    }
  }
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" mdw_status mdw_linear_tree_attention(const mdw_linear_state* state, int32_t B, int32_t T, int32_t qk_heads,
                                                int32_t max_new, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                                const void* v, int64_t ldv, const float* log_decay, int64_t ldd, void* out,
                                                int64_t ldo, const int32_t* row_start, const int32_t* slot_in,
                                                const uint64_t* tree_mask, float scale, uint32_t* status,
                                                mdw_stream_t stream) {
  const mdw_status st = check_linear_call(state, B, T, qk_heads, max_new, k, ldk, v, ldv, log_decay, ldd, row_start, slot_in, status);
  if (st != MDW_OK) return st;
  const int D = state->head_dim;
  if (max_new > MDW_MAX_TREE || !aligned_to(q, 16) || !row_stride_ok(ldq, (int64_t)qk_heads * D) || !aligned_to(out, 16) ||
      !row_stride_ok(ldo, (int64_t)state->heads * D) || !null_or_aligned(tree_mask, 8) || !std::isfinite(scale))
    return MDW_ERR_INVALID_ARG;
  const LinearParams p{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                       log_decay, static_cast<__nv_bfloat16*>(out), ldq, ldk, ldv, ldd, ldo, state->slot_stride, state->s, row_start, slot_in,
                       nullptr, tree_mask, status, scale, B, T, state->heads, state->heads / qk_heads, max_new, state->num_slots, 0, nullptr, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(1, p.H, p.B);
  if (D == 128) tree_kernel<128><<<grid, kThreads, 0, s>>>(p);
  else tree_kernel<64><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
