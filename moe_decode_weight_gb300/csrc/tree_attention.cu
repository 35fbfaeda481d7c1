// mdw_tree_attention: attention of trees of drafted tokens over the paged key/value cache.
#include <cmath>

#include "mdw_attn.cuh"
#include "mdw_device.cuh"

namespace mdw {
namespace {

struct AttnParams {
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride;
  const void* q;
  void* out;
  float* lse;
  int64_t ldq, ldo;
  const int32_t* block_table;
  const int32_t* ctx_len;
  const int32_t* row_start;
  const uint64_t* tree_mask;
  uint32_t* status;
  float scale;
  int B, T, Hq, Hkv, group, max_new, max_pages, num_pages, page_shift;
};

template <typename C> __device__ __forceinline__ float cache_value(const C* p) { return Elem<C>::to_float(*p); }
template <> __device__ __forceinline__ float cache_value<uint8_t>(const uint8_t* p) {
  const uint32_t h = e4m3x2_to_f16x2(*p);
  return __half2float(__ushort_as_half((unsigned short)h));
}

// One block per (request, node, query head): its warps take every fourth key with a running
// maximum and sum of their own and merge them at the end.
template <typename T, typename C, int D>
__global__ void __launch_bounds__(128) tree_attention_kernel(AttnParams p) {
  constexpr int kPer = D / 32;
  const int b = blockIdx.x, node = blockIdx.y, h = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = p.row_start[b], e = p.row_start[b + 1], ctx = p.ctx_len[b];
  const int64_t keys64 = (int64_t)ctx + e - s;
  if (s < 0 || e < s || e > p.T || e - s > p.max_new || ctx < 0 || keys64 > (int64_t)p.max_pages << p.page_shift) {
    raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
    return;
  }
  if (node >= e - s) return;
  const int row = s + node, kvh = h / p.group, keys = (int)keys64, mask_page = (1 << p.page_shift) - 1;
  const uint64_t bits = p.tree_mask ? p.tree_mask[row] : (node < 63 ? (2ull << node) - 1 : ~0ull);
  const float ks = p.k_scale ? p.k_scale[kvh] : 1.f, vs = p.v_scale ? p.v_scale[kvh] : 1.f;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
  for (int i = 0; i < kPer; ++i) {
    q[i] = Elem<T>::to_float(static_cast<const T*>(p.q)[row * p.ldq + (int64_t)h * D + lane * kPer + i]) * p.scale * ks;
    o[i] = 0.f;
  }
  for (int j = warp; j < keys; j += 4) {
    if (j >= ctx && !(bits >> (j - ctx) & 1)) continue;
    const int32_t id = p.block_table[(size_t)b * p.max_pages + (j >> p.page_shift)];
    if (id < 0 || id >= p.num_pages) {
      raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
      continue;
    }
    const int64_t at = id * p.page_stride + (((int64_t)kvh << p.page_shift) + (j & mask_page)) * D + lane * kPer;
    float z = 0.f;
    for (int i = 0; i < kPer; ++i) z = fmaf(q[i], cache_value(static_cast<const C*>(p.k) + at + i), z);
    z = warp_sum(z);
    const float top = fmaxf(m, z);
    const float keep = m == -INFINITY ? 0.f : expf(m - top), w = z == -INFINITY ? 0.f : expf(z - top);
    l = l * keep + w;
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + (z == -INFINITY ? 0.f : w * cache_value(static_cast<const C*>(p.v) + at + i));
    m = top;
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
  for (int i = 0; i < kPer; ++i) so[warp][lane * kPer + i] = o[i];
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float total = 0.f, f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.f : expf(sm[w] - top);
    total += sl[w] * f[w];
  }
  if (threadIdx.x < D) {
    float v = 0.f;
    for (int w = 0; w < 4; ++w) v += so[w][threadIdx.x] * f[w];
    v = total == 0.f ? 0.f : v / total * vs;
    static_cast<T*>(p.out)[row * p.ldo + (int64_t)h * D + threadIdx.x] = Elem<T>::from_float(v);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[(int64_t)row * p.Hq + h] = top + logf(total);
}

template <typename T, typename C>
cudaError_t launch(const AttnParams& p, int D, cudaStream_t s) {
  const dim3 grid(p.B, p.max_new, p.Hq);
  if (D == 64) tree_attention_kernel<T, C, 64><<<grid, 128, 0, s>>>(p);
  else tree_attention_kernel<T, C, 128><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

bool sizes_ok(const mdw_kv_cache* c, int32_t B, int32_t T, int32_t q_heads, int32_t max_new) {
  return B >= 1 && B <= MDW_MAX_REQUESTS && T >= 1 && max_new >= 1 && max_new <= MDW_MAX_TREE && q_heads >= 1 &&
         q_heads % c->kv_heads == 0 && q_heads / c->kv_heads <= MDW_MAX_GROUP;
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" size_t mdw_tree_attention_workspace_bytes(const mdw_kv_cache* cache, int32_t B, int32_t T,
                                                     int32_t q_heads, int32_t max_new) {
  if (check_kv_cache(cache) != MDW_OK || !sizes_ok(cache, B, T, q_heads, max_new)) return 0;
  return 256;
}

extern "C" mdw_status mdw_tree_attention(const mdw_kv_cache* cache, int32_t B, int32_t T, int32_t q_heads,
                                         int32_t max_new, const void* q, int64_t ldq, int32_t q_dtype, void* out,
                                         int64_t ldo, float* lse, const int32_t* block_table, int32_t max_pages,
                                         const int32_t* ctx_len, const int32_t* row_start,
                                         const uint64_t* tree_mask, float scale, uint32_t* status, void* ws,
                                         size_t ws_bytes, mdw_stream_t stream) {
  const mdw_status st = check_kv_cache(cache);
  if (st != MDW_OK) return st;
  if (q_dtype != MDW_DT_BF16 && q_dtype != MDW_DT_F16) return MDW_ERR_FORMAT_MISMATCH;
  const bool fp8 = cache->dtype == MDW_DT_E4M3;
  if (!fp8 && q_dtype != cache->dtype) return MDW_ERR_FORMAT_MISMATCH;
  if (!sizes_ok(cache, B, T, q_heads, max_new)) return MDW_ERR_INVALID_ARG;
  if (max_pages < 1 || (int64_t)max_pages * cache->page_size > 0x7fffffffLL) return MDW_ERR_UNSUPPORTED_SHAPE;
  const int64_t width = (int64_t)q_heads * cache->head_dim;
  if (!aligned_to(q, 16) || !row_stride_ok(ldq, width) || !aligned_to(out, 16) || !row_stride_ok(ldo, width) ||
      !null_or_aligned(lse, 4) || !aligned_to(block_table, 4) || !aligned_to(ctx_len, 4) ||
      !aligned_to(row_start, 4) || !null_or_aligned(tree_mask, 8) || !null_or_aligned(status, 4) || !aligned_to(ws, 16))
    return MDW_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MDW_ERR_INVALID_ARG;
  if (ws_bytes < mdw_tree_attention_workspace_bytes(cache, B, T, q_heads, max_new)) return MDW_ERR_WORKSPACE_TOO_SMALL;
  AttnParams p{cache->k, cache->v, cache->k_scale, cache->v_scale, cache->page_stride, q, out, lse, ldq, ldo,
               block_table, ctx_len, row_start, tree_mask, status, scale, B, T, q_heads, cache->kv_heads,
               q_heads / cache->kv_heads, max_new, max_pages, cache->num_pages, log2_of(cache->page_size)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (q_dtype == MDW_DT_BF16)
    e = fp8 ? launch<__nv_bfloat16, uint8_t>(p, cache->head_dim, s) : launch<__nv_bfloat16, __nv_bfloat16>(p, cache->head_dim, s);
  else
    e = fp8 ? launch<__half, uint8_t>(p, cache->head_dim, s) : launch<__half, __half>(p, cache->head_dim, s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
