// The paged key/value cache: mdw_kv_plan (block tables, slot map, positions and tree masks from
// request lengths) and mdw_kv_write (rows of keys and values to their slots).
#include "mdw_attn.cuh"
#include "mdw_device.cuh"

namespace mdw {

mdw_status check_kv_cache(const mdw_kv_cache* c) {
  if (!c) return MDW_ERR_INVALID_ARG;
  if (c->magic != MDW_MAGIC || c->fmt != MDW_FMT_KV_PAGED) return MDW_ERR_FORMAT_MISMATCH;
  const bool fp8 = c->dtype == MDW_DT_E4M3;
  if (c->dtype != MDW_DT_BF16 && c->dtype != MDW_DT_F16 && !fp8) return MDW_ERR_FORMAT_MISMATCH;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0 || c->num_pages < 1 ||
      c->kv_heads < 1 || c->kv_heads > 1024 || (c->head_dim != 64 && c->head_dim != 128))
    return MDW_ERR_UNSUPPORTED_SHAPE;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return MDW_ERR_INVALID_ARG;
  if (c->page_stride < (int64_t)c->kv_heads * c->page_size * c->head_dim || c->page_stride % (fp8 ? 16 : 8) != 0 ||
      c->page_stride > (int64_t)1 << 32)
    return MDW_ERR_INVALID_ARG;
  if (fp8 ? !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4) : c->k_scale || c->v_scale)
    return MDW_ERR_INVALID_ARG;
  return MDW_OK;
}

namespace {

struct PlanParams {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* parents;
  int32_t* row_start;
  int64_t* slot_map;
  int32_t* positions;
  uint64_t* tree_mask;
  int32_t* pages_taken;
  uint32_t* status;
  int B, T, num_pages, max_pages, num_free, page_shift;
};

constexpr int kPlanThreads = 256;

// First index i of the ascending start[0..n] with start[i + 1] > v.
__device__ __forceinline__ int owner_of(const int32_t* start, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid + 1] > v) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(PlanParams p) {
  __shared__ int32_t start[MDW_MAX_REQUESTS + 1], first[MDW_MAX_REQUESTS + 1];
  __shared__ int bad;
  const int tid = threadIdx.x;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  const int round = (1 << p.page_shift) - 1;
  if (tid == 0) {
    int64_t rows = 0, pages = 0;
    int fail = 0;
    for (int b = 0; b < p.B; ++b) {
      const int64_t c = p.ctx_len[b], n = p.new_len[b];
      if (c < 0 || n < 0 || c + n > most || ((p.parents || p.tree_mask) && n > MDW_MAX_TREE)) { fail = 1; break; }
      start[b] = (int32_t)rows;
      first[b] = (int32_t)pages;
      rows += n;
      pages += ((c + n + round) >> p.page_shift) - ((c + round) >> p.page_shift);
      if (rows > p.T || pages > p.num_free) { fail = 1; break; }
    }
    start[p.B] = (int32_t)rows;
    first[p.B] = (int32_t)pages;
    bad = fail;
    if (fail) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
  }
  __syncthreads();
  const int at = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;
  for (int b = at; b <= p.B; b += step) p.row_start[b] = bad ? 0 : start[b];
  if (at == 0) *p.pages_taken = bad ? 0 : first[p.B];
  if (!bad) {
    for (int i = at; i < first[p.B]; i += step) {
      const int b = owner_of(first, p.B, i);
      const int32_t id = p.free_pages[i];
      const bool ok = id >= 0 && id < p.num_pages;
      if (!ok) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
      p.block_table[(size_t)b * p.max_pages + ((p.ctx_len[b] + round) >> p.page_shift) + i - first[b]] = ok ? id : -1;
    }
  }
  for (int r = at; r < p.T; r += step) {
    int64_t slot = -1;
    int32_t pos = -1;
    uint64_t mask = 0;
    if (!bad && r < start[p.B]) {
      const int b = owner_of(start, p.B, r), node = r - start[b];
      const int32_t ctx = p.ctx_len[b];
      int depth = node;
      bool ok = true;
      mask = node < 63 ? (2ull << node) - 1 : ~0ull;
      if (p.parents) {
        mask = 1ull << node;
        depth = 0;
        for (int cur = node;;) {
          const int up = p.parents[start[b] + cur];
          if (up < -1 || up >= cur) { ok = false; break; }
          if (up < 0) break;
          mask |= 1ull << up;
          ++depth;
          cur = up;
        }
      }
      const int place = ctx + node, page = place >> p.page_shift, have = (int)(((int64_t)ctx + round) >> p.page_shift);
      const int32_t id = page < have ? p.block_table[(size_t)b * p.max_pages + page] : p.free_pages[first[b] + page - have];
      if (id < 0 || id >= p.num_pages) ok = false;
      if (ok) {
        slot = ((int64_t)id << p.page_shift) + (place & round);
        pos = ctx + depth;
      } else {
        mask = 0;
        raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
      }
    }
    p.slot_map[r] = slot;
    p.positions[r] = pos;
    if (p.tree_mask) p.tree_mask[r] = mask;
  }
}

struct WriteParams {
  const void* k;
  const void* v;
  int64_t ldk, ldv;
  void* kc;
  void* vc;
  int64_t page_stride, slots;
  const float* k_scale;
  const float* v_scale;
  const int64_t* slot_map;
  uint32_t* status;
  int64_t items;
  int chunks, dim_shift, page_shift;   // 16-byte pieces of one row's heads; log2 of pieces per head; of page size
};

// One thread per 8 elements of one row's keys or values.
template <typename T, bool kE4M3>
__global__ void __launch_bounds__(256) kv_write_kernel(WriteParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.items) return;
  const int chunk = (int)(i % p.chunks);
  const int64_t row = i / p.chunks >> 1;
  const bool is_v = (i / p.chunks) & 1;
  const int64_t slot = p.slot_map[row];
  if (slot < 0 || slot >= p.slots) {
    if (slot != -1) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
    return;
  }
  const int head = chunk >> p.dim_shift, part = chunk & ((1 << p.dim_shift) - 1);
  const int64_t in_page = slot & ((1 << p.page_shift) - 1);
  const int64_t at = (slot >> p.page_shift) * p.page_stride +
                     ((((int64_t)head << p.page_shift) + in_page) << (p.dim_shift + 3)) + 8 * part;
  const T* src = static_cast<const T*>(is_v ? p.v : p.k) + row * (is_v ? p.ldv : p.ldk) + 8 * chunk;
  const uint4 x = *reinterpret_cast<const uint4*>(src);
  if constexpr (!kE4M3) {
    *reinterpret_cast<uint4*>(static_cast<T*>(is_v ? p.vc : p.kc) + at) = x;
  } else {
    const float s = (is_v ? p.v_scale : p.k_scale)[head];
    T e[8];
    memcpy(e, &x, 16);
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = f32x2_to_e4m3x2(__fdiv_rn(Elem<T>::to_float(e[4 * j]), s), __fdiv_rn(Elem<T>::to_float(e[4 * j + 1]), s));
      const uint32_t hi = f32x2_to_e4m3x2(__fdiv_rn(Elem<T>::to_float(e[4 * j + 2]), s), __fdiv_rn(Elem<T>::to_float(e[4 * j + 3]), s));
      out[j] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? p.vc : p.kc) + at) = make_uint2(out[0], out[1]);
  }
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" mdw_status mdw_kv_plan(int32_t B, const int32_t* ctx_len, const int32_t* new_len, int32_t page_size,
                                  int32_t num_pages, int32_t* block_table, int32_t max_pages,
                                  const int32_t* free_pages, int32_t num_free, const int32_t* parents, int32_t T,
                                  int32_t* row_start, int64_t* slot_map, int32_t* positions, uint64_t* tree_mask,
                                  int32_t* pages_taken, uint32_t* status, mdw_stream_t stream) {
  if (B < 1 || B > MDW_MAX_REQUESTS || T < 1 || num_pages < 1 || max_pages < 1 || num_free < 0)
    return MDW_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return MDW_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)max_pages * page_size > 0x7fffffffLL) return MDW_ERR_UNSUPPORTED_SHAPE;   // positions are int32
  if (!aligned_to(ctx_len, 4) || !aligned_to(new_len, 4) || !aligned_to(block_table, 4) ||
      !null_or_aligned(free_pages, 4) || (num_free > 0 && !free_pages) || !null_or_aligned(parents, 4) ||
      !aligned_to(row_start, 4) || !aligned_to(slot_map, 8) || !aligned_to(positions, 4) ||
      !null_or_aligned(tree_mask, 8) || !aligned_to(pages_taken, 4) || !null_or_aligned(status, 4))
    return MDW_ERR_INVALID_ARG;
  PlanParams p{ctx_len, new_len, block_table, free_pages, parents, row_start, slot_map, positions, tree_mask,
               pages_taken, status, B, T, num_pages, max_pages, num_free, log2_of(page_size)};
  const int blocks = (T + kPlanThreads - 1) / kPlanThreads;
  kv_plan_kernel<<<blocks, kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}

extern "C" mdw_status mdw_kv_write(const mdw_kv_cache* cache, int32_t T, const void* k, int64_t ldk, const void* v,
                                   int64_t ldv, int32_t dtype, const int64_t* slot_map, uint32_t* status,
                                   mdw_stream_t stream) {
  const mdw_status st = check_kv_cache(cache);
  if (st != MDW_OK) return st;
  if (dtype != MDW_DT_BF16 && dtype != MDW_DT_F16) return MDW_ERR_FORMAT_MISMATCH;
  const bool fp8 = cache->dtype == MDW_DT_E4M3;
  if (!fp8 && dtype != cache->dtype) return MDW_ERR_FORMAT_MISMATCH;
  const int64_t width = (int64_t)cache->kv_heads * cache->head_dim;
  if (T < 1 || !aligned_to(k, 16) || !aligned_to(v, 16) || !row_stride_ok(ldk, width) || !row_stride_ok(ldv, width) ||
      !aligned_to(slot_map, 8) || !null_or_aligned(status, 4))
    return MDW_ERR_INVALID_ARG;
  WriteParams p{k, v, ldk, ldv, cache->k, cache->v, cache->page_stride, (int64_t)cache->num_pages * cache->page_size,
                cache->k_scale, cache->v_scale, slot_map, status, 0, (int)(width / 8), log2_of(cache->head_dim / 8),
                log2_of(cache->page_size)};
  p.items = (int64_t)T * 2 * p.chunks;
  const int64_t blocks = (p.items + 255) / 256;
  if (blocks > 0x7fffffffLL) return MDW_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MDW_DT_BF16) {
    if (fp8) kv_write_kernel<__nv_bfloat16, true><<<(unsigned)blocks, 256, 0, s>>>(p);
    else kv_write_kernel<__nv_bfloat16, false><<<(unsigned)blocks, 256, 0, s>>>(p);
  } else {
    if (fp8) kv_write_kernel<__half, true><<<(unsigned)blocks, 256, 0, s>>>(p);
    else kv_write_kernel<__half, false><<<(unsigned)blocks, 256, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
