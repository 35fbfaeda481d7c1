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
  __shared__ int64_t sum_rows[kPlanThreads / 32], sum_pages[kPlanThreads / 32];
  // Every block computes the whole prefix sums (a few kilobytes of lengths): no block waits for another.
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t most = (int64_t)p.max_pages << p.page_shift;
  const int round = (1 << p.page_shift) - 1;
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  const int limit = p.parents || p.tree_mask ? MDW_MAX_TREE : 0x7fffffff;
  int64_t rows = 0, pages = 0;
  int fail = 0;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = p.ctx_len[b], n = p.new_len[b];
    if (c < 0 || n < 0 || c + n > most || n > limit) { fail = 1; break; }
    start[b] = (int32_t)n;
    first[b] = (int32_t)(((c + n + round) >> p.page_shift) - ((c + round) >> p.page_shift));
    rows += n;
    pages += first[b];
  }
  // inclusive sums over the warp's threads, then the warps before
  int64_t rows_to = rows, pages_to = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(0xffffffffu, rows_to, o), g = __shfl_up_sync(0xffffffffu, pages_to, o);
    if (lane >= o) { rows_to += r; pages_to += g; }
  }
  if (lane == 31) { sum_rows[warp] = rows_to; sum_pages[warp] = pages_to; }
  fail = __syncthreads_or(fail);
  int64_t all_rows = 0, all_pages = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) { rows_to += sum_rows[w]; pages_to += sum_pages[w]; }
    all_rows += sum_rows[w];
    all_pages += sum_pages[w];
  }
  const bool bad = fail || all_rows > p.T || all_pages > p.num_free;
  if (bad) {
    if (tid == 0 && blockIdx.x == 0) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
  } else {
    int32_t r = (int32_t)(rows_to - rows), g = (int32_t)(pages_to - pages);
    for (int b = b0; b < b1; ++b) {
      const int32_t n = start[b], f = first[b];
      start[b] = r;
      first[b] = g;
      r += n;
      g += f;
    }
    if (tid == 0) { start[p.B] = (int32_t)all_rows; first[p.B] = (int32_t)all_pages; }
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
  int T, rows;                         // rows of the call, rows per block
  int chunks, dim_shift, page_shift;   // 8-element pieces of a row; log2 of pieces per head; of page size
};

__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// The largest magnitude of two elements in each half (NaN counts as small).
__device__ __forceinline__ __nv_bfloat162 most2(__nv_bfloat162 a, __nv_bfloat162 b) { return __hmax2(__habs2(a), __habs2(b)); }
__device__ __forceinline__ __half2 most2(__half2 a, __half2 b) { return __hmax2(__habs2(a), __habs2(b)); }
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct Two<__half> { using type = __half2; };

// Eight elements over their scale in E4M3: the code of the correctly rounded fp32 quotient, so that it depends
// on nothing but x and scale. With y = RN(1 / s) and q = RN(x y), RN(q + (x - q s) y) is RN(x / s) (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990) if the remainder
// is exact and s has not the largest significand: scales of other magnitudes than 2^-64 .. 2^64 and that
// significand are divided by, and so are eight elements of which one is beyond 1024 s (far above what saturates; infinite
// ones among them). The remainder is taken as q s - x, whose sign leaves -0 as it is.
template <typename T>
__device__ __forceinline__ uint2 to_e4m3(uint4 x, float s) {
  using T2 = typename Two<T>::type;
  T e[8];
  T2 two[4];
  memcpy(e, &x, 16);
  memcpy(two, &x, 16);
  const T2 most = most2(most2(two[0], two[1]), most2(two[2], two[3]));
  const float top = fmaxf(Elem<T>::to_float(most.x), Elem<T>::to_float(most.y)), y = __frcp_rn(s);
  float v[8];
  if (s >= 0x1p-64f && s <= 0x1p64f && (__float_as_uint(s) & 0x7fffffu) != 0x7fffffu && top * y < 1024.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = Elem<T>::to_float(e[j]), q = __fmul_rn(f, y);
      v[j] = __fmaf_rn(-__fmaf_rn(q, s, -f), y, q);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(Elem<T>::to_float(e[j]), s);
  }
  return make_uint2(f32x2_to_e4m3x2(v[0], v[1]) | f32x2_to_e4m3x2(v[2], v[3]) << 16,
                    f32x2_to_e4m3x2(v[4], v[5]) | f32x2_to_e4m3x2(v[6], v[7]) << 16);
}

// A block takes `rows` rows; a thread moves 8 elements of the keys and of the values at a time, two such pairs in
// flight. Neighbouring threads read and write neighbouring pieces; a head's row is the unit of the cache
// that stays whole (64 to 256 bytes). 16381 rows of 8 heads of 128, 16-bit: 22.1 us, 6.1 TB/s; to E4M3: 22.3 us, 4.5 TB/s
// (six blocks an SM; five 22.9, eight 24.0: their registers no longer hold two pairs).
template <typename T, bool kE4M3>
__global__ void __launch_bounds__(256, 6) kv_write_kernel(const WriteParams p) {
  const int row0 = blockIdx.x * p.rows, pieces = min(p.rows, p.T - row0) * p.chunks;
  for (int i = threadIdx.x; i < pieces; i += 512) {
    uint4 k[2], v[2];
    int64_t to[2];
    int head[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int at = i + 256 * j, r = at / p.chunks, chunk = at - r * p.chunks;
      to[j] = -1;
      if (at >= pieces) continue;
      const int64_t slot = p.slot_map[row0 + r];
      if (slot < 0 || slot >= p.slots) {
        if (slot != -1) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
        continue;
      }
      k[j] = ld_once(static_cast<const T*>(p.k) + (row0 + r) * p.ldk + 8 * chunk);
      v[j] = ld_once(static_cast<const T*>(p.v) + (row0 + r) * p.ldv + 8 * chunk);
      head[j] = chunk >> p.dim_shift;
      const int part = chunk & ((1 << p.dim_shift) - 1);
      to[j] = (slot >> p.page_shift) * p.page_stride +
              ((((int64_t)head[j] << p.page_shift) + (slot & ((1 << p.page_shift) - 1))) << (p.dim_shift + 3)) + 8 * part;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (to[j] < 0) continue;
      if constexpr (!kE4M3) {
        *reinterpret_cast<uint4*>(static_cast<T*>(p.kc) + to[j]) = k[j];
        *reinterpret_cast<uint4*>(static_cast<T*>(p.vc) + to[j]) = v[j];
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.kc) + to[j]) = to_e4m3<T>(k[j], p.k_scale[head[j]]);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.vc) + to[j]) = to_e4m3<T>(v[j], p.v_scale[head[j]]);
      }
    }
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
  // four blocks an SM: more repeat the prefix sums, fewer have too few stores on their way (199 prompts with 390k rows 6.1 us; 8:
  // 7.3, 3: 6.3, 2: 7.7)
  const int dev = current_device(), most = 4 * sm_count(dev);
  if (most <= 0) return MDW_ERR_CUDA;
  const int wanted = (T + kPlanThreads - 1) / kPlanThreads, blocks = wanted < most ? wanted : most;
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
  const int sms = sm_count(current_device());
  if (sms <= 0) return MDW_ERR_CUDA;
  // about 512 pieces a block (one round of its threads), fewer where that leaves SMs without a block
  const int chunks = (int)(width / 8);
  int rows = (512 + chunks - 1) / chunks;
  if (T / rows < 4 * sms) rows = T / (4 * sms) < 1 ? 1 : T / (4 * sms);
  const WriteParams p{k, v, ldk, ldv, cache->k, cache->v, cache->page_stride, (int64_t)cache->num_pages * cache->page_size,
                      cache->k_scale, cache->v_scale, slot_map, status, T, rows, chunks, log2_of(cache->head_dim / 8),
                      log2_of(cache->page_size)};
  const unsigned blocks = (unsigned)((T + rows - 1) / rows);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == MDW_DT_BF16) {
    if (fp8) kv_write_kernel<__nv_bfloat16, true><<<blocks, 256, 0, s>>>(p);
    else kv_write_kernel<__nv_bfloat16, false><<<blocks, 256, 0, s>>>(p);
  } else {
    if (fp8) kv_write_kernel<__half, true><<<blocks, 256, 0, s>>>(p);
    else kv_write_kernel<__half, false><<<blocks, 256, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
