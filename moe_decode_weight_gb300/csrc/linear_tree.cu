// mdw_linear_tree_attention: the nodes of trees of drafted tokens against a state that stays as it is.
//
// Mathematics. Node i comes after the nodes j of its mask (itself among them). With e_ij the sum of the log decays of those of
// them that come after j, and e_i that of all,
//   o_i = scale ( e^{e_i} S^T q_i + sum_{j in mask_i} e^{e_ij} (q_i . k_j) v_j ).
// e_ij is summed from node i downwards, so a large sum never leaves a small difference.
//
// What bounds it up to 16 nodes is the state's 64 KB (heads of 128) from memory, so a block requests all of it before
// anything else: a thread's loads are whole operands of m16n8k16 products (four columns of it are four tiles' column, which
// only changes the order of the columns), turned into two bf16 numbers that hold 16 bits together. The scores and weights are
// products of the same kind, the weights as two bf16 numbers too. 16 rows a block, or 32 or 64.
//
// 64 nodes: three quarters of the products are with the state.
#include <cmath>

#include "linear.cuh"

namespace mdw {
namespace {

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two numbers as the sum of two bf16 numbers each; what is not finite is itself and nothing.
__device__ __forceinline__ void split(float a, float b, uint32_t& high, uint32_t& low) {
  high = pack(a, b);
  const float x = a - __uint_as_float(high << 16), y = b - __uint_as_float(high & 0xffff0000u);
  low = pack(isfinite(a) ? x : 0.f, isfinite(b) ? y : 0.f);
}
__device__ __forceinline__ uint32_t lds(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}

// kTiles tiles of 16 nodes.
template <int D, int kTiles>
struct Shape {
  static constexpr int kThreads = 2 * D, kWarps = kThreads / 32, kNodes = 16 * kTiles;
  static constexpr int kRow = D + 8;                            // elements from one row to the next in shared memory: no bank twice
  static constexpr int kWeights = kNodes + 4, kSums = D + 4;
  static constexpr int kSmem = 3 * kNodes * kRow * 2 + kNodes * kWeights * 4 + kNodes * kSums * 4 + kNodes * (4 + 8) + D * 8 + 16;
};

template <int D, int kTiles>
__global__ void __launch_bounds__(2 * D, kTiles == 4 ? 1 : 2) tree_kernel(const LinearParams p) {
  using S = Shape<D, kTiles>;
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16* qs = reinterpret_cast<__nv_bfloat16*>(smem);
  __nv_bfloat16* ks = qs + S::kNodes * S::kRow;
  __nv_bfloat16* vs = ks + S::kNodes * S::kRow;
  uint64_t* bits = reinterpret_cast<uint64_t*>(vs + S::kNodes * S::kRow);
  uint64_t* odd = bits + S::kNodes;                             // per column the nodes whose value is not finite
  float* weights = reinterpret_cast<float*>(odd + D);           // [node][node] e^{e_ij}; -1 where j is not seen
  float* from_state = weights + S::kNodes * S::kWeights;        // [node][D]
  float* whole = from_state + S::kNodes * S::kSums;             // e^{e_i}
  int* any_odd = reinterpret_cast<int*>(whole + S::kNodes);
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  LinearRequest r;
  if (!linear_request(p, b, r) || r.n == 0) return;

  // ---- the state: warp = 32 columns and half of the rows
  constexpr int kColumns = D / 32, kSteps = D / 32;             // groups of columns; 16 rows of half the state
  const int col0 = warp % kColumns * 32, half = warp / kColumns, row0 = half * (D / 2);
  float4 state[kSteps][4];
  if (r.in >= 0) {
    const float* src = p.s + r.in * p.slot_stride + (int64_t)h * D * D + (int64_t)(row0 + 2 * t) * D + col0 + 4 * g;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) state[k][i] = __ldg(reinterpret_cast<const float4*>(src + (16 * k + (i & 1) + 8 * (i >> 1)) * D));
  }

  // ---- rows of q, k and v; zeros behind the last
  const int64_t qk = (int64_t)(h / p.share) * D;
  for (int i = tid; i < D; i += S::kThreads) odd[i] = 0;
  if (tid == 0) *any_odd = 0;
  constexpr int kPieces = S::kNodes * D / 8 / S::kThreads;      // of 8 elements, a thread
  uint4 piece[3][kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = i * S::kThreads + tid, node = at / (D / 8), e = at % (D / 8) * 8;
    piece[0][i] = piece[1][i] = piece[2][i] = make_uint4(0u, 0u, 0u, 0u);
    if (node < r.n) {
      const int64_t row = r.row0 + node;
      piece[0][i] = *reinterpret_cast<const uint4*>(p.q + row * p.ldq + qk + e);
      piece[1][i] = *reinterpret_cast<const uint4*>(p.k + row * p.ldk + qk + e);
      piece[2][i] = *reinterpret_cast<const uint4*>(p.v + row * p.ldv + (int64_t)h * D + e);
    }
  }
  // ---- weights: a warp's rows, two nodes a lane, sums from the row downwards
  const float g0 = 2 * lane < r.n ? log_decay_of(p, r.row0 + 2 * lane, h) : 0.f;
  const float g1 = 2 * lane + 1 < r.n ? log_decay_of(p, r.row0 + 2 * lane + 1, h) : 0.f;
#pragma unroll 4
  for (int j = 0; j < S::kNodes / S::kWarps; ++j) {
    const int i = j * S::kWarps + warp;
    uint64_t seen = 0;
    if (i < r.n) seen = ((p.bits ? p.bits[r.row0 + i] : ~0ull) & ((1ull << i) - 1)) | 1ull << i;
    const bool s0 = seen >> (2 * lane) & 1, s1 = seen >> (2 * lane + 1) & 1;
    const float x1 = s1 ? g1 : 0.f;
    float sum = (s0 ? g0 : 0.f) + x1;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float down = __shfl_down_sync(0xffffffffu, sum, m);
      if (lane + m < 32) sum += down;
    }
    float after = __shfl_down_sync(0xffffffffu, sum, 1);        // of all nodes after the lane's
    if (lane == 31) after = 0.f;
    if (2 * lane < S::kNodes) *reinterpret_cast<float2*>(&weights[i * S::kWeights + 2 * lane]) = make_float2(s0 ? expf(after + x1) : -1.f, s1 ? expf(after) : -1.f);
    if (lane == 0) {
      whole[i] = expf(sum);
      bits[i] = seen;
    }
  }
  __syncthreads();                                              // (odd is cleared)
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = i * S::kThreads + tid, node = at / (D / 8), e = at % (D / 8) * 8;
    uint4 v = piece[2][i];
    const uint32_t m = 0x7f807f80u, one = 0x00800080u;          // (an exponent of ones and one more carry into the sign's place)
    if ((((v.x & m) + one) | ((v.y & m) + one) | ((v.z & m) + one) | ((v.w & m) + one)) & 0x80008000u) {
      // values that are not finite stay out of the product, where they would reach nodes that do not see them
      uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (uint32_t x = word[j >> 1] >> (16 * (j & 1)); (x & 0x7f80u) == 0x7f80u) {
          word[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
          atomicOr(reinterpret_cast<unsigned long long*>(&odd[e + j]), 1ull << node);
        }
      v = make_uint4(word[0], word[1], word[2], word[3]);
      *any_odd = 1;
    }
    *reinterpret_cast<uint4*>(qs + node * S::kRow + e) = piece[0][i];
    *reinterpret_cast<uint4*>(ks + node * S::kRow + e) = piece[1][i];
    *reinterpret_cast<uint4*>(vs + node * S::kRow + e) = v;
  }
  __syncthreads();

  // ---- what the nodes read of the state: halves of the rows one after the other
  if (r.in >= 0) {
    float acc[kTiles][4][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t high[4][2], low[4][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 x = state[k][2 * i], y = state[k][2 * i + 1];
        split(x.x, y.x, high[0][i], low[0][i]);
        split(x.y, y.y, high[1][i], low[1][i]);
        split(x.z, y.z, high[2][i], low[2][i]);
        split(x.w, y.w, high[3][i], low[3][i]);
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const __nv_bfloat16* q = qs + (16 * i + g) * S::kRow + row0 + 16 * k + 2 * t;
        const uint32_t a[4] = {lds(q), lds(q + 8 * S::kRow), lds(q + 8), lds(q + 8 * S::kRow + 8)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma(acc[i][j], a, low[j][0], low[j][1]);
          mma(acc[i][j], a, high[j][0], high[j][1]);
        }
      }
    }
    // a thread's columns: col0 + 8 t .. + 7 of rows g and g + 8 of each tile
#pragma unroll
    for (int turn = 1; turn >= 0; --turn) {
      if (half == turn)
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float4* to = reinterpret_cast<float4*>(&from_state[(16 * i + g + 8 * (e >> 1)) * S::kSums + col0 + 8 * t + 4 * (e & 1)]);
            float4 x = make_float4(acc[i][0][e], acc[i][1][e], acc[i][2][e], acc[i][3][e]);
            if (turn == 0) {
              const float4 y = *to;
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            *to = x;
          }
      __syncthreads();
    }
  }

  // ---- scores, their weights, values: warp = a tile of nodes and 16 kTiles columns
  const int tile = warp % kTiles, first = warp / kTiles * S::kNodes, rows = min(r.n - 16 * tile, 16);
  if (rows <= 0) return;
  float out[2 * kTiles][4];
#pragma unroll
  for (int j = 0; j < 2 * kTiles; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[j][e] = 0.f;
  uint32_t q[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const __nv_bfloat16* at = qs + (16 * tile + g) * S::kRow + 16 * k + 2 * t;
    q[k][0] = lds(at), q[k][1] = lds(at + 8 * S::kRow), q[k][2] = lds(at + 8), q[k][3] = lds(at + 8 * S::kRow + 8);
  }
#pragma unroll 1
  for (int from = 0; from <= tile; ++from) {                    // 16 nodes that come before (or are the tile's own)
    uint32_t high[4], low[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const __nv_bfloat16* k_at = ks + (16 * from + 8 * j + g) * S::kRow + 2 * t;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) mma(s, q[k], lds(k_at + 16 * k), lds(k_at + 16 * k + 8));
      const float2 w0 = *reinterpret_cast<const float2*>(&weights[(16 * tile + g) * S::kWeights + 16 * from + 8 * j + 2 * t]);
      const float2 w1 = *reinterpret_cast<const float2*>(&weights[(16 * tile + g + 8) * S::kWeights + 16 * from + 8 * j + 2 * t]);
      split(w0.x < 0.f ? 0.f : s[0] * w0.x, w0.y < 0.f ? 0.f : s[1] * w0.y, high[2 * j], low[2 * j]);
      split(w1.x < 0.f ? 0.f : s[2] * w1.x, w1.y < 0.f ? 0.f : s[3] * w1.y, high[2 * j + 1], low[2 * j + 1]);
    }
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      uint32_t v[4];                                            // two tiles of 8 columns
      ldmatrix_trans(v, smem_at(vs + (16 * from + (lane & 15)) * S::kRow + first + 16 * j + 8 * (lane >> 4)));
      mma(out[2 * j], low, v[0], v[1]);
      mma(out[2 * j], high, v[0], v[1]);
      mma(out[2 * j + 1], low, v[2], v[3]);
      mma(out[2 * j + 1], high, v[2], v[3]);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int node = 16 * tile + g + 8 * e;
    if (g + 8 * e >= rows) continue;
    const float f = whole[node];
    __nv_bfloat16* dst = p.out + (int64_t)(r.row0 + node) * p.ldo + (int64_t)h * D + first + 2 * t;
#pragma unroll
    for (int j = 0; j < 2 * kTiles; ++j) {
      float x = out[j][2 * e], y = out[j][2 * e + 1];
      if (r.in >= 0) {
        const float2 s = *reinterpret_cast<const float2*>(&from_state[node * S::kSums + first + 8 * j + 2 * t]);
        x = fmaf(s.x, f, x);
        y = fmaf(s.y, f, y);
      }
      if (*any_odd) {
        if (odd[first + 8 * j + 2 * t] & bits[node]) x = __int_as_float(0x7fffffff);
        if (odd[first + 8 * j + 2 * t + 1] & bits[node]) y = __int_as_float(0x7fffffff);
      }
      *reinterpret_cast<uint32_t*>(dst + 8 * j) = pack(x * p.scale, y * p.scale);
    }
  }
}

template <int D, int kTiles>
cudaError_t launch(const LinearParams& p, int dev, cudaStream_t s) {
  using S = Shape<D, kTiles>;
  const cudaError_t e = allow_shared_memory<tree_kernel<D, kTiles>>(dev);
  if (e != cudaSuccess) return e;
  tree_kernel<D, kTiles><<<dim3(p.H, p.B), S::kThreads, S::kSmem, s>>>(p);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch(const LinearParams& p, int dev, cudaStream_t s) {
  if (p.max_new <= 16) return launch<D, 1>(p, dev, s);
  return p.max_new <= 32 ? launch<D, 2>(p, dev, s) : launch<D, 4>(p, dev, s);
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
  const int dev = current_device();
  if (dev < 0) return MDW_ERR_CUDA;
  return (D == 128 ? launch<128>(p, dev, s) : launch<64>(p, dev, s)) == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
