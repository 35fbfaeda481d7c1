// mdw_linear_attention (requests of few rows) and mdw_linear_state_advance: one row after the other.
//
// Mathematics. S <- e^g S + k v^T, o = scale S^T q, for a request's rows in order. The block of a request and value
// head holds S in registers, so the state is read and written once whatever the number of rows.
//
// What bounds it is the state's 64 KB (heads of 128) in and out of memory: D rows of it lie on the warps, four columns on a lane, and all
// loads are requested before the first is used. Measured: 61 requests of 1 to 4 rows and 32 heads 51 us, where a plain copy of
// their states takes 43 (a quarter of a warp's time goes to waiting for memory, as much to the barriers around the rows); one row of
// 20 heads 6 us with its launch. Asking for the state before the request is checked changed nothing; blocks that stay and copy the next state
// to shared memory meanwhile took 57: two of them an SM, with the same barriers.
#include <algorithm>
#include <cmath>
#include <utility>

#include "linear.cuh"
#include "mdw_internal.h"

namespace mdw {

mdw_status check_linear_state(const mdw_linear_state* s) {
  if (!s) return MDW_ERR_INVALID_ARG;
  if (s->magic != MDW_MAGIC || s->fmt != MDW_FMT_LINEAR_STATE) return MDW_ERR_FORMAT_MISMATCH;
  if (s->num_slots < 1 || s->heads < 1 || s->heads > 1024 || (s->head_dim != 64 && s->head_dim != 128)) return MDW_ERR_UNSUPPORTED_SHAPE;
  if (!aligned_to(s->s, 16) || s->slot_stride < (int64_t)s->heads * s->head_dim * s->head_dim || s->slot_stride % 4 != 0 ||
      s->slot_stride > (int64_t)1 << 32)
    return MDW_ERR_INVALID_ARG;
  return MDW_OK;
}

mdw_status check_linear_call(const mdw_linear_state* s, int32_t B, int32_t T, int32_t qk_heads, int32_t max_new, const void* k, int64_t ldk,
                             const void* v, int64_t ldv, const float* log_decay, int64_t ldd, const int32_t* row_start,
                             const int32_t* slot_in, const uint32_t* status) {
  const mdw_status st = check_linear_state(s);
  if (st != MDW_OK) return st;
  if (B < 1 || B > MDW_MAX_REQUESTS || T < 1 || max_new < 1 || qk_heads < 1 || s->heads % qk_heads != 0 ||
      s->heads / qk_heads > MDW_MAX_GROUP)
    return MDW_ERR_INVALID_ARG;
  if (T > 0x7fff0000) return MDW_ERR_UNSUPPORTED_SHAPE;          // rows of a chunk past the last are int32
  if (ldk > (int64_t)1 << 36 || ldv > (int64_t)1 << 36) return MDW_ERR_UNSUPPORTED_SHAPE;   // (strides of a tensor map)
  const int64_t narrow = (int64_t)qk_heads * s->head_dim, wide = (int64_t)s->heads * s->head_dim;
  if (!aligned_to(k, 16) || !row_stride_ok(ldk, narrow) || !aligned_to(v, 16) || !row_stride_ok(ldv, wide) || !aligned_to(log_decay, 4) ||
      (ldd != 0 && ldd < s->heads) || !aligned_to(row_start, 4) || !aligned_to(slot_in, 4) || !null_or_aligned(status, 4))
    return MDW_ERR_INVALID_ARG;
  return MDW_OK;
}

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRows = 8;                                        // rows whose elements are in shared memory at a time

// One block: request blockIdx.z, value head blockIdx.y, kCols of the columns. kOut: outputs of all rows; else the rows
// whose bits are set change the state only.
// Blocks of an SM, 64 of 128 columns: three with 80 registers, 12 bytes of them spilled (two or four: 59 and 52 us for the 61 requests instead of 50).
template <int D, int kCols, bool kOut>
__global__ void __launch_bounds__(kThreads, D * kCols > 64 * 64 ? 3 : 4) step_kernel(const LinearParams p) {
  constexpr int kLanes = kCols / 4, kGroups = kThreads / kLanes, kPer = D / kGroups;   // lanes of a row, rows at once, rows of a thread
  static_assert(kPer * kGroups == D && kPer % 2 == 0, "");
  __shared__ __align__(16) float qs[kOut ? kRows : 1][D], ks[kRows][D], vs[kRows][kCols];
  __shared__ __align__(16) float parts[kOut ? kRows : 1][kWarps][kCols];
  __shared__ float factor[kRows], keep[kRows];
  __shared__ int taken[kRows];
  const int b = blockIdx.z, h = blockIdx.y, col0 = blockIdx.x * kCols, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kOut) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (plan_kernel of longer requests waits for this one's end)
  const int c = tid % kLanes * 4, a0 = tid / kLanes * kPer;
  const int64_t at = ((int64_t)h * D + a0) * D + col0 + c;
  LinearRequest r;
  const bool sound = linear_request(p, b, r);
  if (kOut && p.ok && blockIdx.x == 0 && h == 0 && tid == 0) p.ok[b] = sound;
  if (!sound || (kOut && r.n > p.short_rows)) return;
  if (r.out < 0 && !(kOut && r.n > 0)) return;
  Pair s[kPer][2];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r.in >= 0) x = __ldcs(reinterpret_cast<const float4*>(p.s + r.in * p.slot_stride + at + i * D));
    s[i][0] = Pair(x.x, x.y);
    s[i][1] = Pair(x.z, x.w);
  }
  uint64_t left = 0;                                            // accepted rows that are still to come
  if (!kOut) left = p.bits[b] & (r.n < 64 ? (1ull << r.n) - 1 : ~0ull);
  int next = 0;
  for (;;) {
    int count;
    if (kOut) {
      count = min(r.n - next, kRows);
    } else {
      count = min(__popcll(left), kRows);
      if (tid < count) {
        uint64_t from = left;                                   // without its first tid bits
        for (int i = 0; i < tid; ++i) from &= from - 1;
        taken[tid] = r.row0 + __ffsll((long long)from) - 1;
      }
      for (int i = 0; i < count; ++i) left &= left - 1;
      __syncthreads();
    }
    if (count <= 0) break;
    auto row_of = [&](int i) { return kOut ? r.row0 + next + i : taken[i]; };
    // pieces of 8 elements: k, then v's columns of the block, then q
    constexpr int kOfRow = D / 8 + kCols / 8 + (kOut ? D / 8 : 0);
    for (int i = tid; i < count * kOfRow; i += kThreads) {
      const int t = i / kOfRow, piece = i % kOfRow, row = row_of(t);
      const __nv_bfloat16* src;
      float* dst;
      if (piece < D / 8) {
        src = p.k + row * p.ldk + (int64_t)(h / p.share) * D + 8 * piece;
        dst = &ks[t][8 * piece];
      } else if (piece < D / 8 + kCols / 8) {
        src = p.v + row * p.ldv + (int64_t)h * D + col0 + 8 * (piece - D / 8);
        dst = &vs[t][8 * (piece - D / 8)];
      } else {
        src = p.q + row * p.ldq + (int64_t)(h / p.share) * D + 8 * (piece - D / 8 - kCols / 8);
        dst = &qs[t][8 * (piece - D / 8 - kCols / 8)];
      }
      const uint4 x = *reinterpret_cast<const uint4*>(src);
      reinterpret_cast<float4*>(dst)[0] = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                                                      __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
      reinterpret_cast<float4*>(dst)[1] = make_float4(__uint_as_float(x.z << 16), __uint_as_float(x.z & 0xffff0000u),
                                                      __uint_as_float(x.w << 16), __uint_as_float(x.w & 0xffff0000u));
    }
    if (tid < count) {
      const Decay decay(log_decay_of(p, row_of(tid), h));
      factor[tid] = decay.f;
      keep[tid] = decay.near ? 1.f : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < count; ++t) {
      const Pair f(factor[t], factor[t]), same(keep[t], keep[t]);
      const float4 v4 = *reinterpret_cast<const float4*>(&vs[t][c]);
      const Pair v[2] = {Pair(v4.x, v4.y), Pair(v4.z, v4.w)};
      Pair o[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 k = *reinterpret_cast<const float2*>(&ks[t][a0 + i]);
        float2 q = make_float2(0.f, 0.f);
        if (kOut) q = *reinterpret_cast<const float2*>(&qs[t][a0 + i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float kk = j < 2 ? k.x : k.y;
          Pair& x = s[i + (j >> 1)][j & 1];
          x = fma(x, same, fma(x, f, Pair(kk, kk) * v[j & 1]));  // (the product of two bf16 numbers is exact)
          if (kOut) {
            const float qq = j < 2 ? q.x : q.y;
            o[j & 1] = fma(Pair(qq, qq), x, o[j & 1]);
          }
        }
      }
      if (kOut) {
        float4 sum = make_float4(o[0].floats().x, o[0].floats().y, o[1].floats().x, o[1].floats().y);
#pragma unroll
        for (int m = kLanes; m < 32; m <<= 1) {
          sum.x += __shfl_xor_sync(0xffffffffu, sum.x, m);
          sum.y += __shfl_xor_sync(0xffffffffu, sum.y, m);
          sum.z += __shfl_xor_sync(0xffffffffu, sum.z, m);
          sum.w += __shfl_xor_sync(0xffffffffu, sum.w, m);
        }
        if (lane < kLanes) *reinterpret_cast<float4*>(&parts[t][warp][c]) = sum;
      }
    }
    __syncthreads();
    if (kOut)
      for (int i = tid; i < count * (kCols / 2); i += kThreads) {
        const int t = i / (kCols / 2), col = i % (kCols / 2) * 2;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 part = *reinterpret_cast<const float2*>(&parts[t][w][col]);
          x += part.x;
          y += part.y;
        }
        *reinterpret_cast<__nv_bfloat162*>(p.out + (int64_t)(r.row0 + next + t) * p.ldo + (int64_t)h * D + col0 + col) =
            __floats2bfloat162_rn(x * p.scale, y * p.scale);
      }
    next += count;
  }
  if (r.out >= 0)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float2 x = s[i][0].floats(), y = s[i][1].floats();
      __stcs(reinterpret_cast<float4*>(p.s + r.out * p.slot_stride + at + i * D), make_float4(x.x, x.y, y.x, y.y));
    }
}

template <int D, int kCols, bool kOut>
void launch_cols(const LinearParams& p, cudaStream_t s) {
  step_kernel<D, kCols, kOut><<<dim3(D / kCols, p.H, p.B), kThreads, 0, s>>>(p);
}
template <bool kOut>
cudaError_t launch_step(const LinearParams& p, int D, int sms, cudaStream_t s) {
  // columns are split further where few requests and heads leave SMs without a block (20 heads, 4 rows: one request 9.4 us instead of 11.4,
  // 4 the same, 8 15.5 instead of 14.4, 16 21.6 instead of 19.6)
  const bool few = (int64_t)p.B * p.H * (D / 64) <= sms;
  if (D == 128) {
    if (few) launch_cols<128, 32, kOut>(p, s);
    else launch_cols<128, 64, kOut>(p, s);
  } else {
    if (few) launch_cols<64, 32, kOut>(p, s);
    else launch_cols<64, 64, kOut>(p, s);
  }
  return cudaGetLastError();
}

// The parts of the workspace, and its bytes. Segments of requests that have several: their number times the heads is at most the number of
// blocks (a segment is at least a block's share of all chunks and heads); each has three pieces, and a set of states for a piece.
std::pair<LinearPlan, size_t> plan_of(uint8_t* ws, int B, int D, int grid) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = ws + at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  LinearPlan w;
  w.head = reinterpret_cast<int32_t*>(take(256));
  w.ok = reinterpret_cast<int32_t*>(take((size_t)B * 4));
  w.all = reinterpret_cast<LinearEntry*>(take((size_t)(B + grid) * sizeof(LinearEntry)));
  w.first = reinterpret_cast<LinearEntry*>(take((size_t)kLinearPieces * grid * sizeof(LinearEntry)));
  w.joins = reinterpret_cast<LinearEntry*>(take((size_t)grid * sizeof(LinearEntry)));
  w.logs = reinterpret_cast<float*>(take((size_t)kLinearPieces * grid * 4));
  w.states = reinterpret_cast<float*>(take((size_t)kLinearPieces * grid * D * D * 4));
  return {w, at};
}

}  // namespace
}  // namespace mdw

using namespace mdw;

extern "C" size_t mdw_linear_attention_workspace_bytes(const mdw_linear_state* state, int32_t B, int32_t T,
                                                       int32_t qk_heads, int32_t max_new) {
  if (check_linear_state(state) != MDW_OK || B < 1 || B > MDW_MAX_REQUESTS || T < 1 || T > 0x7fff0000 || max_new < 1 || qk_heads < 1 ||
      state->heads % qk_heads != 0 || state->heads / qk_heads > MDW_MAX_GROUP)
    return 0;
  const int grid = sm_count(current_device());
  return plan_of(nullptr, B, state->head_dim, std::max(grid, 1)).second;
}

extern "C" mdw_status mdw_linear_attention(const mdw_linear_state* state, int32_t B, int32_t T, int32_t qk_heads,
                                           int32_t max_new, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                           const void* v, int64_t ldv, const float* log_decay, int64_t ldd, void* out,
                                           int64_t ldo, const int32_t* row_start, const int32_t* slot_in,
                                           const int32_t* slot_out, float scale, uint32_t* status, void* ws,
                                           size_t ws_bytes, mdw_stream_t stream) {
  const mdw_status st = check_linear_call(state, B, T, qk_heads, max_new, k, ldk, v, ldv, log_decay, ldd, row_start, slot_in, status);
  if (st != MDW_OK) return st;
  const int D = state->head_dim;
  if (!aligned_to(q, 16) || !row_stride_ok(ldq, (int64_t)qk_heads * D) || !aligned_to(out, 16) || !row_stride_ok(ldo, (int64_t)state->heads * D) ||
      !aligned_to(slot_out, 4) || !std::isfinite(scale) || !aligned_to(ws, 16))
    return MDW_ERR_INVALID_ARG;
  if (ldq > (int64_t)1 << 36 || ldo > (int64_t)1 << 36) return MDW_ERR_UNSUPPORTED_SHAPE;
  if (ws_bytes < mdw_linear_attention_workspace_bytes(state, B, T, qk_heads, max_new)) return MDW_ERR_WORKSPACE_TOO_SMALL;
  const int sms = sm_count(current_device());
  if (sms <= 0) return MDW_ERR_CUDA;
  const LinearPlan w = plan_of(static_cast<uint8_t*>(ws), B, D, sms).first;
  const bool chunks = max_new > kLinearShort;
  const LinearParams p{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                       log_decay, static_cast<__nv_bfloat16*>(out), ldq, ldk, ldv, ldd, ldo, state->slot_stride, state->s, row_start, slot_in,
                       slot_out, nullptr, status, scale, B, T, state->heads, state->heads / qk_heads, max_new, state->num_slots,
                       kLinearShort, chunks ? w.ok : nullptr, mdw_spin_budget()};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool windows = !chunks && max_new >= kLinearWindow;     // (linear.cuh)
  cudaError_t e = windows ? launch_windows(p, D, current_device(), s) : launch_step<true>(p, D, sms, s);
  if (e == cudaSuccess && chunks) e = launch_prompts(p, w, D, sms, current_device(), s);
  return e == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}

extern "C" mdw_status mdw_linear_state_advance(const mdw_linear_state* state, int32_t B, int32_t T, int32_t qk_heads,
                                               int32_t max_new, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                               const float* log_decay, int64_t ldd, const int32_t* row_start,
                                               const uint64_t* accepted, const int32_t* slot_in,
                                               const int32_t* slot_out, uint32_t* status, mdw_stream_t stream) {
  const mdw_status st = check_linear_call(state, B, T, qk_heads, max_new, k, ldk, v, ldv, log_decay, ldd, row_start, slot_in, status);
  if (st != MDW_OK) return st;
  if (max_new > MDW_MAX_TREE || !aligned_to(accepted, 8) || !aligned_to(slot_out, 4)) return MDW_ERR_INVALID_ARG;
  const int sms = sm_count(current_device());
  if (sms <= 0) return MDW_ERR_CUDA;
  const LinearParams p{nullptr, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), log_decay, nullptr, 0, ldk, ldv,
                       ldd, 0, state->slot_stride, state->s, row_start, slot_in, slot_out, accepted, status, 0.f, B, T, state->heads,
                       state->heads / qk_heads, max_new, state->num_slots, 0, nullptr, 0};
  return launch_step<false>(p, state->head_dim, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MDW_OK : MDW_ERR_CUDA;
}
