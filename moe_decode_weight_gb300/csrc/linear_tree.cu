// mdw_linear_tree_attention: the nodes of trees of drafted tokens against a state that stays as it is; and mdw_linear_attention for
// windows of 12 to 16 rows, as chains whose state is stored.
//
// Mathematics. Node i comes after the nodes j of its mask (itself among them). With e_ij the sum of the log decays of those of
// them that come after j, and e_i that of all,
//   o_i = scale ( e^{e_i} S^T q_i + sum_{j in mask_i} e^{e_ij} (q_i . k_j) v_j ).
// e_ij is summed from node i downwards, so a large sum never leaves a small difference. Windows: S <- e^{e_n} S + sum_j k_j (e^{e_nj} v_j)^T too.
//
// What bounds it up to 16 nodes is the state's 64 KB (heads of 128) from memory, so a block requests all of it before
// anything else: a thread's loads are whole operands of m16n8k16 products (four columns of it are four tiles' column, which
// only changes the order of the columns), turned into two bf16 numbers that hold 16 bits together. The scores and weights are
// products of the same kind, the weights as two bf16 numbers too. A block asks for its next unit's state as soon as it has used up the
// one before. Measured: 48 requests of up to 16 nodes and 32 heads 31 to 33 us, half of the copy rate; 12 requests of 64 nodes and 64 heads of 64 25 us,
// where the split states, two products each, and the barriers between the steps of a unit bound it (16 warps an SM).
// Windows of 16 rows, the same 48 requests: 71 us; the products for the state come between its use and the next one's loads.
#include <cmath>

#include "linear.cuh"

namespace mdw {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two numbers as the sum of two bf16 numbers each: 8 leading bits, and the rest rounded to 8 (a number that is not finite: itself and NaN).
__device__ __forceinline__ void split(float a, float b, uint32_t& high, uint32_t& low) {
  high = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  const Pair rest = fma(Pair(__uint_as_float(__float_as_uint(a) & 0xffff0000u), __uint_as_float(__float_as_uint(b) & 0xffff0000u)), Pair(-1.f, -1.f), Pair(a, b));
  low = pack(rest.floats().x, rest.floats().y);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}

// kTiles tiles of 16 nodes. 128 registers spill 456 bytes a thread with two tiles of 128, 256 where a state of 128 is stored, 192 with four tiles of 64.
template <int D, int kTiles>
struct Shape {
  static constexpr int kWarps = D == 128 || kTiles == 4 ? 8 : 4, kThreads = 32 * kWarps, kNodes = 16 * kTiles;
  static constexpr int kResident = kWarps == 4 ? 4 : D == 128 && kTiles == 4 ? 1 : 2;   // blocks an SM
  static constexpr int kColumns = D / 32, kSplits = kWarps / kColumns;   // groups of 32 columns, parts of the state's rows
  static constexpr int kRow = D + 8;                            // elements from one row to the next in shared memory: no bank twice
  static constexpr int kWeights = kNodes + 4, kSums = D + 4;
  // q, k and v; weights; sums (4 tiles: in q's and k's place); per node mask and e^{e_i}; per column a mask
  static constexpr bool kApart = kTiles < 4;
  static constexpr int kV = 2 * kRow * 2 * kNodes, kSumsAt = kApart ? kV + kNodes * kRow * 2 : 0;
  static constexpr int kWeightsAt = kV + kNodes * kRow * 2 + (kApart ? kNodes * kSums * 4 : 0);
  static_assert(kApart || kSums * 4 <= 2 * kRow * 2, "");
  static constexpr int kBits = kWeightsAt + kNodes * kWeights * 4, kSmem = kBits + kNodes * 12 + D * 8 + 32 + kNodes * 4;
};

// kStore: the nodes are a chain, and the state after them goes to slot_out.
template <int D, int kTiles, bool kStore>
__global__ void __launch_bounds__(Shape<D, kTiles>::kThreads, Shape<D, kTiles>::kResident) tree_kernel(const LinearParams p) {
  using S = Shape<D, kTiles>;
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16* qs = reinterpret_cast<__nv_bfloat16*>(smem);
  __nv_bfloat16* ks = qs + S::kNodes * S::kRow;
  __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(smem + S::kV);
  float* sums = reinterpret_cast<float*>(smem + S::kSumsAt);    // [node][D]
  float* weights = reinterpret_cast<float*>(smem + S::kWeightsAt);   // [node][node] e^{e_ij}, -1 where j is not seen; then weighted scores
  uint64_t* bits = reinterpret_cast<uint64_t*>(smem + S::kBits);
  uint64_t* odd = bits + S::kNodes;                             // per column the nodes whose value is not finite
  float* whole = reinterpret_cast<float*>(odd + D);             // e^{e_i}
  int* any_odd = reinterpret_cast<int*>(whole + S::kNodes);
  float* decay = reinterpret_cast<float*>(any_odd + 4);         // of all rows: factor, and 1 if it is given less 1
  float* rest = decay + 4;                                      // from a row to the end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, units = p.B * p.H;

  // ---- requests: a block has several units (request, head), and asks for the next one's data as soon as it has room for it
  struct Unit {
    int row0, n, in, h, out;                                    // n = 0 and out < 0: nothing to do
  };
  auto look = [&](int u) {
    Unit r{0, 0, -1, 0, -1};
    if (u >= units) return r;
    const int b = u / p.H;
    r.h = u - b * p.H;
    if (kStore) {
      LinearRequest x;
      if (linear_request(p, b, x) && (x.n > 0 || x.out >= 0)) r.row0 = x.row0, r.n = x.n, r.in = x.in, r.out = x.out;
      return r;
    }
    const int end = p.row_start[b + 1];
    r.row0 = p.row_start[b];
    r.in = p.slot_in[b];
    const bool bad = r.row0 < 0 || end < r.row0 || end > p.T || r.in < -1 || r.in >= p.num_slots || end - r.row0 > p.max_new;
    r.n = bad ? 0 : end - r.row0;
    if (bad && tid == 0) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
    return r;
  };
  // the state: warp = 32 columns and a part of the rows
  constexpr int kSteps = D / 16 / S::kSplits;                   // of 16 rows
  const int col0 = warp % S::kColumns * 32, part = warp / S::kColumns, row0 = part * (D / S::kSplits);
  float4 state[kSteps][4];
  auto ask_state = [&](const Unit& r) {
    if (kStore && r.in < 0)
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) state[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((r.n == 0 && r.out < 0) || r.in < 0) return;
    const float* src = p.s + r.in * p.slot_stride + (int64_t)r.h * D * D + (int64_t)(row0 + 2 * t) * D + col0 + 4 * g;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4* at = reinterpret_cast<const float4*>(src + (16 * k + (i & 1) + 8 * (i >> 1)) * D);
        state[k][i] = kStore ? __ldcs(at) : __ldg(at);          // (what is stored to is not read-only)
      }
  };
  auto store_state = [&](const Unit& r) {
    float* dst = p.s + r.out * p.slot_stride + (int64_t)r.h * D * D + (int64_t)(row0 + 2 * t) * D + col0 + 4 * g;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) __stcs(reinterpret_cast<float4*>(dst + (16 * k + (i & 1) + 8 * (i >> 1)) * D), state[k][i]);
  };
  // rows of q, k and v, zeros behind the last; two decays a lane; masks of a warp's rows, one a lane
  constexpr int kPieces = (S::kNodes * D / 8 + S::kThreads - 1) / S::kThreads, kMasks = S::kNodes / S::kWarps;   // of 8 elements, a thread
  constexpr bool kEarly = D == 64 || kTiles != 2;               // (else there are no registers for it before)
  uint4 piece[3][kPieces];
  float g0 = 0.f, g1 = 0.f;
  uint64_t mask = ~0ull;
  auto ask_rows = [&](const Unit& r) {
    if (r.n == 0) return;
    const int64_t qk = (int64_t)(r.h / p.share) * D;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = i * S::kThreads + tid, node = at / (D / 8), e = at % (D / 8) * 8;
      piece[0][i] = piece[1][i] = piece[2][i] = make_uint4(0u, 0u, 0u, 0u);
      if (node < r.n) {
        const int64_t row = r.row0 + node;
        piece[0][i] = *reinterpret_cast<const uint4*>(p.q + row * p.ldq + qk + e);
        piece[1][i] = *reinterpret_cast<const uint4*>(p.k + row * p.ldk + qk + e);
        piece[2][i] = *reinterpret_cast<const uint4*>(p.v + row * p.ldv + (int64_t)r.h * D + e);
      }
    }
    g0 = 2 * lane < r.n ? log_decay_of(p, r.row0 + 2 * lane, r.h) * kLog2e : 0.f;
    g1 = 2 * lane + 1 < r.n ? log_decay_of(p, r.row0 + 2 * lane + 1, r.h) * kLog2e : 0.f;
    if (p.bits && lane < kMasks && lane * S::kWarps + warp < r.n) mask = p.bits[r.row0 + lane * S::kWarps + warp];
  };

  for (int i = tid; i < D; i += S::kThreads) odd[i] = 0;
  if (tid == 0) *any_odd = 0;
  Unit r = look(blockIdx.x);
  ask_state(r);
  ask_rows(r);
  __syncthreads();                                              // (odd is cleared)
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit next = look(u + gridDim.x);
    if (r.n > 0) {
      // ---- weights: a warp's rows, sums from the row downwards
#pragma unroll 4
      for (int j = 0; j < kMasks; ++j) {
        const int i = j * S::kWarps + warp;
        const uint64_t own = __shfl_sync(0xffffffffu, mask, j);
        const uint64_t seen = i < r.n ? (own & ((1ull << i) - 1)) | 1ull << i : 0;
        const bool s0 = seen >> (2 * lane) & 1, s1 = seen >> (2 * lane + 1) & 1;
        const float x1 = s1 ? g1 : 0.f;
        float sum = (s0 ? g0 : 0.f) + x1;
#pragma unroll
        for (int m = 1; m < S::kNodes / 2; m <<= 1) {
          const float down = __shfl_down_sync(0xffffffffu, sum, m);
          if (lane + m < 32) sum += down;
        }
        float after = __shfl_down_sync(0xffffffffu, sum, 1);        // of all nodes after the lane's
        if (lane == 31) after = 0.f;
        if (2 * lane < S::kNodes) *reinterpret_cast<float2*>(&weights[i * S::kWeights + 2 * lane]) = make_float2(s0 ? exp2_fast(after + x1) : -1.f, s1 ? exp2_fast(after) : -1.f);
        if (lane == 0) {
          whole[i] = exp2_fast(sum);
          bits[i] = seen;
        }
        if (kStore && i == r.n - 1) {
          if (2 * lane < S::kNodes) *reinterpret_cast<float2*>(&rest[2 * lane]) = make_float2(exp2f(after + x1), exp2f(after));
          if (lane == 0) {
            const Decay all(sum * 0.6931471805599453f);
            decay[0] = all.f;
            decay[1] = all.near ? 1.f : 0.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = i * S::kThreads + tid, node = at / (D / 8), e = at % (D / 8) * 8;
        if (S::kNodes * D / 8 % S::kThreads != 0 && node >= S::kNodes) break;
        uint32_t v[4] = {piece[2][i].x, piece[2][i].y, piece[2][i].z, piece[2][i].w};
        const uint32_t m = 0x7f807f80u, one = 0x00800080u;          // (an exponent of ones and one more carry into the sign's place)
        if ((((v[0] & m) + one) | ((v[1] & m) + one) | ((v[2] & m) + one) | ((v[3] & m) + one)) & 0x80008000u) {
          // values that are not finite stay out of the product, where they would reach nodes that do not see them
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (const uint32_t x = v[j >> 1] >> (16 * (j & 1)); (x & 0x7f80u) == 0x7f80u) {
              v[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
              atomicOr(reinterpret_cast<unsigned long long*>(&odd[e + j]), 1ull << node);
            }
          *any_odd = 1;
        }
        *reinterpret_cast<uint4*>(qs + node * S::kRow + e) = piece[0][i];
        *reinterpret_cast<uint4*>(ks + node * S::kRow + e) = piece[1][i];
        // column 32 a + 4 x + j at 32 a + 8 j + x, the order of the state's columns
        __nv_bfloat16* to = vs + node * S::kRow + (e & ~31) + (e >> 2 & 7);
        *reinterpret_cast<uint32_t*>(to) = __byte_perm(v[0], v[2], 0x5410);
        *reinterpret_cast<uint32_t*>(to + 8) = __byte_perm(v[0], v[2], 0x7632);
        *reinterpret_cast<uint32_t*>(to + 16) = __byte_perm(v[1], v[3], 0x5410);
        *reinterpret_cast<uint32_t*>(to + 24) = __byte_perm(v[1], v[3], 0x7632);
      }
      __syncthreads();
      if (kTiles == 1) ask_rows(next);

      // ---- weighted scores, 16 nodes x 8 earlier ones at a time, as two bf16 numbers in the weights' place
      constexpr int kPairs = kTiles * (kTiles + 1);
      for (int u = warp; u < kPairs; u += S::kWarps) {
        int tile = 0;
        while ((tile + 1) * (tile + 2) <= u) ++tile;
        const int first = (u - tile * (tile + 1)) * 8;
        if (16 * tile >= r.n) break;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};   // two chains of products
        const __nv_bfloat16 *q = qs + (16 * tile + g) * S::kRow + 2 * t, *k_at = ks + (first + g) * S::kRow + 2 * t;
#pragma unroll
        for (int k = 0; k < D; k += 16) {
          const uint32_t a[4] = {lds(q + k), lds(q + k + 8 * S::kRow), lds(q + k + 8), lds(q + k + 8 * S::kRow + 8)};
          mma(k & 16 ? s2 : s, a, lds(k_at + k), lds(k_at + k + 8));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += s2[e];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float2* at = reinterpret_cast<float2*>(&weights[(16 * tile + g + 8 * e) * S::kWeights + first + 2 * t]);
          const float2 w = *at;
          uint32_t high, low;
          split(w.x < 0.f ? 0.f : s[2 * e] * w.x, w.y < 0.f ? 0.f : s[2 * e + 1] * w.y, high, low);
          *at = make_float2(__uint_as_float(high), __uint_as_float(low));
        }
      }

      // ---- what the nodes read of the state
      float acc[kTiles][4][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
      if (r.in >= 0) {
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
            for (int j = 0; j < 4; ++j) mma(acc[i][j], a, low[j][0], low[j][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma(acc[i][j], a, high[j][0], high[j][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const float f0 = whole[16 * i + g], f1 = whole[16 * i + g + 8];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j][0] *= f0, acc[i][j][1] *= f0, acc[i][j][2] *= f1, acc[i][j][3] *= f1;
        }
      }
      if (kStore && r.out >= 0) {
        // ---- the state after the rows, columns x rows: a thread's numbers of the state are those of its sums, and the values that the
        // outputs take as second operand are the first one here, times their decays in three bf16 numbers that hold all 24 bits
        const float2 r0 = *reinterpret_cast<const float2*>(&rest[2 * t]), r1 = *reinterpret_cast<const float2*>(&rest[2 * t + 8]);
        const float f = decay[0], same = decay[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t v[4], a[3][4];
          ldmatrix_trans(v, smem_at(vs + (lane & 15) * S::kRow + col0 + 16 * j + 8 * (lane >> 4)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {                         // 8 columns and 8 rows: v[column half * 2 + row half], a[row half * 2 + column half]
            Pair x = Pair(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u)) * (i & 1 ? Pair(r1.x, r1.y) : Pair(r0.x, r0.y));
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const uint32_t lo = __float_as_uint(x.floats().x), hi = __float_as_uint(x.floats().y);
              a[part][(i & 1) * 2 + (i >> 1)] = __byte_perm(lo, hi, 0x7632);
              x = fma(Pair(__uint_as_float(lo & 0xffff0000u), __uint_as_float(hi & 0xffff0000u)), Pair(-1.f, -1.f), x);
            }
          }
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t b[4];                                      // 16 rows of the state: the first 8 of them, the others
            ldmatrix_trans(b, smem_at(ks + (lane & 15) * S::kRow + row0 + 16 * k + 8 * (lane >> 4)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int part = 2; part >= 0; --part) mma(add, a[part], b[2 * i], b[2 * i + 1]);
              auto next_of = [&](float& s, float x) { s = fmaf(s, same, fmaf(s, f, x)); };
              float4 &s0 = state[k][2 * i], &s1 = state[k][2 * i + 1];
              next_of(j ? s0.z : s0.x, add[0]);
              next_of(j ? s1.z : s1.x, add[1]);
              next_of(j ? s0.w : s0.y, add[2]);
              next_of(j ? s1.w : s1.y, add[3]);
            }
          }
        }
        if (*any_odd)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (odd[col0 + 4 * g + j])
#pragma unroll
              for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) (&state[k][i].x)[j] = __int_as_float(0x7fffffff);
        store_state(r);
      }
      if (kEarly) ask_state(next);
      __syncthreads();

      // ---- weighted scores x values, 16 earlier nodes at a time, taken in turns by the warps of the same columns
#pragma unroll
      for (int from = 0; from < kTiles; ++from) {
        if ((from & 1 ? from ^ 2 : from) % S::kSplits != part && kTiles > 1) continue;
        if (kTiles == 1 && part != 0) continue;
        if (16 * from >= r.n) continue;
        uint32_t v[2][4];                                           // each: two tiles of 8 columns
#pragma unroll
        for (int j = 0; j < 2; ++j) ldmatrix_trans(v[j], smem_at(vs + (16 * from + (lane & 15)) * S::kRow + col0 + 16 * j + 8 * (lane >> 4)));
#pragma unroll
        for (int i = from; i < kTiles; ++i) {
          uint2 w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = *reinterpret_cast<const uint2*>(&weights[(16 * i + g + 8 * (e & 1)) * S::kWeights + 16 * from + 2 * t + 8 * (e >> 1)]);
          const uint32_t high[4] = {w[0].x, w[1].x, w[2].x, w[3].x}, low[4] = {w[0].y, w[1].y, w[2].y, w[3].y};
#pragma unroll
          for (int j = 0; j < 4; ++j) mma(acc[i][j], low, v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma(acc[i][j], high, v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1]);
        }
      }

      if (!kEarly) ask_state(next);

      // ---- the parts together; a thread's columns: col0 + 8 t .. + 7 of rows g and g + 8 of each tile
      const bool bad = *any_odd;
#pragma unroll
      for (int turn = S::kSplits - 1; turn >= 0; --turn) {
        if (part == turn)
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int node = 16 * i + g + 8 * e, col = col0 + 8 * t;
              float4* at = reinterpret_cast<float4*>(&sums[node * S::kSums + col]);
              float x[8] = {acc[i][0][2 * e], acc[i][1][2 * e], acc[i][2][2 * e], acc[i][3][2 * e],
                            acc[i][0][2 * e + 1], acc[i][1][2 * e + 1], acc[i][2][2 * e + 1], acc[i][3][2 * e + 1]};
              if (turn < S::kSplits - 1) {
                const float4 a = at[0], c = at[1];
                x[0] += a.x, x[1] += a.y, x[2] += a.z, x[3] += a.w, x[4] += c.x, x[5] += c.y, x[6] += c.z, x[7] += c.w;
              }
              if (turn > 0) {
                at[0] = make_float4(x[0], x[1], x[2], x[3]);
                at[1] = make_float4(x[4], x[5], x[6], x[7]);
              } else if (node < r.n) {
                if (bad)
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (odd[col + j] & bits[node]) x[j] = __int_as_float(0x7fffffff);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= p.scale;
                *reinterpret_cast<uint4*>(p.out + (int64_t)(r.row0 + node) * p.ldo + (int64_t)r.h * D + col) =
                    make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
              }
            }
        if (turn > 0 || !S::kApart) __syncthreads();
      }
      if (bad) {                                                // (of all threads)
        __syncthreads();
        for (int i = tid; i < D; i += S::kThreads) odd[i] = 0;
        if (tid == 0) *any_odd = 0;
        __syncthreads();
      }
      if (kTiles > 1) ask_rows(next);
    } else {
      if (kStore && r.out >= 0) store_state(r);
      ask_state(next);
      ask_rows(next);
    }
    r = next;
  }
}

template <int D, int kTiles, bool kStore>
cudaError_t launch(const LinearParams& p, int dev, cudaStream_t s) {
  using S = Shape<D, kTiles>;
  const cudaError_t e = allow_shared_memory<tree_kernel<D, kTiles, kStore>>(dev);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.H * p.B, most = (int64_t)S::kResident * sm_count(dev);
  tree_kernel<D, kTiles, kStore><<<(unsigned)(units < most ? units : most), S::kThreads, S::kSmem, s>>>(p);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch(const LinearParams& p, int dev, cudaStream_t s) {
  // as few tiles as the nodes need (48 requests of 32 heads, 16 nodes: one tile 40 us, two 53, four 71; 32 nodes: two 61, four 77)
  if (p.max_new <= 16) return launch<D, 1, false>(p, dev, s);
  return p.max_new <= 32 ? launch<D, 2, false>(p, dev, s) : launch<D, 4, false>(p, dev, s);
}

}  // namespace

cudaError_t launch_windows(const LinearParams& p, int D, int dev, cudaStream_t s) {
  return D == 128 ? launch<128, 1, true>(p, dev, s) : launch<64, 1, true>(p, dev, s);
}

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
