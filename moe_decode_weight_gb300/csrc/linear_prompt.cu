// mdw_linear_attention for requests of more rows than linear_step.cu takes one by one: chunks of 128 rows on tcgen05.
//
// Mathematics. With c_t the sum of the log decays from the chunk's first row to row t, and S the state before the chunk,
//   o_i = scale ( sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j + e^{c_i} S^T q_i ),
//   S'  = e^{c_last} S + sum_j k_j (e^{c_last - c_j} v_j)^T.
// Four products of a chunk: scores Q K^T (128 x 128), weighted by the decays, times V; Q times the state; K^T times
// the decayed values. Sums of log decays have 48 bits and only differences leave them; those within 32 rows are of fp32 sums from the start of
// the 32, so that weights are off by less than their rounding to bf16 even where each row's decay is e^-200. A row's outputs are summed before its factor
// e^{c_i} comes, in units of 2^-30 (the state as it is read) to 2^30, so that terms from 2^-96 to 2^96 keep their digits.
//
// Roundings to bf16, the operands' type: the weighted scores and the state as the outputs read it (outputs are off by 0.0024 of
// their norm instead of the 0.0017 of their own rounding). The decayed values enter the state's product as
// three bf16 numbers that hold 24 bits together, so a state carries the error of fp32 sums only; it is kept in registers.
//
// Split. A unit is a value head of a request; where these are fewer than the SMs, or one is far longer than the others, a
// request's rows are cut into segments: a first pass computes what each segment adds to the state, and a
// segment then starts from the sums before it. plan_kernel lays the units out, longest first, from the lengths on the
// device; block i takes units i, 2 G - 1 - i, 2 G + i, ... of G blocks, one on each SM.
//
// What bounds it: neither memory (50 to 58 % of its peak) nor the matrix unit (41 to 44 %) nor the issue of instructions (45 to 52 %), but
// the chain of a chunk: the outputs of the last one read the state, the state takes its products and is rounded, the tile of q is
// free and filled again, scores, weights, products with the values. It takes 6,000 to 7,000 cycles and only parts of two chunks overlap;
// heads whose decays pass 2^-60 within a chunk wait for q to be scaled too. Measured: 16,301 rows of 32 heads from an empty state 189 us
// (of them the first pass 46, its sums 10), 24 requests of up to 2,100 rows of 20 heads 131 us. Roles of a block:
//   warp 0       requests the tiles of q, k and v by TMA (swizzled, 128 rows x 128 bytes)
//   warp 1       issues the products for the state
//   warp 2       sums the decays of the next chunk
//   warp 3       issues the products for the outputs
//   warps 4-7    weight the scores, one thread a row
//   warps 8-11   the outputs, one thread a row
//   warps 12-19  the decayed values
//   warps 20-27  the state, two threads a column of it
#include <cuda.h>

#include <algorithm>

#include "linear.cuh"
#include "mdw_tcgen05.cuh"

namespace mdw {
namespace {

constexpr int kChunk = kLinearChunk, kConvertWarps = 8, kStateWarps = 8, kThreads = 32 * (12 + kConvertWarps + kStateWarps);
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kCentre = 30.f;                                 // (see Sums)
constexpr uint32_t kStateUnit = 0x30803080u;                    // 2^-kCentre, two bf16 numbers

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int head, int row) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
               :: "r"(dst), "l"(map), "r"(x), "r"(head), "r"(row), "r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 lanes x 8 columns of tensor memory: a thread has columns lane % 4 and lane % 4 + 4 of lanes lane / 4 and lane / 4 + 8.
__device__ __forceinline__ void tc_st_16x128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// Two fp32 numbers as bf16 (low half: a), and back.
__device__ __forceinline__ uint32_t pack(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ Pair unpack(uint32_t v) { return Pair(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
__device__ __forceinline__ uint32_t pack(Pair a) {
  const float2 f = a.floats();
  return pack(f.x, f.y);
}

// Products of two pairs of bf16 numbers.
__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A sum of log decays in two fp32 numbers, 48 bits: only differences of sums are used, and those of long ones would lose their digits.
// (64-bit additions take 16 cycles of issue each here, and the sums of a chunk took longer than all else.)
struct Sum {
  float hi, lo;
  // v * log2(e)
  static __device__ __forceinline__ Sum log2_of_e_to(float v) {
    const float h = v * 1.44269502162933349609375f;             // log2(e) = this + 1.9259629...e-8
    return {h, fmaf(v, 1.44269502162933349609375f, -h) + v * 1.92596303339e-8f};
  }
  __device__ __forceinline__ Sum operator+(Sum b) const {
    const float s = __fadd_rn(hi, b.hi), t = __fsub_rn(s, hi);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)), __fadd_rn(lo, b.lo));
    const float h = __fadd_rn(s, e);
    return {h, __fsub_rn(e, __fsub_rn(h, s))};
  }
  __device__ __forceinline__ float less(Sum b) const { return __fadd_rn(__fsub_rn(hi, b.hi), __fsub_rn(lo, b.lo)); }
  __device__ __forceinline__ float natural() const { return fmaf(hi, kLn2, lo * kLn2) + hi * -1.9046542e-9f; }
};

// Registers of a thread. A block starts with 72 for each of its seven groups of four warps, 504 together; the two groups that hold the
// state take more from what the others give up: 56 + 88 + 56 + 2 * 56 + 2 * 96 = 504.
template <int kCount> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kCount)); }
template <int kCount> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kCount)); }

// The kernels of a call start while the one before them ends, and wait here for its results.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ the units

__global__ void __launch_bounds__(1024) plan_kernel(const LinearParams p, const LinearPlan w, int blocks) {
  constexpr int kBuckets = 1024;                                // units of so many chunks (the last: and more)
  __shared__ int at[kBuckets], sums[32], sets, extra, joins;
  __shared__ unsigned long long total;
  const int tid = threadIdx.x;
  if (tid == 0) total = 0, sets = 0, extra = 0, joins = 0;
  at[tid] = 0;
  after_previous();
  __syncthreads();
  auto chunks_of = [&](int b) {
    const int n = p.row_start[b + 1] - p.row_start[b];
    return w.ok[b] && n > kLinearShort ? (n + kChunk - 1) / kChunk : 0;
  };
  unsigned long long mine = 0;
  for (int b = tid; b < p.B; b += blockDim.x) mine += chunks_of(b);
  if (mine) atomicAdd(&total, mine);
  __syncthreads();
  // A segment is at least an SM's share of all work, and four chunks: its start costs about one. (32 heads, one request with and without
  // segments: 1,000 rows 44 and 43 us, 1,500 47 and 56, 2,000 52 and 71, 4,000 73 and 126, 16,301 194 and 469; four of 1,000 rows 54
  // and 48, of 2,000 84 and 79, of 4,000 145 and 138: they fill the SMs without. At least eight chunks: 1,500 rows 59, 2,000 61, four of 1,000
  // rows 50; at least three: 46, 52, 54.) The first pass has all segments but each request's last, in three pieces each, so that it
  // fills the SMs too (16,301 rows: 4 segments, so 96 units of 32 chunks there or 288 of about 11 on 152 SMs: 202 us with one piece, 194).
  const long long share = max((long long)kLinearSegment, ((long long)total * p.H + blocks - 1) / blocks);
  auto cut = [&](int chunks, int& n) {                          // segments and the chunks of one
    n = (int)max(1ll, chunks / share);
    const int each = (chunks + n - 1) / n;
    n = (chunks + each - 1) / each;
    return each;
  };
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int chunks = chunks_of(b);
    if (!chunks) continue;
    int n;
    const int each = cut(chunks, n);                            // (in a statement of its own: it gives n)
    atomicAdd(&at[min(each, kBuckets - 1)], n);
  }
  __syncthreads();
  // first place of each bucket, the longest first (sums of all buckets above)
  const int own = at[kBuckets - 1 - tid];
  int sum = own;
  for (int m = 1; m < 32; m <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, m);
    if ((tid & 31) >= m) sum += up;
  }
  if ((tid & 31) == 31) sums[tid >> 5] = sum;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < 32; ++i) {
    if (i < tid >> 5) before += sums[i];
    all += sums[i];
  }
  __syncthreads();
  at[kBuckets - 1 - tid] = before + sum - own;
  __syncthreads();
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int chunks = chunks_of(b);
    if (!chunks) continue;
    int n;
    const int each = cut(chunks, n), rows = p.row_start[b + 1] - p.row_start[b];
    LinearEntry e{p.row_start[b], 0, p.slot_in[b], p.slot_out[b], 0, n, 0, 0};
    // sets of states: the one before the request, then what each piece of all segments but the last adds
    const int pieces = (n - 1) * kLinearPieces;
    if (n > 1) {
      e.set = atomicAdd(&sets, pieces + 1);
      w.joins[atomicAdd(&joins, 1)] = e;
    }
    const int to = atomicAdd(&at[min(each, kBuckets - 1)], n);
    for (int s = 0; s < n; ++s) {
      e.seg = s;
      e.row0 = p.row_start[b] + s * each * kChunk;
      e.rows = min(rows - s * each * kChunk, each * kChunk);
      w.all[to + s] = e;
    }
    for (int s = 0; s < pieces; ++s) {
      auto start = [&](int s) { return s / kLinearPieces * each + s % kLinearPieces * each / kLinearPieces; };
      w.first[atomicAdd(&extra, 1)] = LinearEntry{p.row_start[b] + start(s) * kChunk, (start(s + 1) - start(s)) * kChunk, p.slot_in[b], -1, s, pieces + 1, e.set, 0};
    }
  }
  __syncthreads();
  if (tid == 0) {
    w.head[0] = all * p.H;
    w.head[1] = extra * p.H;
    w.head[2] = 0;
    w.head[3] = joins * p.H;
  }
}

// The states at the starts of a request's segments from what each piece adds: block (request and head, part of the elements). A segment's pieces
// are asked for at once, those of the next one before these are summed.
constexpr int kSumsParts = 16;
__global__ void __launch_bounds__(256) sums_kernel(const LinearPlan w, int H, int elements) {
  after_previous();
  if ((int)blockIdx.x >= w.head[3]) return;
  const LinearEntry e = w.joins[blockIdx.x / H];
  const int h = blockIdx.x % H, i = (blockIdx.y * blockDim.x + threadIdx.x) * 4;
  if (i >= elements) return;
  auto at = [&](int set) { return reinterpret_cast<float4*>(w.states + ((int64_t)(e.set + set) * H + h) * elements + i); };
  float4 x[kLinearPieces], s = make_float4(0.f, 0.f, 0.f, 0.f);
  float logs[kLinearPieces];
  auto ask = [&](int seg) {
#pragma unroll
    for (int k = 0; k < kLinearPieces; ++k) {
      const int set = seg * kLinearPieces + k + 1;
      x[k] = *at(set);
      logs[k] = w.logs[(size_t)(e.set + set) * H + h];
    }
  };
  ask(0);
  for (int seg = 0; seg + 1 < e.segs; ++seg) {
    float4 now[kLinearPieces];
    float decays[kLinearPieces];
#pragma unroll
    for (int k = 0; k < kLinearPieces; ++k) now[k] = x[k], decays[k] = logs[k];
    if (seg + 2 < e.segs) ask(seg + 1);
#pragma unroll
    for (int k = 0; k < kLinearPieces; ++k) {
      if (seg == 0 && k == 0) {                                 // holds the request's own state
        s = now[0];
        continue;
      }
      const Decay f(decays[k]);
      s.x = fmaf(s.x, f.f, f.near ? s.x : 0.f) + now[k].x;
      s.y = fmaf(s.y, f.f, f.near ? s.y : 0.f) + now[k].y;
      s.z = fmaf(s.z, f.f, f.near ? s.z : 0.f) + now[k].z;
      s.w = fmaf(s.w, f.f, f.near ? s.w : 0.f) + now[k].w;
    }
    *at((seg + 1) * kLinearPieces) = s;
  }
}

// ------------------------------------------------------------------ the kernel

// Shared memory: a tile of q, two of k and of v, the state as the outputs read it (rows: columns of the state).
template <int D, bool kRows>
struct Shape {
  static constexpr int kTile = kChunk * D * 2, kHalves = D / 64;
  static constexpr int kStep = 16, kSteps = kChunk / kStep;     // rows of a step of the state's product
  static constexpr int kQ = 0, kK = kTile, kV = 3 * kTile, kS = 5 * kTile;
  static constexpr int kSmall = kS + D * D * 2, kBarriers = 35;
  static constexpr int kSmem = kSmall + 2 * (5 * kChunk * 4 + 28 * 4) + kBarriers * 8 + 32;   // sums, barriers, words
  // Tensor memory columns: scores (the weighted ones take their first half when D = 128), outputs, what a chunk adds to the state (a lane is a
  // column of the state), and four steps of decayed values, each in three parts.
  static constexpr int kOut = 256 - D, kAdd = 256, kParts = 384, kProb = D == 128 ? 0 : 128;
  static constexpr int kCols = D / 2;                           // rows of the state, a thread
};

// What the warps of a block take from the sums of a chunk's decays (in log2), and how the chunk lies.
struct alignas(16) Sums {
  float d[kChunk];                 // from the start of the row's 32 rows to the row
  float after[kChunk];             // factor from the row to the end of its 32 rows
  float rest[kChunk];              // factor from the row to the end of the chunk
  // A row's outputs are summed without its factor from the chunk's start, 2^c: what the row reads of the state counts 2^-30 (the state is
  // stored so), scores 2^(-c - 30), and the sum is scaled. Where c is below -60 a power of two of it, 2^down, is left to the row of q
  // instead. So no row's sum is off its outputs by more than 2^30 either way: without the 2^-30, scores would count up to 2^60.
  float lift[kChunk];              // down - c - 30
  float from[kChunk];              // 2^(c - down + 30)
  float gap[16];                   // [block][earlier block]: from the end of the earlier one to the start of the block
  float base[4];                   // from the start of the chunk to the start of the block
  float factor;                    // of the chunk, less 1 if near
  int near, valid, more;           // valid rows; whether the block has another chunk
  int strong, pad[3];              // whether any row's power of two is not 1
};

template <int D, bool kRows>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const LinearParams p, const LinearPlan w, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<D, kRows>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, blocks = gridDim.x;
  Sums* sums_at = reinterpret_cast<Sums*>(smem + S::kSmall);   // [2]
  uint32_t bar = smem_u32(sums_at + 2);
  auto take = [&](int n) { const uint32_t r = bar; bar += 8 * n; return r; };
  const uint32_t q_full = take(1), q_free = take(1), q_ok = take(1), k_full = take(2), k_free = take(2), v_full = take(2), v_free = take(2), v_done = take(2);
  const uint32_t sums_full = take(2), sums_free = take(2), s_full = take(1), p_full = take(1), o_full = take(2), o_free = take(1);
  const uint32_t w_full = take(4), w_free = take(4), state_full = take(1), state_read = take(1);
  const uint32_t add_full = take(1), add_read = take(1), end = take(1);
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + (bar - base));
  volatile uint32_t* bad_values = words + 4;                    // [4], by chunk: whether values that are not finite were taken out
  volatile int* dead = reinterpret_cast<volatile int*>(words);
  after_previous();
  const int units = w.head[kRows ? 0 : 1];
  // a first pass that gave up leaves the whole call without the outputs of this one
  const bool failed = kRows && w.head[2] != 0;
  if ((int)blockIdx.x >= units || failed) return;               // the whole block
  if (base & 1023) {
    if (threadIdx.x == 0) {
      raise_status(p.status, MDW_ERR_UNSUPPORTED_SHAPE);
      if (!kRows) w.head[2] = 1;
    }
    return;
  }
  if (threadIdx.x == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    if (kRows) prefetch_map(&qmap);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_free + 8 * i, kRows ? 2 : 1);
      mbar_init(v_full + 8 * i, 1);
      mbar_init(v_free + 8 * i, kConvertWarps + (kRows ? 1 : 0));
      mbar_init(v_done + 8 * i, kConvertWarps);
      for (int j = i; j < 4; j += 2) {
        mbar_init(w_full + 8 * j, 4);
        mbar_init(w_free + 8 * j, 1);
      }
      mbar_init(sums_full + 8 * i, 1);
      mbar_init(sums_free + 8 * i, kConvertWarps + kStateWarps + (kRows ? 8 : 0));
    }
    for (const uint32_t b : {q_full, q_free, s_full, o_full, o_full + 8, state_read, add_full}) mbar_init(b, 1);
    mbar_init(end, kRows ? 2 : 1);
    for (const uint32_t b : {p_full, q_ok, o_free}) mbar_init(b, 4);
    mbar_init(state_full, kStateWarps);
    mbar_init(add_read, kStateWarps);
    *dead = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(words + 1)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, words[1], 0);
  // As mbar_wait(), in line: around a call the state's registers would go to memory and come back.
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (mbar_test(b, parity)) return;
    const long long t0 = clock64();
    do {
      if (*dead) return;
      if (clock64() - t0 > p.spin_budget) {
        *dead = 1;
        raise_status(p.status, MDW_ERR_TIMEOUT);
        return;
      }
    } while (!mbar_try(b, parity));
  };
  auto arrive = [&](uint32_t b) {                               // of the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };
  // Every role goes over the block's units and their chunks in the same order; g counts the chunks.
  auto unit_of = [&](int k) {                                   // the block's k-th unit; `units` or more: none
    return k * blocks + (k & 1 ? blocks - 1 - (int)blockIdx.x : (int)blockIdx.x);
  };
  auto entry_of = [&](int u) -> const LinearEntry& { return (kRows ? w.all : w.first)[u / p.H]; };
  auto each_unit = [&](auto&& unit) {
    int g = 0;
    for (int k = 0; unit_of(k) < units; ++k) {
      const int chunks = (entry_of(unit_of(k)).rows + kChunk - 1) / kChunk;
      unit(unit_of(k), chunks, g, k);
      g += chunks;
    }
  };

  // The roles; their order is that of the code, whose instructions seven warps a scheduler fetch in turn: of seven orders 189 us (this one) to
  // 199 for 16,301 rows, 132 to 138 for the 24 requests.
  if (warp >= 20) {
    // ---- the state: thread = column of it (lane of tensor memory), half of the rows
    more_registers<96>();
    const int quad = warp & 3, a = quad * 32 + lane, col0 = ((warp - 20) >> 2) * S::kCols;
    const bool holds = quad * 32 < D;
    const uint32_t lanes = (uint32_t)quad * 32 << 16;
    float s[S::kCols];
    auto at_state = [&](float* pool, int64_t first) { return pool + first + ((int64_t)col0 * D + a); };
    auto load_state = [&](const float* src) {
#pragma unroll
      for (int i = 0; i < S::kCols; ++i) s[i] = src[i * D];
    };
    auto store_state = [&](float* dst) {
#pragma unroll
      for (int i = 0; i < S::kCols; ++i) dst[i * D] = s[i];
    };
    auto set_at = [&](int set, int h) { return at_state(w.states, ((int64_t)set * p.H + h) * D * D); };
    auto publish = [&](int g) {                                 // the state as the outputs of chunk g read it
      if (g > 0) wait(state_read, (g - 1) & 1);
      if (holds)
#pragma unroll
        for (int i = 0; i < S::kCols; i += 8) {
          const int at = (col0 + i) >> 3;
          sts16(base + S::kS + (at >> 3) * (D * 128) + a * 128 + (((at & 7) ^ (a & 7)) << 4),
                make_uint4(times(pack(s[i], s[i + 1]), kStateUnit), times(pack(s[i + 2], s[i + 3]), kStateUnit), times(pack(s[i + 4], s[i + 5]), kStateUnit),
                           times(pack(s[i + 6], s[i + 7]), kStateUnit)));
        }
      fence_async_proxy();
      arrive(state_full);
    };
    each_unit([&](int u, int chunks, int g0, int k) {
#pragma unroll
      for (int i = 0; i < S::kCols; ++i) s[i] = 0.f;
      if (holds) {
        const int h = u % p.H;
        const LinearEntry e = entry_of(u);
        const int64_t own = (int64_t)h * D * D;
        if (e.seg == 0 && (!kRows || e.segs == 1)) {
          if (e.slot_in >= 0) load_state(at_state(p.s, e.slot_in * p.slot_stride + own));
          // (the last segment may store to the slot before the first one reads it)
          if (!kRows) store_state(set_at(e.set, h));
        } else if (kRows) {
          load_state(set_at(e.set + e.seg * kLinearPieces, h));
        }
      }
      if (kRows) publish(g0);
      for (int c = 0; c < chunks; ++c) {
        const int g = g0 + c;
        wait(sums_full + 8 * (g & 1), g >> 1 & 1);
        const Sums& sums = sums_at[g & 1];
        const float f = sums.factor;
        const float keep = sums.near ? 1.f : 0.f;
        arrive(sums_free + 8 * (g & 1));
        wait(add_full, g & 1);
        tc_fence_after();
        if (holds)
#pragma unroll
          for (int i = 0; i < S::kCols; i += 16) {
            float x[16];
            tc_ld16(x, tmem + lanes + S::kAdd + col0 + i);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              // (keep: 1 where the factor is given less 1; a branch would cost the registers of both ways)
              const Pair was(s[i + j], s[i + j + 1]), now = fma(was, Pair(keep, keep), fma(was, Pair(f, f), Pair(x[j], x[j + 1])));
              s[i + j] = now.floats().x;
              s[i + j + 1] = now.floats().y;
            }
          }
        tc_fence_before();
        arrive(add_read);
        if (kRows && c + 1 < chunks) publish(g + 1);
      }
      if (holds && !*dead) {
        const int h = u % p.H;
        const LinearEntry e = entry_of(u);
        if (!kRows) store_state(set_at(e.set + e.seg + 1, h));
        else if (e.seg == e.segs - 1 && e.slot_out >= 0) store_state(at_state(p.s, e.slot_out * p.slot_stride + (int64_t)h * D * D));
      }
    });
  } else if (warp >= 12 && warp < 20) {
    // ---- values: 16 columns x 16 rows at a time
    fewer_registers<56>();
    const int quad = warp & 3, group = (warp - 12) >> 2, id = threadIdx.x & 127;
    const bool holds = quad * 32 < D;
    const uint32_t lanes = (uint32_t)quad * 32 << 16;
    // The decayed values of a step of rows as three bf16 numbers, by 4 of the warps (the others have the next step), into tensor
    // memory: a lane is a column of the values, which the transposing loads from shared memory give. A thread has two neighbouring
    // rows of 8 and two of the other 8.
    auto convert = [&](int g, int step) {
      const int slot = g & 1, use = g * S::kSteps + step;
      const int at_slot = step & 3;
      if (step == group) {
        wait(sums_full + 8 * slot, g >> 1 & 1);
        wait(v_full + 8 * slot, g >> 1 & 1);
      }
      const Sums& sums = sums_at[slot];
      const int row = step * S::kStep, valid = sums.valid;
      const uint32_t v_at = base + S::kV + slot * S::kTile, k_at = base + S::kK + slot * S::kTile;
      // of a row and a column's piece of 8
      auto place = [&](int r, int piece) { return (uint32_t)((piece >> 3) * (kChunk * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4)); };
      uint32_t word[2][4];                                      // [16 columns][rows 0-7: columns 0-7, 8-15; rows 8-15: the same]
      if (holds)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          ldmatrix_trans(word[n], v_at + place(row + (lane & 7) + (lane >> 4) * 8, quad * 4 + 2 * n + (lane >> 3 & 1)));
      const float2 r0 = *reinterpret_cast<const float2*>(&sums.rest[row + 2 * (lane & 3)]), r1 = *reinterpret_cast<const float2*>(&sums.rest[row + 8 + 2 * (lane & 3)]);
      if (row + S::kStep > valid) {
        // rows behind the last are another request's, or nobody's
        wait(k_full + 8 * slot, g >> 1 & 1);
        for (int i = id; i < S::kStep * (D / 8); i += 128)
          if (row + i / (D / 8) >= valid) {
            const uint32_t at = place(row + i / (D / 8), i % (D / 8));
            sts16(v_at + at, make_uint4(0u, 0u, 0u, 0u));
            sts16(k_at + at, make_uint4(0u, 0u, 0u, 0u));
          }
        fence_async_proxy();
        const int t = row + 2 * (lane & 3);
        const uint32_t keep0 = t + 1 < valid ? ~0u : t < valid ? 0xffffu : 0u, keep1 = t + 9 < valid ? ~0u : t + 8 < valid ? 0xffffu : 0u;
#pragma unroll
        for (int n = 0; n < 2; ++n) word[n][0] &= keep0, word[n][1] &= keep0, word[n][2] &= keep1, word[n][3] &= keep1;
      }
      Pair x[8], none(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = unpack(word[i >> 2][i & 3]) * (i & 2 ? Pair(r1.x, r1.y) : Pair(r0.x, r0.y));
        none = fma(x[i], Pair(0.f, 0.f), none);
      }
      if (kRows && holds && !(none.floats().x == 0.f && none.floats().y == 0.f)) {
        // values that are not finite leave the product with the scores, where they would reach earlier rows too
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
          const int r = row + 2 * (lane & 3) + (i & 1) + (i >> 2 & 1) * 8, c = quad * 32 + (i >> 3) * 16 + (i >> 1 & 1) * 8 + (lane >> 2);
          uint16_t* at = reinterpret_cast<uint16_t*>(smem + S::kV + slot * S::kTile + place(r, c >> 3)) + (c & 7);
          if ((*at & 0x7f80) == 0x7f80) *at = 0;
        }
        bad_values[g & 3] = 1;
        fence_async_proxy();
      }
      if (use >= 4) wait(w_free + 8 * at_slot, (use >> 2 & 1) ^ 1);
      tc_fence_after();
      // 8 leading bits at a time: the three parts are the whole number (infinities are themselves, and NaN)
      if (holds)
#pragma unroll
        for (int part = 2; part >= 0; --part) {
          uint32_t to[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = x[i].floats();
            to[i] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
            if (part > 0) x[i] = fma(Pair(__uint_as_float(__float_as_uint(f.x) & 0xffff0000u), __uint_as_float(__float_as_uint(f.y) & 0xffff0000u)), Pair(-1.f, -1.f), x[i]);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
            tc_st_16x128(tmem + lanes + ((uint32_t)n * 16 << 16) + S::kParts + 8 * (3 * at_slot + part), to[4 * n], to[4 * n + 1], to[4 * n + 2], to[4 * n + 3]);
        }
      tc_wait_st();
      tc_fence_before();
      arrive(w_full + 8 * at_slot);
    };
    bool more = true;
    for (int g = 0; more; ++g) {
#pragma unroll 1
      for (int step = group; step < S::kSteps; step += 2) convert(g, step);
      more = sums_at[g & 1].more;
      arrive(sums_free + 8 * (g & 1));
      arrive(v_done + 8 * (g & 1));
      arrive(v_free + 8 * (g & 1));
      if (__any_sync(0xffffffffu, *dead)) break;                // (more may be anything)
    }
  } else if (warp >= 8 && warp < 12) {
    // ---- outputs: thread = row
    fewer_registers<56>();
    if (kRows) {
      const int own = warp & 3, row = own * 32 + lane;
      const uint32_t lanes = (uint32_t)own * 32 << 16;
      // (a scale whose product with the row's factor could leave fp32 comes after it)
      const float size = fabsf(p.scale);
      const bool apart = size > 0x1p60f || (size < 0x1p-60f && size > 0.f);
      each_unit([&](int u, int chunks, int g0, int k) {
        const int h = u % p.H, row0 = entry_of(u).row0;
        for (int c = 0; c < chunks; ++c) {
          const int g = g0 + c, slot = g & 1, first = row0 + c * kChunk;
          wait(sums_full + 8 * slot, g >> 1 & 1);
          const float f = (apart ? 1.f : p.scale) * sums_at[slot].from[row];
          const int valid = sums_at[slot].valid;
          arrive(sums_free + 8 * slot);
          wait(v_done + 8 * slot, g >> 1 & 1);
          wait(o_full + 8 * slot, g >> 1 & 1);
          tc_fence_after();
          const bool alive = !*dead, bad = alive && bad_values[g & 3] != 0, store = alive && row < valid;   // (not alive: valid may be anything)
          __nv_bfloat16* dst = p.out + (int64_t)(first + min(row, valid - 1)) * p.ldo + (int64_t)h * D;
          float o[16];
          tc_ld16(o, tmem + lanes + S::kOut);
#pragma unroll 1
          for (int i = 0; i < D; i += 16) {
            uint32_t x[8];
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 2) x[j / 2] = pack(Pair(o[j], o[j + 1]) * Pair(f, f));
            if (apart)
#pragma unroll
              for (int j = 0; j < 16; j += 2) x[j / 2] = pack(Pair(o[j], o[j + 1]) * Pair(f, f) * Pair(p.scale, p.scale));
            if (i + 16 < D) tc_ld16(o, tmem + lanes + S::kOut + i + 16);   // (the next ones while these are stored)
            if (bad) {
              // rare: values that are not finite, which were left out; they make what comes after them in their column so
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const __nv_bfloat16* v = p.v + (int64_t)first * p.ldv + (int64_t)h * D + i + j;
#pragma unroll 1
                for (int before = 0; before <= min(row, valid - 1); ++before)
                  if (!isfinite(__bfloat162float(v[(int64_t)before * p.ldv]))) x[j / 2] |= j & 1 ? 0x7fff0000u : 0x7fffu;
              }
            }
            if (store) {
              if (p.wide) {                                     // rows on 32-byte boundaries
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                             :: "l"(dst + i), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]) : "memory");
              } else {
                *reinterpret_cast<uint4*>(dst + i) = make_uint4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4*>(dst + i + 8) = make_uint4(x[4], x[5], x[6], x[7]);
              }
            }
          }
          tc_fence_before();
          arrive(o_free);
        }
      });
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- weights of the scores: thread = row; 32 columns at a time, none above the diagonal
    more_registers<88>();
    if (kRows) {
      const int own = warp & 3, row = own * 32 + lane;
      const uint32_t lanes = (uint32_t)own * 32 << 16;
      each_unit([&](int u, int chunks, int g0, int k) {
        for (int c = 0; c < chunks; ++c) {
          const int g = g0 + c;
          wait(sums_full + 8 * (g & 1), g >> 1 & 1);
          const Sums& sums = sums_at[g & 1];
          if (!sums.strong) arrive(q_ok);
          wait(s_full, g & 1);
          tc_fence_after();
          if (sums.strong) {
            // (before the scores take their registers, four loads at a time: one, four, eight at a time 216, 190, 198 us for 16,301 rows)
            const float down = rintf(sums.base[own] + sums.d[row] + sums.lift[row]) + kCentre;
            if (down < 0.f) {
              const uint32_t f = pack(exp2f(down), exp2f(down));
#pragma unroll 1
              for (int i = 0; i < D / 8; i += 4) {
                auto at = [&](int i) { return base + S::kQ + (i >> 3) * (kChunk * 128) + row * 128 + (((i & 7) ^ (row & 7)) << 4); };
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = lds16(at(i + j));
#pragma unroll
                for (int j = 0; j < 4; ++j) sts16(at(i + j), make_uint4(times(x[j].x, f), times(x[j].y, f), times(x[j].z, f), times(x[j].w, f)));
              }
            }
            fence_async_proxy();
            arrive(q_ok);
          }
          float v[32];
          tc_ld32(v, tmem + lanes);
          const float d = sums.d[row] + sums.lift[row];
          tc_wait_ld();
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t packed[16];
            if (b < own) {
              const float f = exp2_fast(d + sums.gap[4 * own + b]);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 a = *reinterpret_cast<const float4*>(&sums.after[32 * b + i]);
                packed[i / 2] = pack(Pair(v[i], v[i + 1]) * (Pair(a.x, a.y) * Pair(f, f)));
                packed[i / 2 + 1] = pack(Pair(v[i + 2], v[i + 3]) * (Pair(a.z, a.w) * Pair(f, f)));
              }
              tc_ld32(v, tmem + lanes + 32 * (b + 1));          // (the next ones while these are stored)
            } else if (b == own) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 a = *reinterpret_cast<const float4*>(&sums.d[32 * b + i]);
                packed[i / 2] = pack(i <= lane ? v[i] * exp2_fast(d - a.x) : 0.f, i + 1 <= lane ? v[i + 1] * exp2_fast(d - a.y) : 0.f);
                packed[i / 2 + 1] = pack(i + 2 <= lane ? v[i + 2] * exp2_fast(d - a.z) : 0.f, i + 3 <= lane ? v[i + 3] * exp2_fast(d - a.w) : 0.f);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) packed[i] = 0;
            }
            tc_wait_ld();                                       // (before these go to where they came from)
            tc_st16(tmem + lanes + S::kProb + 16 * b, packed);
          }
          tc_wait_st();
          tc_fence_before();
          arrive(p_full);
          arrive(sums_free + 8 * (g & 1));
        }
      });
    }
  } else {
    fewer_registers<56>();                                      // (one instruction, of the four warps together)
    if (warp == 0) {
      // ---- copies
      int asked[3] = {0, 0, 0};                                   // tiles of k, v and q
      each_unit([&](int u, int chunks, int g0, int k) {
        const int h = u % p.H, row0 = entry_of(u).row0;
        for (int c = 0; c < chunks; ++c) {
          const int g = g0 + c, slot = g & 1, row = row0 + c * kChunk;
          const uint32_t again = (g >> 1 & 1) ^ 1;
          auto load = [&](int which, uint32_t to, const CUtensorMap* map, uint32_t full, uint32_t free, uint32_t parity, int head) {
            wait(free, parity);
            if (__any_sync(0xffffffffu, *dead)) return;
            if (lane == 0) {
              mbar_arrive_tx(full, S::kTile);
#pragma unroll
              for (int i = 0; i < S::kHalves; ++i) tma_load(to + i * (kChunk * 128), map, full, 64 * i, head, row);
            }
            __syncwarp();
            ++asked[which];
          };
          load(1, base + S::kV + slot * S::kTile, &vmap, v_full + 8 * slot, v_free + 8 * slot, again, h);
          load(0, base + S::kK + slot * S::kTile, &kmap, k_full + 8 * slot, k_free + 8 * slot, again, h / p.share);
          if (kRows) load(2, base + S::kQ, &qmap, q_full, q_free, (g & 1) ^ 1, h / p.share);
        }
      });
      // every copy arrives before the block ends, also where a wait ran out
      for (int i = 0; i < 2; ++i) {
        const int k = (asked[0] + 1 - i) >> 1, v = (asked[1] + 1 - i) >> 1;
        if (k > 0) mbar_drain_inline(k_full + 8 * i, (k - 1) & 1);
        if (v > 0) mbar_drain_inline(v_full + 8 * i, (v - 1) & 1);
      }
      if (asked[2] > 0) mbar_drain_inline(q_full, (asked[2] - 1) & 1);
    } else if (warp == 1) {
      // ---- products for the state
      each_unit([&](int u, int chunks, int g0, int k) {
        for (int c = 0; c < chunks; ++c) {
          const int g = g0 + c, slot = g & 1;
          const uint32_t k_at = base + S::kK + slot * S::kTile;
          wait(k_full + 8 * slot, g >> 1 & 1);
          if (g > 0) wait(add_read, (g - 1) & 1);                 // the sums of the last chunk are out of their columns
#pragma unroll 1
          for (int step = 0; step < S::kSteps; ++step) {
            const int use = g * S::kSteps + step, at = use & 3;
            wait(w_full + 8 * at, use >> 2 & 1);
            tc_fence_after();
            if (elect_one()) {
              // the smallest part of the values is summed first
              const uint32_t kl = operand_low(k_at + step * (S::kStep * 128), kChunk * 128);
#pragma unroll
              for (int part = 0; part < 3; ++part)
                tc_mma_tmem(tmem + S::kAdd, tmem + S::kParts + 8 * (3 * at + part), kl, mma_shape(true, true, D), step > 0 || part > 0);
              tc_commit(w_free + 8 * at);
              if (step == S::kSteps - 1) {
                tc_commit(add_full);
                tc_commit(k_free + 8 * slot);
              }
            }
            __syncwarp();
          }
        }
      });
      if (elect_one()) tc_commit(end);                            // (by the thread that issued the products)
      __syncwarp();
      mbar_drain_inline(end, 0);                                  // nothing is in flight when the columns are given back
    } else if (warp == 3) {
      // ---- products for the outputs
      if (kRows) {
        each_unit([&](int u, int chunks, int g0, int k) {
          for (int c = 0; c < chunks; ++c) {
            const int g = g0 + c, slot = g & 1;
            const uint32_t ql = operand_low(base + S::kQ, 16), out = tmem + S::kOut;
            wait(k_full + 8 * slot, g >> 1 & 1);
            wait(q_full, g & 1);
            if (g > 0) wait(o_full + 8 * (slot ^ 1), (g - 1) >> 1 & 1);   // (the weighted scores lie in the scores' columns)
            tc_fence_after();
            if (elect_one()) {
              const uint32_t kl = operand_low(base + S::kK + slot * S::kTile, 16);
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint32_t off = ((i >> 2) * (kChunk * 128) + (i & 3) * 32) >> 4;
                tc_mma(tmem, ql + off, kl + off, mma_shape(true, false, kChunk), i > 0);
              }
              tc_commit(s_full);
              tc_commit(k_free + 8 * slot);
            }
            __syncwarp();
            wait(q_ok, g & 1);
            wait(state_full, g & 1);
            wait(o_free, (g & 1) ^ 1);
            tc_fence_after();
            if (elect_one()) {
              const uint32_t sl = operand_low(base + S::kS, 16);
#pragma unroll
              for (int i = 0; i < D / 16; ++i)
                tc_mma(out, ql + (((i >> 2) * (kChunk * 128) + (i & 3) * 32) >> 4), sl + (((i >> 2) * (D * 128) + (i & 3) * 32) >> 4), mma_shape(true, false, D), i > 0);
              tc_commit(state_read);
              tc_commit(q_free);
            }
            __syncwarp();
            wait(p_full, g & 1);
            wait(v_done + 8 * slot, g >> 1 & 1);                  // values that are not finite, and rows behind the last, are out of the tile
            tc_fence_after();
            if (elect_one()) {
              const uint32_t vl = operand_low(base + S::kV + slot * S::kTile, kChunk * 128);
#pragma unroll
              for (int i = 0; i < kChunk / 16; ++i)
                tc_mma_tmem(out, tmem + S::kProb + 8 * i, vl + i * (2048 >> 4), mma_shape(true, true, D), true);
              tc_commit(o_full + 8 * slot);
              tc_commit(v_free + 8 * slot);
            }
            __syncwarp();
          }
        });
        if (elect_one()) tc_commit(end);                            // (by the thread that issued the products)
        __syncwarp();
        mbar_drain_inline(end, 0);
      }
    } else {
      // ---- sums of the decays: a lane has four rows
      each_unit([&](int u, int chunks, int g0, int k) {
        const int h = u % p.H;
        const LinearEntry e = entry_of(u);
        const bool others = unit_of(k + 1) < units;
        Sum unit{0.f, 0.f};
        auto ask = [&](int c, int i) {
          const int row = c * kChunk + 4 * lane + i;
          return row < e.rows ? log_decay_of(p, e.row0 + row, h) : 0.f;
        };
        float next[4] = {ask(0, 0), ask(0, 1), ask(0, 2), ask(0, 3)};
        for (int c = 0; c < chunks; ++c) {
          const int g = g0 + c;
          Sum x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = next[i];
            if (v < -200.f) v = -200.f;                           // below every fp32 number, and sums stay finite
            x[i] = Sum::log2_of_e_to(v);
          }
          if (c + 1 < chunks)
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i] = ask(c + 1, i);
#pragma unroll
          for (int i = 1; i < 4; ++i) x[i] = x[i - 1] + x[i];
          Sum sum = x[3];
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const Sum more = Sum{__shfl_up_sync(0xffffffffu, sum.hi, m), __shfl_up_sync(0xffffffffu, sum.lo, m)} + sum;
            if (lane >= m) sum = more;
          }
          auto of_lane = [&](Sum v, int l) { return Sum{__shfl_sync(0xffffffffu, v.hi, l), __shfl_sync(0xffffffffu, v.lo, l)}; };
          Sum before = of_lane(sum, lane - 1 & 31);
          if (lane == 0) before = Sum{0.f, 0.f};
          const Sum last = of_lane(sum, 31), stop = of_lane(sum, lane | 7), start = of_lane(before, lane & ~7);
          float d[4], after[4], rest[4], from[4], lift[4];
          bool strong = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Sum c_t = before + x[i];
            d[i] = c_t.less(start);
            after[i] = exp2f(stop.less(c_t));
            rest[i] = exp2f(last.less(c_t));
            const float down = c_t.hi < -60.f ? floorf(c_t.hi) + 60.f : 0.f;
            strong |= down != 0.f;
            lift[i] = Sum{down - kCentre, 0.f}.less(c_t);
            from[i] = exp2f(-lift[i]);
          }
          // [lane >> 2][lane & 3], lanes below 16
          const float gap = of_lane(before, (lane >> 2 & 3) * 8).less(of_lane(sum, (lane & 3) * 8 + 7));
          strong = __any_sync(0xffffffffu, strong);
          const Decay whole(last.natural());
          const bool more = c + 1 < chunks || others;
          wait(sums_free + 8 * (g & 1), (g >> 1 & 1) ^ 1);
          Sums& sums = sums_at[g & 1];
          *reinterpret_cast<float4*>(&sums.d[4 * lane]) = make_float4(d[0], d[1], d[2], d[3]);
          *reinterpret_cast<float4*>(&sums.after[4 * lane]) = make_float4(after[0], after[1], after[2], after[3]);
          *reinterpret_cast<float4*>(&sums.rest[4 * lane]) = make_float4(rest[0], rest[1], rest[2], rest[3]);
          *reinterpret_cast<float4*>(&sums.from[4 * lane]) = make_float4(from[0], from[1], from[2], from[3]);
          *reinterpret_cast<float4*>(&sums.lift[4 * lane]) = make_float4(lift[0], lift[1], lift[2], lift[3]);
          if ((lane & 7) == 0) sums.base[lane >> 3] = start.hi;
          if (lane < 16) sums.gap[lane] = gap;
          if (lane == 0) {
            sums.factor = whole.f;
            sums.near = whole.near;
            sums.valid = min(e.rows - c * kChunk, kChunk);
            sums.more = more;
            bad_values[g & 3] = 0;                                // (the outputs of the chunk four before were taken before the weights of the one after)
            sums.strong = strong;
          }
          if (!kRows) unit = unit + last;
          arrive(sums_full + 8 * (g & 1));
        }
        if (!kRows && lane == 0) w.logs[(size_t)(e.set + e.seg + 1) * p.H + h] = unit.natural();
      });
    }
  }
  tc_fence_before();
  __syncthreads();
  if (!kRows && threadIdx.x == 0 && *dead) w.head[2] = 1;
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ host

// Rows [heads][d] as [T][heads][d]; a box is 128 rows of 64 elements of a head, swizzled.
bool encode_rows(CUtensorMap* map, const void* data, int64_t ld, int heads, int d, int T) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T}, strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, 1, kChunk}, ones[3] = {1, 1, 1};
  const EncodeTiledFn fn = encode_tiled();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(data), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... Args>
cudaError_t launch_next(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t launch(const LinearParams& p, const LinearPlan& w, const CUtensorMap (&m)[3], int grid, int dev, bool segments, cudaStream_t s) {
  cudaError_t e = allow_shared_memory<prompt_kernel<D, true>>(dev);
  if (e == cudaSuccess) e = allow_shared_memory<prompt_kernel<D, false>>(dev);
  if (e == cudaSuccess) e = launch_next(plan_kernel, dim3(1), 1024, 0, s, p, w, grid);
  if (segments) {
    if (e == cudaSuccess) e = launch_next(prompt_kernel<D, false>, dim3(grid), kThreads, Shape<D, false>::kSmem, s, p, w, m[0], m[1], m[2]);
    if (e == cudaSuccess) e = launch_next(sums_kernel, dim3(grid, kSumsParts), 256, 0, s, w, (int)p.H, D * D);
  }
  if (e == cudaSuccess) e = launch_next(prompt_kernel<D, true>, dim3(grid), kThreads, Shape<D, true>::kSmem, s, p, w, m[0], m[1], m[2]);
  return e;
}

}  // namespace

cudaError_t launch_prompts(const LinearParams& p0, const LinearPlan& w, int D, int grid, int dev, cudaStream_t s) {
  static_assert(kLinearPieces <= kLinearSegment, "a piece has a chunk at least");
  static_assert(sizeof(Sums) == 5 * kChunk * 4 + 28 * 4 && Shape<128, true>::kSmem <= 227 * 1024, "");
  LinearParams p = p0;
  p.wide = (reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)p.ldo * 2) % 32 == 0;
  CUtensorMap m[3];
  if (!encode_rows(&m[0], p.q, p.ldq, p.H / p.share, D, p.T) || !encode_rows(&m[1], p.k, p.ldk, p.H / p.share, D, p.T) ||
      !encode_rows(&m[2], p.v, p.ldv, p.H, D, p.T))
    return cudaErrorInvalidValue;
  // a request has two segments only where its chunks are two shares, a share being the chunks of all units over the SMs
  const bool segments = p.H <= grid / 2 && p.max_new > (2 * kLinearSegment - 1) * kChunk;
  return D == 128 ? launch<128>(p, w, m, grid, dev, segments, s) : launch<64>(p, w, m, grid, dev, segments, s);
}

}  // namespace mdw
