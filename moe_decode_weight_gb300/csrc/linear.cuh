// Shared by the linear-attention kernels (linear_step.cu: single rows, linear_prompt.cu: chunks of rows, linear_tree.cu):
// parameters, a request's rows and slots.
#pragma once

#include "mdw_attn.cuh"

namespace mdw {

struct LinearParams {
  const __nv_bfloat16* q;          // [T][Hqk][D]
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;          // [T][H][D]
  const float* decay;              // [T][H] (row stride ldd), or [H] with ldd = 0
  __nv_bfloat16* out;
  int64_t ldq, ldk, ldv, ldd, ldo, slot_stride;
  float* s;
  const int32_t* row_start;
  const int32_t* slot_in;
  const int32_t* slot_out;         // null: nothing is stored
  const uint64_t* bits;            // per row the nodes it comes after (trees), per request the accepted rows
  uint32_t* status;
  float scale;
  int B, T, H, share, max_new, num_slots;
  int short_rows;                  // requests of more rows are left to the other kernel
  int32_t* ok;                     // [B] whether a request is sound, for the kernels that follow; or null
  long long spin_budget;
  int wide;                        // rows of out lie on 32-byte boundaries
};

// Rows of a chunk; least chunks of a segment, and its pieces in the first pass. Requests of up to kLinearShort rows take them one by one (in calls
// with longer ones; else see below): rows then cost 0.5 us (3 requests of 32 heads) to 5 us (48) each, and chunks of 128 rows as much for one row
// as for all: the two are even at 20 rows of 3 requests (both 22 us), 16 of 8 (30 us), 11 of 48 (86 us; 16 rows one by one 110). A call of
// few rows is one launch then.
constexpr int kLinearChunk = 128, kLinearShort = 16, kLinearSegment = 4, kLinearPieces = 3;
// Calls of at most 16 rows a request, and possibly of so many, take the products on mma.sync instead of row by row: whatever the rows, 48 requests
// of 32 heads 69 to 71 us (row by row 4 rows 54, 8 69, 12 89, 16 110), 10 26 (20, 25, 30, 34), 3 14 (13, 16, 18, 20), one of 20 heads 13.5 (9,
// 11, 13, 15.5).
// max_new is a bound only, and where the rows are fewer, row by row is as fast or faster; so not from 9 on.
constexpr int kLinearWindow = 12;

// A part of a request's rows, for all value heads, in the workspace.
struct LinearEntry {
  int row0, rows, slot_in, slot_out;
  int seg, segs;                   // segment of how many; in the first pass piece of how many, and one
  int set, pad;                    // set of states before the request; those after each of its pieces follow
};

// The workspace of mdw_linear_attention.
struct LinearPlan {
  int32_t* head;                   // units; units of the first pass; whether that was cut short; requests of several segments and heads
  int32_t* ok;
  LinearEntry* all;                // [B + blocks] every segment, longest first
  LinearEntry* first;              // [3 blocks] pieces of segments whose state others start from
  LinearEntry* joins;              // [blocks] requests of several segments
  float* logs;                     // [3 blocks] log decay of a piece, by set and head
  float* states;                   // [3 blocks][D][D] by set and head
};
// Requests of up to kLinearShort rows, by the kernel of linear_tree.cu.
cudaError_t launch_windows(const LinearParams& p, int D, int dev, cudaStream_t s);
cudaError_t launch_prompts(const LinearParams& p, const LinearPlan& w, int D, int grid, int dev, cudaStream_t s);

// Rows [row0, row0 + n) and slots of a request.
struct LinearRequest {
  int row0, n, in, out;
};

// Request b, read by all threads of a block together; false (for all) if it has to be skipped. A slot that is
// stored to by one request and read or stored to by another one would make results depend on timing, so every
// block looks through the list of slots: B loads of 4 bytes from L2.
__device__ __forceinline__ bool linear_request(const LinearParams& p, int b, LinearRequest& r) {
  r.row0 = p.row_start[b];
  const int end = p.row_start[b + 1];
  r.in = p.slot_in[b];
  r.out = p.slot_out ? p.slot_out[b] : -1;
  int bad = 0;
  if (p.slot_out)
    for (int i = threadIdx.x; i < p.B; i += blockDim.x) {
      const int other = p.slot_out[i];
      bad |= i != b && other >= 0 && (other == r.in || other == r.out);
    }
  bad |= r.row0 < 0 || end < r.row0 || end > p.T || r.in < -1 || r.in >= p.num_slots || r.out < -1 || r.out >= p.num_slots;
  r.n = bad ? 0 : end - r.row0;
  bad |= r.n > p.max_new;
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) raise_status(p.status, MDW_ERR_DEVICE_BOUNDS);
  return !bad;
}

__device__ __forceinline__ float log_decay_of(const LinearParams& p, int row, int h) { return p.decay[(int64_t)row * p.ldd + h]; }

// S <- e^g S, with e^g - 1 where e^g is near 1: over a thousand tokens the rounding of e^g itself would add up.
struct Decay {
  float f;
  bool near;
  __device__ __forceinline__ explicit Decay(float g) : near(g > -0.5f && g < 0.5f) { f = near ? expm1f(g) : expf(g); }
};

// Pairs of fp32 numbers, which one instruction takes together.
struct Pair {
  uint64_t v;
  __device__ __forceinline__ Pair() {}
  __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ float2 floats() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
  return a;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c.v) : "l"(a.v), "l"(b.v));
  return c;
}

// ------------------------------------------------------------------ host

mdw_status check_linear_state(const mdw_linear_state* s);
// Sizes and pointers that the three calls share.
mdw_status check_linear_call(const mdw_linear_state* s, int32_t B, int32_t T, int32_t qk_heads, int32_t max_new, const void* k, int64_t ldk,
                             const void* v, int64_t ldv, const float* log_decay, int64_t ldd, const int32_t* row_start,
                             const int32_t* slot_in, const uint32_t* status);

}  // namespace mdw
