// Linear attention with a decay per head: shared declarations of its kernels.
//
//   S_t = alpha_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
// and, with A_t the gradient of S_t by everything behind token t,
//   A_t = alpha_{t+1} A_{t+1} + scale do_t q_t^T,
//   dq_t = scale S_t^T do_t,  dk_t = A_t^T v_t,  dv_t = A_t k_t,
//   dlog_alpha_t = alpha_t <S_{t-1}, A_t>.
//
// The recurrence is linear, so a sequence is cut into segments that are worked
// on side by side: what a segment adds to the state behind it (its sum) comes
// first, a short pass along the segments turns the sums into the states on
// entry, and then every segment runs with its own.  Segments are dealt by slot
// in the way of the gated delta rule's chunks (gdr.cuh), a segment in the place
// of a chunk.
//
// A segment's log decay is summed in float64 (token by token) or as an integer (in chunks; where only the way
// back wants it in float32, over at most 1536 tokens).
#pragma once

#include "gdr.cuh"

namespace llattn {

struct LaArgs {
  int B, H, Hk, T, dk, dv, n_seqs;  // n_seqs = 0: unpacked
  ll_dtype io;
  int per_head;  // log_alpha is [H], else [B,H,T]
  float scale;
  const int32_t* seq_starts;
  const void *q, *k, *v;
  const float *log_alpha, *state_in;
  // forward
  void* o;
  float* state_out;
  // backward
  const void* dout;
  const float* dstate_out;
  void *dq, *dkey, *dval;
  float *dlog_alpha, *dstate_in;
  void* ws;
  size_t ws_bytes;
  cudaStream_t stream;
  unsigned* err;
};

inline int la_sequences(const LaArgs& a) { return a.n_seqs ? a.n_seqs : a.B; }
inline GdrSeqs la_seqs(const LaArgs& a) {
  return GdrSeqs{a.n_seqs ? a.seq_starts : nullptr, la_sequences(a), a.T, a.H, a.Hk};
}
inline size_t la_slots(const LaArgs& a, int seg) {
  return a.n_seqs ? (size_t)(a.T / seg) + a.n_seqs : (size_t)a.B * (((size_t)a.T + seg - 1) / seg);
}
// Can a sequence have more than one segment?
inline bool la_split(const LaArgs& a, int seg) { return a.T > seg; }

// The segment of slot `c`: its sequence, number within it, first row and length;
// `seq_len` that of the sequence (0: nothing of it but its state, on its first
// slot).  False when no valid segment owns the slot.
struct LaSegment {
  int seq, num, row_b, start, n, seq_len;
};
__device__ __forceinline__ bool la_find(const GdrSeqs& s, int c, int seg, LaSegment& r, unsigned* err) {
  GdrSeq q;
  if (!s.starts) {
    const int per = (s.T + seg - 1) / seg;
    r.seq = c / per;
    r.num = c - r.seq * per;
    q = GdrSeq{r.seq, 0, s.T};
  } else {
    int lo = 0, hi = s.n - 1;  // the last sequence with base <= c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.starts[mid] / seg + mid <= c) lo = mid;
      else hi = mid - 1;
    }
    if (!gdr_seq(s, lo, q)) {
      if (err && threadIdx.x == 0) raise_error(err, kErrDeviceArg);
      return false;
    }
    r.seq = lo;
    r.num = c - (q.start / seg + lo);
    if (r.num < 0) return false;
  }
  const long long at = (long long)r.num * seg;
  r.row_b = q.row_b;
  r.seq_len = q.len;
  r.start = q.start + (int)(at < q.len ? at : 0);
  r.n = at < q.len ? (int)(q.len - at < seg ? q.len - at : seg) : 0;
  return r.n > 0 || r.num == 0;
}

// log alpha below -1e4 is alpha = 0 in float32 either way; the bound keeps sums finite for
// alpha = 0 (log alpha = -inf).  A NaN stays one.
__device__ __forceinline__ float la_log(float la) { return la < kGdrMinLog ? kGdrMinLog : la; }

// What an element of a state is multiplied by over some tokens of log decay g:
// near 1 as x + expm1(g) x, since a rounded factor applied again and again adds up.
struct LaDecay {
  float f;
  bool near;
};
__device__ __forceinline__ LaDecay la_decay(float g) {
  const bool near = g > -0.5f;
  return LaDecay{near ? expm1f(g) : expf(g), near};
}
// (the product is of a finite value, since infinity takes nothing off infinity)
__device__ __forceinline__ float la_apply(const LaDecay& d, float x) {
  constexpr float kMost = 3.402823466e38f;
  return d.near ? fmaf(d.f, fminf(fmaxf(x, -kMost), kMost), x) : d.f * x;
}

// The kernels of a call follow one another closely: each lets the next one be set up
// once all of its CTAs run, and the next waits, first of all and in every CTA, until
// the one before has ended and its writes can be read.  (No effect in the first.)
__device__ __forceinline__ void la_chain() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// `after`: the kernel follows another of the same call
template <typename... P, typename... A>
ll_status la_launch(bool after, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                    const A&... args) {
  if (smem > 48 * 1024)
    LL_CUDA_OK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = &at;
  c.numAttrs = after ? 1 : 0;
  LL_CUDA_OK(cudaLaunchKernelEx(&c, kernel, args...));
  return LL_OK;
}

// ---- launchers
size_t la_fwd_workspace(const LaArgs& a);
ll_status la_fwd_launch(const LaArgs& a);
int la_fwd_launches(const LaArgs& a);
size_t la_bwd_workspace(const LaArgs& a);
ll_status la_bwd_launch(const LaArgs& a);
int la_bwd_launches(const LaArgs& a);

// the states on entry to every segment from the sums of the segments (la_rec.cu)
struct LaCarry {
  GdrSeqs seqs;
  int seg, elems;                        // tokens of a segment, elements of a state
  float* sums[2];                        // [slot, H, elems]: forwards, backwards (null: not wanted); in place
  const float* log_decay;                // [slot, H]
  const float* init[2];                  // [sequence, H, elems] or null
};

// in chunks on the tensor cores (la_tc.cu)
bool la_tc_formats(const LaArgs& a);
ll_status la_tc_sum_launch(const LaArgs& a, int seg, size_t slots, int dirs, float* sum_s, float* sum_a,
                           float* log_decay);
ll_status la_tc_fwd_main(const LaArgs& a, int seg, size_t slots, const float* states, bool by_slot, bool after);
ll_status la_tc_bwd_main(const LaArgs& a, int seg, size_t slots, const float* states, const float* adjoints,
                         bool by_slot, float* before, float* ends, float* dq32, float* dk32, float* part_q, float* part_v, bool after);

struct LaRope {
  int rot, interleaved;
  const float* inv_freq;
  float amp;
};
struct LaStepArgs {
  int B, H, Hk, dk, dv;
  ll_dtype io;
  int per_head;
  float scale;
  const int64_t* slots;
  int n_slots;
  const void *q, *k, *v;
  const float *log_alpha;
  float* states;
  LaRope rope;  // rot = 0: none
  const int64_t* positions;
  void* o;
  cudaStream_t stream;
  unsigned* err;
};
ll_status la_step_launch(const LaStepArgs& a);

struct RopeArgs {
  int B, H, Hk, T, d;
  ll_dtype io;
  LaRope rope;
  const int64_t* positions;  // [B,T] or null: 0 .. T-1
  const void *q, *k;
  void *q_out, *k_out;
  bool back;
  cudaStream_t stream;
};
ll_status rope_launch(const RopeArgs& a);

}  // namespace llattn
