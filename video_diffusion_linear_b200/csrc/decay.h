// Interface between the host entry points of the decayed linear attention and its kernels.
//
// Forward, every gradient and the per-segment states are one scan with its operands in other roles:
//   S_t = lambda S_{t-1} + z_t y_t^T,   o_t = S_t x_t      (S: rows z channel, columns y channel)
// run forwards or, for the gradients that flow back in time, from the last token to the first.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "vdn.h"

namespace vdn {

constexpr int kDecayChunk = 128;    // tokens per chunk of the tensor-core scan

// How the token axis is split: nseg segments of `len` tokens (a multiple of kDecayChunk on the
// tensor-core path).  nseg == 1: one launch, no workspace states.
struct DecayPlan {
  int nseg = 1;
  int len = 0;
  size_t status = 0, states = 0, rstates = 0, total = 0;   // workspace offsets
};
DecayPlan plan_decay(const vdn_shape& sh, bool backward);

struct DecayScan {
  int B, H, T, d;
  const void *x, *y, *z;       // [B, T, H, d]
  const float* decay;          // [H]
  const int* lengths;          // [B] or NULL
  // reverse: tokens from the last to the first.  The state enters the first token of the order
  // undecayed and is decayed once more after the last one (the gradient of the forward order).
  bool reverse;
  const float* init;           // [B, H, d, d] or NULL (zero): state before the order's first token
  const float* seg_states;     // [nseg][B, H, d, d] states before each segment, or NULL when nseg == 1
  bool transposed;             // init / seg_states / final hold S^T
  float out_near, out_far;     // o = out_near (terms inside the chunk) + out_far (terms of the state)
  float add;                   // factor of z y^T
  bool exact_state;            // the state can leave the call: keep it to fp32 rounding (tensor-core path)
  bool clear;                  // rows of out behind a sequence: to zero (else left as they were)
  void* out;
  float* final;                // [B, H, d, d] or NULL: state after the order's last token
  uint32_t* status;
  bool clear_status;           // this launch clears the status word: the first of a call
  cudaStream_t stream;
};

// every segment's own state: sum over its tokens, at the segment's end in scan order (none for the
// order's last segment, which no other follows)
cudaError_t launch_decay_segments_tc(const DecayScan& s, const DecayPlan& p, float* states);
cudaError_t launch_decay_scan_tc(const DecayScan& s, const DecayPlan& p);
cudaError_t launch_decay_segments_simt(const DecayScan& s, const DecayPlan& p, float* states);
cudaError_t launch_decay_scan_simt(const DecayScan& s, const DecayPlan& p);
// in place: every segment's own state -> the state before it (from s.init)
cudaError_t launch_decay_prefix(const DecayScan& s, const DecayPlan& p, float* states);
cudaError_t launch_decay_step(const vdn_shape& sh, const void* q, const void* k, const void* v, const float* decay,
                              float* state, const int* slots, int n_slots, float scale, void* out,
                              cudaStream_t stream);

// decay as a power of two: lambda^n = 2^(n l2).  lambda = 0 has l2 = -1e30, so that lambda^0 = 1 and
// lambda^n = 0 need no branch.  A NaN or negative decay is NaN here (the maximum that keeps a NaN; fmaxf drops it)
// and in decay_factor, so that every form of the operator shows it in all results of its head.
__device__ __forceinline__ float decay_log2(float lambda) {
  float l2;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(l2) : "f"(log2f(lambda)), "f"(-1e30f));
  return l2;
}
__device__ __forceinline__ float decay_factor(float lambda) { return lambda >= 0.f ? lambda : __int_as_float(0x7fffffff); }

// tokens of sequence b: lengths[b] clamped to [0, T]
__device__ __forceinline__ int decay_tokens(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : n > T ? T : n;
}

}  // namespace vdn
