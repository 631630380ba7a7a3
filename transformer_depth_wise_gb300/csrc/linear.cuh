// linear.cuh -- what the linear-attention kernels share: a launch's
// parameters, the sequences' lengths, decay powers, first states.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace attnres {

struct LinearParams {
  const void *a, *b, *c;
  int64_t a_stride, b_stride, c_stride;
  void *out;
  int64_t T, seg_len;
  int H, da, dc, nseg, slices;         // slices: CTAs over the columns of c (fp32 kernel)
  const float *log_decay;
  const int32_t *lengths;
  float alpha, carry, gain;            // of the masked products, of the state read out, of what enters it
  int reverse;
  const float *first;
  int first_t, first_pow;
  float *last;
  int last_pow;
  // The states that the segments begin with (nseg > 1): [B, H, nstates, da, dc],
  // segment s of this launch's begins with state s * step.  The states' kernel
  // may cut the segments finer than the main one.
  float *states;
  int nstates, step;
  int states_t;                        // or [.., dc, da], for the main kernel
  // Tensor-core form, nseg > 1: which columns of a segment's last state hold
  // what is no number, [B, H, nseg][kMarks] words, and a count of the (sequence,
  // head)'s CTAs that are done, [B, H]: zero before the main kernel and after it.
  uint32_t *marks, *done;
  float piece;                         // tokens that a CTA of the states' kernel had
  long long wait_limit;                // SM clock cycles any wait of the tensor-core kernel may take
};

constexpr int kMarks = 8;              // 128 columns for each half of the rows

__device__ __forceinline__ int64_t seq_length(const LinearParams &p, int64_t b) {
  if (!p.lengths) return p.T;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n < p.T ? n : p.T;
}
// lambda^n; lambda^0 = 1 whatever g is.
__device__ __forceinline__ float decay_pow(float g, int64_t n) { return n == 0 ? 1.f : expf(g * (float)n); }

// The first state's element (m, n).
__device__ __forceinline__ float first_at(const LinearParams &p, int64_t bh, int m, int n) {
  const float *f = p.first + bh * p.da * p.dc;
  return p.first_t ? f[(int64_t)n * p.da + m] : f[(int64_t)m * p.dc + n];
}

// Token i of the walk (reverse: from the last token back) as a row of the [B, T] axis.
__device__ __forceinline__ int64_t walk_row(const LinearParams &p, int64_t b, int64_t n, int64_t i) {
  return b * p.T + (p.reverse ? n - 1 - i : i);
}

// Segments hold whole chunks of 64 tokens.
constexpr int kChunk = 64;

// How the time axis is cut: nseg segments of seg_len tokens, each of nsub
// pieces (whole chunks) for the states' kernel.
struct Split {
  int64_t seg_len;
  int nseg, nsub;
};
// The tensor-core form (bf16): its split, and the launches of the states'
// kernel and of the main one.
// Every bf16 prompt of one token or more takes it: on the CUDA cores, in
// 64-token chunks whatever they hold, 4 heads of 128 x 128 took 19.4 us against
// 9.9 for one token and 26.2 against 9.6 for 63.
inline bool linear_tc_supported(int64_t T, int dtype) { return dtype == ATTNRES_BF16 && T > 0; }
Split linear_tc_split(int64_t BH, int64_t T);
cudaError_t launch_linear_tc(const LinearParams &p, int64_t BH, bool states, cudaStream_t stream);

}  // namespace attnres
