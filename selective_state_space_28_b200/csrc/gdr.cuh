// gdr.cuh -- what the gated delta rule's kernels share: a sequence's rows and
// state slot, and a token's decay, write strength and norm factors.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace ssm {

// st() under a name that a kernel's own variables do not hide.
template <typename T> __device__ __forceinline__ void st_io(T *p, float v) { IO<T>::store(p, v); }

// Sequence `seq`: the row of its state, its first row of q, k, v and y, and
// its length.  False: nothing of it is read or written (a slot out of range).
// Bounds that are out of order or out of the buffer make it empty.
__device__ __forceinline__ bool gdr_sequence(const GdrParams &p, int64_t seq, int64_t &slot,
                                             int64_t &t0, int64_t &len) {
  slot = p.slots ? (int64_t)p.slots[seq] : seq;
  // (without slots the host has checked state_rows, or there are no states)
  if (p.slots && (slot < 0 || slot >= p.state_rows)) return false;
  t0 = seq * p.L;
  len = p.L;
  if (p.cu) {
    t0 = p.cu[seq];
    len = (int64_t)p.cu[seq + 1] - t0;
    if (t0 < 0 || len < 0 || t0 + len > p.rows) t0 = len = 0;
  }
  return true;
}

// Logarithm of the decay of the token in row `row`, head `hd`: d A, 0 without
// a step input.
template <typename T>
__device__ __forceinline__ float gdr_log_decay(const GdrParams &p, int64_t row, int64_t hd) {
  if (!p.dt) return 0.f;
  float d = ld(static_cast<const T *>(p.dt) + row * p.dt_row + hd);
  if (p.dt_bias) d += p.dt_bias[hd];
  if (p.flags & SSM_DT_SOFTPLUS) d = softplus(d);
  return d * p.A[hd];
}

template <typename T>
__device__ __forceinline__ float gdr_beta(const GdrParams &p, int64_t row, int64_t hd) {
  const float b = ld(static_cast<const T *>(p.beta) + row * p.beta_row + hd);
  return (p.flags & GDR_BETA_SIGMOID) ? 1.f / (1.f + ex2(-b * kLog2e)) : b;
}

// 1 / sqrt(|x|^2 + eps) from |x|^2 (1 without the norm; 0 for a row of zeros,
// whatever eps).
__device__ __forceinline__ float gdr_norm_factor(const GdrParams &p, float ss) {
  if (!(p.flags & GDR_QK_L2NORM)) return 1.f;
  return ss == 0.f ? 0.f : 1.f / sqrtf(ss + p.l2_eps);
}

}  // namespace ssm
