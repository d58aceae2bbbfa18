// head_norm.cu -- the gated delta rule mixer's norm: per token and head,
//
//   out = x / sqrt(mean(x^2) + eps) * weight * silu(z).
//
// Bound by its bytes: x and z read once, out written once.  A row (one head
// of one token) is held in the registers of LPR lanes, NV 16-byte vectors a
// lane, so the mean and the scaling share one read (two rows a lane group were
// slower: 16384 x 32 rows of 128 bf16 79 us, one 68).  Widths that do not fit,
// or are not whole vectors, go value by value, the row read twice.
#include "common.cuh"
#include "internal.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

template <typename T> struct V16;
template <> struct V16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const uint4 &w, float (&f)[8]) {
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z); f[5] = bf16hi(w.z); f[6] = bf16lo(w.w); f[7] = bf16hi(w.w);
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  // (z / (1 + e^-z) keeps the digits of small values: 16384 x 32 rows of 128 76 us, this 73)
  static __device__ __forceinline__ float gate(float z) { return silu_tanh(z); }
};
template <> struct V16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(const uint4 &w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float gate(float z) { return silu(z); }
};

template <typename T, int LPR, int NV>
__global__ void __launch_bounds__(kThreads) head_norm_vec_kernel(const HeadNormParams p) {
  constexpr int N = V16<T>::N;
  constexpr int G = kThreads / LPR;  // rows a CTA holds at once
  const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int nvec = (int)(p.width / N);
  const int64_t rows = p.tokens * p.heads;
  const int64_t row = (int64_t)blockIdx.x * G + grp;
  const float inv = 1.f / (float)p.width;
  uint4 x[NV], z[NV];
  const int64_t tok = row / p.heads, hd = row - tok * p.heads;
  const uint4 *xp = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.x) + row * p.width);
  const uint4 *zp = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.z) + tok * p.z_row +
                                                    hd * p.width);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool on = row < rows && lane + LPR * v < nvec;
    x[v] = on ? __ldcs(xp + lane + LPR * v) : make_uint4(0u, 0u, 0u, 0u);
    z[v] = on && p.z ? __ldcs(zp + lane + LPR * v) : make_uint4(0u, 0u, 0u, 0u);
  }
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float f[N];
    V16<T>::widen(x[v], f);
#pragma unroll
    for (int e = 0; e < N; ++e) ss = fmaf(f[e], f[e], ss);
  }
#pragma unroll
  for (int off = LPR / 2; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float r = 1.f / sqrtf(ss * inv + p.eps);
  if (row >= rows) return;
  uint4 *op = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * p.width);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = lane + LPR * v;
    if (at >= nvec) continue;
    float f[N], g[N];
    V16<T>::widen(x[v], f);
    V16<T>::widen(z[v], g);
#pragma unroll
    for (int e4 = 0; e4 < N; e4 += 4) {
      const float4 w = p.weight ? __ldg(reinterpret_cast<const float4 *>(p.weight + at * N + e4))
                                : make_float4(1.f, 1.f, 1.f, 1.f);
      const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e4 + e] *= r * wv[e];
        if (p.z) f[e4 + e] *= V16<T>::gate(g[e4 + e]);
      }
    }
    __stcs(op + at, V16<T>::narrow(f));
  }
}

// A warp a row, value by value, the row read twice.
template <typename T>
__global__ void __launch_bounds__(kThreads) head_norm_any_kernel(const HeadNormParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.tokens * p.heads) return;
  const int64_t tok = row / p.heads, hd = row - tok * p.heads;
  const T *xp = static_cast<const T *>(p.x) + row * p.width;
  const T *zp = static_cast<const T *>(p.z) + tok * p.z_row + hd * p.width;
  T *op = static_cast<T *>(p.out) + row * p.width;
  float ss = 0.f;
  for (int i = lane; i < p.width; i += 32) {
    const float v = ld(xp + i);
    ss = fmaf(v, v, ss);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float r = 1.f / sqrtf(ss / (float)p.width + p.eps);
  for (int i = lane; i < p.width; i += 32) {
    float v = ld(xp + i) * r;
    if (p.weight) v *= __ldg(p.weight + i);
    if (p.z) v *= V16<T>::gate(ld(zp + i));
    st(op + i, v);
  }
}

template <typename T, int LPR, int NV>
cudaError_t run_vec(const HeadNormParams &p, cudaStream_t s) {
  constexpr int per = kThreads / LPR;
  const int64_t blocks = (p.tokens * p.heads + per - 1) / per;
  if (blocks >= (1ll << 31)) return cudaErrorNotSupported;
  head_norm_vec_kernel<T, LPR, NV><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run_io(const HeadNormParams &p, cudaStream_t s) {
  constexpr int N = V16<T>::N;
  if (p.width % N == 0 && p.z_row % N == 0) {
    const int64_t nv = p.width / N;
    if (nv <= 8) return run_vec<T, 8, 1>(p, s);
    if (nv <= 16) return run_vec<T, 16, 1>(p, s);
    if (nv <= 32) return run_vec<T, 32, 1>(p, s);
    if (nv <= 64) return run_vec<T, 32, 2>(p, s);
    if (nv <= 128) return run_vec<T, 32, 4>(p, s);
  }
  const int64_t blocks = (p.tokens * p.heads + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks >= (1ll << 31)) return cudaErrorNotSupported;
  head_norm_any_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head_norm(const HeadNormParams &p, cudaStream_t s) {
  return p.io == 1 ? run_io<__nv_bfloat16>(p, s) : run_io<float>(p, s);
}

}  // namespace ssm
