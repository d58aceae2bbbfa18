// conv1d_packed.cu -- the mixers' causal depthwise convolution (+ silu) over
// packed sequences, conv states in a cache by slot:
//
//   u[t, c] = silu(bias[c] + sum_{k<W} w[c, k] x[t - (W - 1) + k, c]),
//
// inputs before a sequence's first token from its state (zeros without one),
// the state left holding the sequence's last W - 1 inputs.
//
// Bound by its bytes.  A thread takes V consecutive channels over a run of
// kRun tokens of one sequence, the W - 1 previous inputs in registers, kBatch
// rows loaded together.  Runs are numbered so that every sequence starts a run
// of its own without a scan over the lengths: sequence i, from row s_i, has
// the runs floor(s_i / kRun) + i and on, which leaves it at least
// ceil(len / kRun); a thread finds its sequence by bisection.  The thread
// with a sequence's first run is the only one that touches its state: it
// reads the old inputs, and takes the new ones from x, so no other thread's
// order matters and one launch does.
#include "common.cuh"
#include "internal.h"

namespace ssm {
namespace {

constexpr int kThreads = 128, kRun = 32, kBatch = 8;

template <typename T, int V> struct Vec {  // V = 1
  using Raw = T;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[V]) { f[0] = ld(&w); }
  static __device__ __forceinline__ Raw zero() { return T(0.f); }
  static __device__ __forceinline__ void store(T *p, const float (&f)[V]) { st(p, f[0]); }
};
template <> struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[8]) {
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z); f[5] = bf16hi(w.z); f[6] = bf16lo(w.w); f[7] = bf16hi(w.w);
  }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4 *>(p),
           make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7])));
  }
};
template <> struct Vec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[4]) {
    f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w;
  }
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void store(float *p, const float (&f)[4]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
  }
};

template <typename T> __device__ __forceinline__ float gate(float z);
template <> __device__ __forceinline__ float gate<__nv_bfloat16>(float z) { return silu_tanh(z); }
template <> __device__ __forceinline__ float gate<float>(float z) { return silu(z); }

// N floats from / to p: 16-byte accesses where N floats are whole ones (every
// such offset from the aligned base is a multiple of N).
template <int N> __device__ __forceinline__ void load_floats(const float *p, float (&f)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(p + i);
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = p[i];
  }
}
template <int N> __device__ __forceinline__ void store_floats(float *p, const float (&f)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4 *>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = f[i];
  }
}

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv1d_packed_kernel(const ConvPackedParams p) {
  using Vc = Vec<T, V>;
  constexpr int B = W - 1;  // inputs before a token
  const int64_t chunks = (p.Cc + V - 1) / V;
  const int64_t ch = ((int64_t)blockIdx.x * kThreads + threadIdx.x);
  const int64_t run = (int64_t)blockIdx.y + (int64_t)blockIdx.z * 65535;
  if (ch >= chunks || run >= p.tokens / kRun + p.nseq) return;
  const int64_t c = ch * V;
  // the last sequence whose first run is not after this one
  int64_t lo = 0, hi = p.nseq - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if ((int64_t)p.cu[mid] / kRun + mid <= run) lo = mid;
    else hi = mid - 1;
  }
  const int64_t begin = p.cu[lo], end = p.cu[lo + 1];
  const int64_t j = run - (begin / kRun + lo);
  if (begin < 0 || end < begin || end > p.tokens || j < 0) return;
  const int64_t slot = p.slots ? (int64_t)p.slots[lo] : lo;
  if (p.slots && (slot < 0 || slot >= p.state_rows)) return;
  const int64_t t0 = begin + j * kRun;
  const int64_t t1 = t0 + kRun < end ? t0 + kRun : end;
  if (t0 >= t1) return;  // an empty sequence keeps its state

  const T *x = static_cast<const T *>(p.x) + c;
  using Raw = typename Vc::Raw;
  float win[B > 0 ? B : 1][V];
  if constexpr (B > 0) {
    if (j > 0) {
#pragma unroll
      for (int q = 0; q < B; ++q)
        Vc::widen(*reinterpret_cast<const Raw *>(x + (t0 - B + q) * p.x_row), win[q]);
    } else {
      float old[V * B];
#pragma unroll
      for (int i = 0; i < V * B; ++i) old[i] = 0.f;
      float *sp = p.state ? p.state + (slot * p.Cc + c) * B : nullptr;
      if (sp) load_floats(sp, old);
#pragma unroll
      for (int q = 0; q < B; ++q)
#pragma unroll
        for (int e = 0; e < V; ++e) win[q][e] = old[e * B + q];
      if (sp) {  // the last B inputs: of x, or of the old state where the sequence is shorter
        const int64_t len = end - begin;
        float now[V * B];
#pragma unroll
        for (int q = 0; q < B; ++q) {
          float f[V];
          const int64_t t = len - B + q;
          if (t >= 0) {
            Vc::widen(*reinterpret_cast<const Raw *>(x + (begin + t) * p.x_row), f);
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              f[e] = 0.f;
#pragma unroll
              for (int o = 0; o < B; ++o)
                if (o == B + t) f[e] = win[o][e];
            }
          }
#pragma unroll
          for (int e = 0; e < V; ++e) now[e * B + q] = f[e];
        }
        store_floats(sp, now);
      }
    }
  }
  float w[V * W], bias[V];
  load_floats(p.w + c * W, w);
#pragma unroll
  for (int e = 0; e < V; ++e) bias[e] = p.bias ? __ldg(p.bias + c + e) : 0.f;
  T *u = static_cast<T *>(p.u) + c;
  for (int64_t t = t0; t < t1; t += kBatch) {
    Raw raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      raw[i] = t + i < t1 ? __ldcs(reinterpret_cast<const Raw *>(x + (t + i) * p.x_row)) : Vc::zero();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (t + i >= t1) break;
      float f[V], o[V];
      Vc::widen(raw[i], f);
#pragma unroll
      for (int e = 0; e < V; ++e) {  // the newest input first, as ssm_conv1d_fwd
        float acc = fmaf(w[e * W + W - 1], f[e], bias[e]);
#pragma unroll
        for (int q = B - 1; q >= 0; --q) acc = fmaf(w[e * W + q], win[q][e], acc);
        o[e] = SILU ? gate<T>(acc) : acc;
      }
      Vc::store(u + (t + i) * p.Cc, o);
      if constexpr (B > 0) {
#pragma unroll
        for (int q = 0; q + 1 < B; ++q)
#pragma unroll
          for (int e = 0; e < V; ++e) win[q][e] = win[q + 1][e];
#pragma unroll
        for (int e = 0; e < V; ++e) win[B - 1][e] = f[e];
      }
    }
  }
}

template <typename T, int V, int W>
cudaError_t run_w(const ConvPackedParams &p, cudaStream_t s) {
  const int64_t chunks = (p.Cc + V - 1) / V, runs = p.tokens / kRun + p.nseq;
  const int64_t gy = runs < 65535 ? runs : 65535, gz = (runs + 65534) / 65535;
  if (gz > 65535) return cudaErrorNotSupported;
  const dim3 grid((unsigned)((chunks + kThreads - 1) / kThreads), (unsigned)gy, (unsigned)gz);
  if (p.silu) conv1d_packed_kernel<T, V, W, true><<<grid, kThreads, 0, s>>>(p);
  else conv1d_packed_kernel<T, V, W, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_v(const ConvPackedParams &p, cudaStream_t s) {
  switch (p.W) {
    case 1: return run_w<T, V, 1>(p, s);
    case 2: return run_w<T, V, 2>(p, s);
    case 3: return run_w<T, V, 3>(p, s);
    default: return run_w<T, V, 4>(p, s);
  }
}

}  // namespace

cudaError_t launch_conv1d_packed(const ConvPackedParams &p, cudaStream_t s) {
  // whole 16-byte vectors of x's and u's rows, or value by value
  if (p.io == 1)
    return p.Cc % 8 == 0 && p.x_row % 8 == 0 ? run_v<__nv_bfloat16, 8>(p, s)
                                             : run_v<__nv_bfloat16, 1>(p, s);
  return p.Cc % 4 == 0 && p.x_row % 4 == 0 ? run_v<float, 4>(p, s) : run_v<float, 1>(p, s);
}

}  // namespace ssm
