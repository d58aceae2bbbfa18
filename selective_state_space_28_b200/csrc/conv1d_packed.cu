// conv1d_packed.cu -- the mixers' causal depthwise convolution (+ silu) over
// packed sequences, conv states in a cache by slot:
//
//   u[t, c] = silu(bias[c] + sum_{k<W} w[c, k] x[t - (W - 1) + k, c]),
//
// inputs before a sequence's first token from its state (zeros without one),
// the state left holding the sequence's last W - 1 inputs.
//
// Bound by its bytes.  A thread takes V consecutive channels over a run of RUN
// tokens of one sequence, the W - 1 previous inputs in registers.  Runs are
// numbered without a scan over the lengths, whatever the order of the sequences:
// sequence i's first run is tokens / RUN + i, and a later one, from row t, is
// t / RUN - 1 (the RUN rows before it are its sequence's, so among sequences that
// are apart no two later runs start within the same RUN rows); a CTA's run is one,
// and each warp looks for its sequence together.  The thread with a sequence's
// first run is the only one that touches its state: it reads the old inputs, and
// takes the new ones from x, so no other thread's order matters and one launch
// does.
//
// Two forms.  Runs of 64 tokens are copied ahead into the thread's own
// shared-memory slots (three batches of eight, as ssm_conv1d_fwd, whose
// arithmetic this is bit for bit).  Sequences of under 16 tokens on average (a
// decode batch) take runs of 8 through registers, four channels a thread: the
// other form's 49 KB of slots and 8-channel registers leave too few threads in
// flight to cover the latency of finding the sequence, its state and its row.
#include "common.cuh"
#include "internal.h"

namespace ssm {
namespace {

constexpr int kThreads = 128, kStages = 3;
constexpr int kLong = 64, kShort = 8;  // tokens a run

template <typename T, int V> struct Vec {  // V = 1
  using Raw = T;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[V]) { f[0] = ld(&w); }
  static __device__ __forceinline__ Raw zero() { return T(0.f); }
  static __device__ __forceinline__ Raw load(const T *p) { return *p; }
  static __device__ __forceinline__ void store(T *p, const float (&f)[V]) { st(p, f[0]); }
};
template <> struct Vec<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[8]) {
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z); f[5] = bf16hi(w.z); f[6] = bf16lo(w.w); f[7] = bf16hi(w.w);
  }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p) {
    return __ldcs(reinterpret_cast<const uint4 *>(p));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4 *>(p),
           make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7])));
  }
};
template <> struct Vec<__nv_bfloat16, 4> {
  using Raw = uint2;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[4]) {
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
  }
  static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
  static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p) {
    return __ldcs(reinterpret_cast<const uint2 *>(p));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[4]) {
    __stcs(reinterpret_cast<uint2 *>(p), make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])));
  }
};
template <> struct Vec<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ void widen(const Raw &w, float (&f)[4]) {
    f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w;
  }
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ Raw load(const float *p) {
    return __ldcs(reinterpret_cast<const float4 *>(p));
  }
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

// Whether run `run` is one of sequence i's behind its first (a valid pair of
// bounds, a slot that is not padding).
template <int RUN>
__device__ __forceinline__ bool has_run(const ConvPackedParams &p, int64_t i, int64_t run) {
  const int64_t b = p.cu[i], e = p.cu[i + 1], first = b / RUN;
  const int64_t slot = p.slots ? (int64_t)p.slots[i] : 0;
  return b >= 0 && e > b && e <= p.tokens && first <= run && run < first + (e - b - 1) / RUN &&
         (!p.slots || (slot >= 0 && slot < p.state_rows));
}

// The sequence with run `run`, by a whole warp (-1: none).  Of a later run the last
// that does not start behind the RUN rows before it has it where the bounds do not
// decrease: among up to 1024 by counting (one round of loads), among more by
// bisection.  Where it does not, the up to 1024 are looked through.
template <int RUN>
__device__ __forceinline__ int64_t find_sequence(const ConvPackedParams &p, int64_t run) {
  if (run >= p.tokens / RUN) return run - p.tokens / RUN;
  if (p.nseq <= 1024) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int i = lane; i < (int)p.nseq; i += 32) n += p.cu[i] / RUN <= run;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n > 0 && has_run<RUN>(p, n - 1, run)) return n - 1;
    int at = -1;
    for (int i = lane; i < (int)p.nseq; i += 32)
      if (has_run<RUN>(p, i, run)) at = i;
    return __reduce_max_sync(0xffffffffu, at);
  }
  int64_t lo = 0, hi = p.nseq - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (p.cu[mid] / RUN <= run) lo = mid;
    else hi = mid - 1;
  }
  return p.cu[lo] / RUN <= run ? lo : -1;
}

template <int BYTES> __device__ __forceinline__ void cp_async(void *dst, const void *src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES)
                 : "memory");
}

template <typename T, int V, int W, int RUN, bool SILU>
__global__ void __launch_bounds__(kThreads, RUN == kShort ? 8 : 1) conv1d_packed_kernel(const ConvPackedParams p) {
  using Vc = Vec<T, V>;
  using Raw = typename Vc::Raw;
  constexpr int B = W - 1;  // inputs before a token
  constexpr bool kAhead = RUN == kLong && V > 1;
  constexpr int kBatch = RUN == kLong ? 8 : 2;  // tokens loaded together
  __shared__ Raw stage[kAhead ? kStages : 1][kAhead ? kBatch : 1][kAhead ? kThreads : 1];
  const int tid = threadIdx.x;
  const int64_t run = (int64_t)blockIdx.y + (int64_t)blockIdx.z * 65535;
  if (run >= p.tokens / RUN + p.nseq) return;
  const int64_t c = ((int64_t)blockIdx.x * kThreads + tid) * V;
  const bool mine = c < p.Cc;
  // Channel pairs (each lane of a pair is exactly the scalar fmaf / multiply);
  // V = 1 leaves the second lane unused.
  constexpr int VP = (V + 1) / 2;
  f2 w[VP][W], bias[VP], hist[B > 0 ? B : 1][VP];  // hist: oldest first
  {
    float f[V * W];
    load_floats(p.w + (mine ? c : 0) * W, f);
#pragma unroll
    for (int e = 0; e < VP; ++e) {
#pragma unroll
      for (int q = 0; q < W; ++q) w[e][q] = mk2(f[2 * e * W + q], V > 1 ? f[((2 * e + 1) % V) * W + q] : 0.f);
      bias[e] = p.bias ? mk2(__ldg(p.bias + (mine ? c : 0) + 2 * e), V > 1 ? __ldg(p.bias + (mine ? c : 0) + 2 * e + 1) : 0.f)
                       : mk2(0.f, 0.f);
    }
  }
  auto pairs = [](const float(&f)[V], f2(&h)[VP]) {
#pragma unroll
    for (int e = 0; e < VP; ++e) h[e] = mk2(f[2 * e], V > 1 ? f[(2 * e + 1) % V] : 0.f);
  };
  const int64_t seq = find_sequence<RUN>(p, run);
  if (!mine || seq < 0) return;
  const int64_t begin = p.cu[seq], end = p.cu[seq + 1];
  if (begin < 0 || end < begin || end > p.tokens) return;
  const int64_t j = run >= p.tokens / RUN ? 0 : run - begin / RUN + 1;
  const int64_t slot = p.slots ? (int64_t)p.slots[seq] : seq;
  if (p.slots && (slot < 0 || slot >= p.state_rows)) return;
  const int64_t t0 = begin + j * RUN;
  const int64_t t1 = t0 + RUN < end ? t0 + RUN : end;
  if (t0 >= t1) return;  // an empty sequence keeps its state
  const int n = (int)(t1 - t0);

  const T *x = static_cast<const T *>(p.x) + c;
  const T *px = x + t0 * p.x_row;
  int at = 0;  // tokens copied
  auto issue = [&](int k) {
#pragma unroll
    for (int a = 0; a < kBatch; ++a, ++at)
      if (at < n) cp_async<sizeof(Raw)>(&stage[k][a][tid], px + at * p.x_row);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k);
  }

  if constexpr (B > 0) {
    if (j > 0) {
#pragma unroll
      for (int q = 0; q < B; ++q) {
        float f[V];
        Vc::widen(Vc::load(x + (t0 - B + q) * p.x_row), f);
        pairs(f, hist[q]);
      }
    } else {
      float old[V * B];  // the state's layout: a channel's inputs, oldest first
#pragma unroll
      for (int i = 0; i < V * B; ++i) old[i] = 0.f;
      float *sp = p.state ? p.state + (slot * p.Cc + c) * B : nullptr;
      if (sp) load_floats(sp, old);
#pragma unroll
      for (int q = 0; q < B; ++q) {
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = old[e * B + q];
        pairs(f, hist[q]);
      }
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
                if (o == B + t) f[e] = old[e * B + o];
            }
          }
#pragma unroll
          for (int e = 0; e < V; ++e) now[e * B + q] = f[e];
        }
        store_floats(sp, now);
      }
    }
  }
  T *u = static_cast<T *>(p.u) + t0 * p.Cc + c;
  auto token = [&](const Raw &raw) {
    float f[V], o[V];
    Vc::widen(raw, f);
    f2 xv[VP];
    pairs(f, xv);
#pragma unroll
    for (int e = 0; e < VP; ++e) {
      f2 acc = fma2(w[e][W - 1], xv[e], bias[e]);  // the newest input first
#pragma unroll
      for (int q = B - 1; q >= 0; --q) acc = fma2(w[e][q], hist[q][e], acc);
      o[2 * e] = SILU ? gate<T>(acc.x) : acc.x;
      if (V > 1) o[(2 * e + 1) % V] = SILU ? gate<T>(acc.y) : acc.y;
    }
    Vc::store(u, o);
    u += p.Cc;
    if constexpr (B > 0) {
#pragma unroll
      for (int e = 0; e < VP; ++e) {
#pragma unroll
        for (int q = 0; q + 1 < B; ++q) hist[q][e] = hist[q + 1][e];
        hist[B - 1][e] = xv[e];
      }
    }
  };
  if constexpr (kAhead) {
    int k = 0;
    for (int t = 0; t < n; t += kBatch) {
      issue(k == 0 ? kStages - 1 : k - 1);  // the slots of the batch before
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
      for (int a = 0; a < kBatch; ++a) {
        if (t + a >= n) break;
        token(stage[k][a][tid]);
      }
      k = k == kStages - 1 ? 0 : k + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else {
    for (int t = 0; t < n; t += kBatch) {
      Raw raw[kBatch];
#pragma unroll
      for (int a = 0; a < kBatch; ++a) raw[a] = t + a < n ? Vc::load(px + (t + a) * p.x_row) : Vc::zero();
#pragma unroll
      for (int a = 0; a < kBatch; ++a) {
        if (t + a >= n) break;
        token(raw[a]);
      }
    }
  }
}

template <typename T, int V, int W, int RUN>
cudaError_t run_w(const ConvPackedParams &p, cudaStream_t s) {
  const int64_t chunks = (p.Cc + V - 1) / V, runs = p.tokens / RUN + p.nseq;
  const int64_t gy = runs < 65535 ? runs : 65535, gz = (runs + 65534) / 65535;
  if (gz > 65535) return cudaErrorNotSupported;
  const dim3 grid((unsigned)((chunks + kThreads - 1) / kThreads), (unsigned)gy, (unsigned)gz);
  if (p.silu) conv1d_packed_kernel<T, V, W, RUN, true><<<grid, kThreads, 0, s>>>(p);
  else conv1d_packed_kernel<T, V, W, RUN, false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, int RUN>
cudaError_t run_v(const ConvPackedParams &p, cudaStream_t s) {
  if constexpr (RUN == kLong && V > 1) {
    // (several CTAs' slots on an SM need the shared-memory carve-out, a
    // preference of the current device: never fail the call on it)
    const void *k = p.silu ? (const void *)conv1d_packed_kernel<T, V, 4, RUN, true>
                           : (const void *)conv1d_packed_kernel<T, V, 4, RUN, false>;
    if (p.W == 4 && cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
      cudaGetLastError();
  }
  switch (p.W) {
    case 1: return run_w<T, V, 1, RUN>(p, s);
    case 2: return run_w<T, V, 2, RUN>(p, s);
    case 3: return run_w<T, V, 3, RUN>(p, s);
    default: return run_w<T, V, 4, RUN>(p, s);
  }
}

}  // namespace

cudaError_t launch_conv1d_packed(const ConvPackedParams &p, cudaStream_t s) {
  // whole vectors of x's and u's rows, or value by value
  const bool brief = p.tokens < 16 * p.nseq;
  if (p.io == 1) {
    if (p.Cc % 8 == 0 && p.x_row % 8 == 0)
      return brief ? run_v<__nv_bfloat16, 4, kShort>(p, s) : run_v<__nv_bfloat16, 8, kLong>(p, s);
    return brief ? run_v<__nv_bfloat16, 1, kShort>(p, s) : run_v<__nv_bfloat16, 1, kLong>(p, s);
  }
  if (p.Cc % 4 == 0 && p.x_row % 4 == 0)
    return brief ? run_v<float, 4, kShort>(p, s) : run_v<float, 4, kLong>(p, s);
  return brief ? run_v<float, 1, kShort>(p, s) : run_v<float, 1, kLong>(p, s);
}

}  // namespace ssm
