// gdr_recurrent.cu -- the gated delta rule token by token, in float32: the
// decode step (one token per sequence against a cache of states), and the
// prompt scan of the shapes and types the chunked tensor-core kernel does not
// take.  Per (sequence, value head), with decay a, write strength b and the
// key and query scaled to k and q:
//
//   u = b (v - a S^T k),  S <- a S + k u^T,  y = scale S^T q.
//
// y is read as scale (a S_old^T q + (q . k) u), so that both products with the
// state use the state before the write and are reduced together; the scalar
// q . k comes from the token alone.  A decay is applied as S + (a - 1) S with
// a - 1 = expm1(d A): decays close to 1, which a long memory multiplies a
// thousand times, then lose nothing to the rounding of a itself.
#include "common.cuh"
#include "gdr.cuh"
#include "internal.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ the step
// One CTA per (128 value columns, head, batch row).  Thread (pq, rg) holds
// VEC columns of the state rows rg, rg + RS, ...: a row group of threads reads
// whole rows, so the state moves in 16-byte accesses of whole sectors (VEC 4),
// all of a thread's loads in flight before the first is used.  Bound by the
// state's bytes, read and written once.  The two products' partial sums go
// through shared memory once.  250 rows of 32 heads, 128 x 128: 204 us, 5.2 TB/s,
// 79 % of a copy.  Slower there: 64 or 32 columns a CTA (225, 317 us), 512 threads
// (236), 32-byte accesses (272), accesses without the streaming hint (212), three
// CTAs to an SM (216), CTAs that stay and copy ahead asynchronously (250).
template <typename T, int VEC, int KPT>
__global__ void __launch_bounds__(kThreads) gdr_step_kernel(const GdrParams p) {
  __shared__ float kq[2][kGdrMaxKeyDim];
  __shared__ float dots[3];
  extern __shared__ __align__(16) float red[];  // [RS][2][vt]
  const int64_t b = blockIdx.x / p.H, hd = blockIdx.x % p.H;
  const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
  if (slot < 0 || slot >= p.state_rows) return;  // padding
  const int K = (int)p.K;
  const int v0 = blockIdx.y * 128;
  const int vt = (int)(p.V - v0 < 128 ? p.V - v0 : 128);
  const int P = vt / VEC, RS = kThreads / P;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pq = tid % P, rg = tid / P;
  const bool on = rg < RS;
  float *st = p.h_last + ((slot * p.H + hd) * p.K) * p.V + v0 + pq * VEC;

  float s[KPT][VEC];
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int r = rg + RS * j;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[j][e] = 0.f;
    if (on && r < K) {
      if (VEC == 4) {
        const float4 v = ld_stream4(reinterpret_cast<const float4 *>(st + (int64_t)r * p.V));
        s[j][0] = v.x; s[j][1 % VEC] = v.y; s[j][2 % VEC] = v.z; s[j][3 % VEC] = v.w;
      } else {
        s[j][0] = st[(int64_t)r * p.V];
      }
    }
  }
  const int64_t g = hd / (p.H / p.Hk);
  const T *kp = static_cast<const T *>(p.k) + b * p.k_row + g * p.K;
  const T *qp = static_cast<const T *>(p.q) + b * p.q_row + g * p.K;
  for (int i = tid; i < K; i += kThreads) {
    kq[0][i] = ld(kp + i);
    kq[1][i] = ld(qp + i);
  }
  const float am1 = expm1f(gdr_log_decay<T>(p, b, hd)), a = 1.f + am1;
  const float beta = gdr_beta<T>(p, b, hd);
  float vv[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    vv[e] = on ? ld(static_cast<const T *>(p.v) + b * p.v_row + hd * p.V + v0 + pq * VEC + e) : 0.f;
  __syncthreads();
  if (warp < 3) {  // k.k, q.q and q.k, a warp each
    const float *x = kq[warp == 0 ? 0 : 1], *y = kq[warp == 1 ? 1 : 0];
    float acc = 0.f;
    for (int i = lane; i < K; i += 32) acc = fmaf(x[i], y[i], acc);
#pragma unroll
    for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (lane == 0) dots[warp] = acc;
  }
  float ks[VEC], qs[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) ks[e] = qs[e] = 0.f;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int r = rg + RS * j;
    if (on && r < K) {
      const float kr = kq[0][r], qr = kq[1][r];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        ks[e] = fmaf(kr, s[j][e], ks[e]);
        qs[e] = fmaf(qr, s[j][e], qs[e]);
      }
    }
  }
  if (on) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      red[(2 * rg) * vt + pq * VEC + e] = ks[e];
      red[(2 * rg + 1) * vt + pq * VEC + e] = qs[e];
    }
  }
  __syncthreads();
  if (!on) return;
  const float nk = gdr_norm_factor(p, dots[0]), nq = gdr_norm_factor(p, dots[1]);
  float u[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) ks[e] = 0.f;
  for (int i = 0; i < RS; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) ks[e] += red[(2 * i) * vt + pq * VEC + e];
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) u[e] = nk * beta * (vv[e] - a * nk * ks[e]);  // against the raw k
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int r = rg + RS * j;
    if (r < K) {
      const float kr = kq[0][r];
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[j][e] = fmaf(kr, u[e], fmaf(am1, s[j][e], s[j][e]));
      if (VEC == 4)
        st_stream4(reinterpret_cast<float4 *>(st + (int64_t)r * p.V),
                   make_float4(s[j][0], s[j][1 % VEC], s[j][2 % VEC], s[j][3 % VEC]));
      else
        st[(int64_t)r * p.V] = s[j][0];
    }
  }
  if (rg == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) qs[e] = 0.f;
    for (int i = 0; i < RS; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) qs[e] += red[(2 * i + 1) * vt + pq * VEC + e];
    }
    T *yp = static_cast<T *>(p.y) + (b * p.H + hd) * p.V + v0 + pq * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) st_io(yp + e, p.scale * nq * fmaf(dots[2], u[e], a * qs[e]));
  }
}

template <typename T, int VEC>
cudaError_t step_vec(const GdrParams &p, int kpt, dim3 grid, size_t smem, cudaStream_t s) {
#define GDR_STEP(N)                                                        \
  if (kpt <= N) {                                                          \
    gdr_step_kernel<T, VEC, N><<<grid, kThreads, smem, s>>>(p);            \
    return cudaGetLastError();                                             \
  }
  GDR_STEP(4)
  GDR_STEP(8)
  GDR_STEP(16)
  GDR_STEP(32)
  if constexpr (VEC == 1) { GDR_STEP(128) }
#undef GDR_STEP
  return cudaErrorNotSupported;
}

template <typename T>
cudaError_t step_io(const GdrParams &p, cudaStream_t s) {
  const int vt = (int)(p.V < 128 ? p.V : 128);
  const bool vec = p.V % 4 == 0;
  const int RS = kThreads / (vec ? vt / 4 : vt);
  const int64_t blocks = p.nseq * p.H;
  if (blocks >= (1ll << 31)) return cudaErrorNotSupported;
  const dim3 grid((unsigned)blocks, (unsigned)((p.V + 127) / 128));
  // (the last, narrower tile of value columns has more row groups)
  const int tail = (int)(p.V % 128);
  const int RSt = tail ? kThreads / (vec ? tail / 4 : tail) : 0;
  const size_t words = 2 * (size_t)(RS * vt > RSt * tail ? RS * vt : RSt * tail);
  const int kpt = (int)((p.K + RS - 1) / RS);
  return vec ? step_vec<T, 4>(p, kpt, grid, words * 4, s) : step_vec<T, 1>(p, kpt, grid, words * 4, s);
}

// ------------------------------------------------------- the prompt, by token
// One CTA per (32 value columns, head, sequence).  Warps 0-3 run the chain with
// the state in registers: eight lanes to a pair of columns, each with 4 J of its
// K rows (float4 groups 8 lanes apart, so a warp's shared-memory reads of k and
// q are whole 128-byte lines, and serve two columns); a token's two products
// are reduced with three shuffles.  Warps 4-7 bring the next TOK tokens to
// shared memory as float32 and make their scalars, with the ones after in
// flight, and store the last ones' y.  The chain from token to token (products,
// shuffles, write) bounds it, not bytes or flops: some 370 cycles a token at K =
// 128 (one group of warps for both took 620).
constexpr int kCols = 32, kGroup = 128;

template <typename T, int J, int TOK>
__global__ void __launch_bounds__(2 * kGroup, 1) gdr_recurrent_kernel(const GdrParams p) {
  constexpr int KP = 32 * J;
  constexpr int kPre = TOK * 2 * KP / kGroup, kPreV = TOK * kCols / kGroup;
  constexpr int kPer = TOK / (kGroup / 32);  // tokens whose scalars a warp makes
  __shared__ __align__(16) float kq[2][TOK][2][KP];
  __shared__ float vs[2][TOK][kCols], ys[2][TOK][kCols];
  __shared__ float sc[2][TOK][5];  // a - 1, b nk, a nk, scale nq a, scale nq nk (q . k)
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int64_t vtiles = (p.V + kCols - 1) / kCols;
  const int64_t v0 = (blockIdx.x % vtiles) * kCols;
  const int64_t unit = blockIdx.x / vtiles;
  const int64_t hd = unit % p.H, seq = unit / p.H;
  int64_t slot, t0, len;
  if (!gdr_sequence(p, seq, slot, t0, len)) return;
  const int K = (int)p.K;
  const int64_t g = hd / (p.H / p.Hk);
  const int64_t stages = (len + TOK - 1) / TOK;

  if (threadIdx.x >= kGroup) {
    // ---------------------------------------------------------- staging
    const int tid = threadIdx.x - kGroup;
    const T *kb = static_cast<const T *>(p.k) + g * p.K;
    const T *qb = static_cast<const T *>(p.q) + g * p.K;
    const T *vb = static_cast<const T *>(p.v) + hd * p.V + v0;
    T *yb = static_cast<T *>(p.y) + (t0 * p.H + hd) * p.V + v0;
    // the gates of a warp's tokens: lanes 0 ..
    const float Ah = p.dt ? p.A[hd] : 0.f, bias = p.dt && p.dt_bias ? p.dt_bias[hd] : 0.f;
    T pdt = T(0.f), pbe = T(0.f), pre[kPre], prev[kPreV];
    auto fetch = [&](int64_t t) {
      if (lane < kPer && t + kPer * warp + lane < len) {
        const int64_t row = t0 + t + kPer * warp + lane;
        if (p.dt) pdt = static_cast<const T *>(p.dt)[row * p.dt_row + hd];
        pbe = static_cast<const T *>(p.beta)[row * p.beta_row + hd];
      }
#pragma unroll
      for (int i = 0; i < kPre; ++i) {
        const int idx = tid + kGroup * i;
        const int tok = idx / (2 * KP), w = idx / KP % 2, c = idx % KP;
        const int64_t row = t0 + t + tok;
        pre[i] = T(0.f);
        if (t + tok < len && c < K) pre[i] = w ? qb[row * p.q_row + c] : kb[row * p.k_row + c];
      }
#pragma unroll
      for (int i = 0; i < kPreV; ++i) {
        const int idx = tid + kGroup * i;
        const int tok = idx / kCols, c = idx % kCols;
        prev[i] = T(0.f);
        if (t + tok < len && v0 + c < p.V) prev[i] = vb[(t0 + t + tok) * p.v_row + c];
      }
    };
    auto stage = [&](int64_t st) {  // what fetch(st TOK) brought
      const int b = (int)(st & 1);
#pragma unroll
      for (int i = 0; i < kPre; ++i) {
        const int idx = tid + kGroup * i;
        kq[b][idx / (2 * KP)][idx / KP % 2][idx % KP] = ld(&pre[i]);
      }
#pragma unroll
      for (int i = 0; i < kPreV; ++i) {
        const int idx = tid + kGroup * i;
        vs[b][idx / kCols][idx % kCols] = ld(&prev[i]);
      }
      const float dt = ld(&pdt), be = ld(&pbe);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (st + 1 < stages) fetch((st + 1) * TOK);
      float mine[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        float dot[3] = {0.f, 0.f, 0.f};  // k.k, q.q, q.k
#pragma unroll
        for (int c = 0; c < J; ++c) {
          const float x = kq[b][kPer * warp + i][0][lane + 32 * c];
          const float y = kq[b][kPer * warp + i][1][lane + 32 * c];
          dot[0] = fmaf(x, x, dot[0]);
          dot[1] = fmaf(y, y, dot[1]);
          dot[2] = fmaf(x, y, dot[2]);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1)
#pragma unroll
          for (int e = 0; e < 3; ++e) dot[e] += __shfl_xor_sync(0xffffffffu, dot[e], off);
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (lane == i) mine[e] = dot[e];
      }
      if (lane < kPer) {
        float d = dt + bias;
        if (p.flags & SSM_DT_SOFTPLUS) d = softplus(d);
        const float am1 = p.dt ? expm1f(d * Ah) : 0.f, a = 1.f + am1;
        const float beta = (p.flags & GDR_BETA_SIGMOID) ? 1.f / (1.f + ex2(-be * kLog2e)) : be;
        const float nk = gdr_norm_factor(p, mine[0]), nq = p.scale * gdr_norm_factor(p, mine[1]);
        float *o = sc[b][kPer * warp + lane];
        o[0] = am1;
        o[1] = beta * nk;
        o[2] = a * nk;
        o[3] = nq * a;
        o[4] = nq * mine[2];
      }
    };
    auto output = [&](int64_t st) {
      const int n = (int)(len - st * TOK < TOK ? len - st * TOK : TOK);
      if (v0 + lane < p.V) {
        for (int tok = warp; tok < n; tok += kGroup / 32)
          st_io(yb + (st * TOK + tok) * p.H * p.V + lane, ys[st & 1][tok][lane]);
      }
    };
    if (stages > 0) {
      fetch(0);
      stage(0);
    }
    __syncthreads();
    for (int64_t st = 0; st < stages; ++st) {
      if (st > 0) output(st - 1);
      if (st + 1 < stages) stage(st + 1);
      __syncthreads();
    }
    if (stages > 0) output(stages - 1);
    return;
  }

  // ------------------------------------------------------------ the chain
  const int r = lane & 7;
  const int cl = 2 * (warp * 4 + (lane >> 3));  // columns cl and cl + 1 of the tile
  const bool live[2] = {v0 + cl < p.V, v0 + cl + 1 < p.V};
  const int64_t so = (slot * p.H + hd) * p.K * p.V + v0 + cl;
  f2 s[2][J][2];  // [column]
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 32 * j + 4 * r + e;
        x[e] = p.h0 && live[w] && row < K ? p.h0[so + (int64_t)row * p.V + w] : 0.f;
      }
      s[w][j][0] = mk2(x[0], x[1]);
      s[w][j][1] = mk2(x[2], x[3]);
    }
  __syncthreads();
  for (int64_t st = 0; st < stages; ++st) {
    const int b = (int)(st & 1);
    const int n = (int)(len - st * TOK < TOK ? len - st * TOK : TOK);
    auto token = [&](int tok) {
      const float4 *k4 = reinterpret_cast<const float4 *>(kq[b][tok][0]) + r;
      const float4 *q4 = reinterpret_cast<const float4 *>(kq[b][tok][1]) + r;
      const float *c = sc[b][tok];
      const f2 zero = mk2(0.f, 0.f);
      f2 k2[J][2], ka[2] = {zero, zero}, qa[2] = {zero, zero}, kc[2] = {zero, zero}, qc[2] = {zero, zero};
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float4 kv = k4[8 * j], qv = q4[8 * j];
        k2[j][0] = mk2(kv.x, kv.y);
        k2[j][1] = mk2(kv.z, kv.w);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          ka[w] = fma2(k2[j][0], s[w][j][0], ka[w]);
          kc[w] = fma2(k2[j][1], s[w][j][1], kc[w]);
          qa[w] = fma2(mk2(qv.x, qv.y), s[w][j][0], qa[w]);
          qc[w] = fma2(mk2(qv.z, qv.w), s[w][j][1], qc[w]);
        }
      }
      float ks[2], qs[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const f2 x = add2(ka[w], kc[w]), y = add2(qa[w], qc[w]);
        ks[w] = x.x + x.y;
        qs[w] = y.x + y.y;
      }
#pragma unroll
      for (int off = 1; off < 8; off <<= 1)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          ks[w] += __shfl_xor_sync(0xffffffffu, ks[w], off);
          qs[w] += __shfl_xor_sync(0xffffffffu, qs[w], off);
        }
      const f2 am1 = mk2(c[0], c[0]);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        // u against the raw key: S <- a S + k_raw u
        const float u = c[1] * (vs[b][tok][cl + w] - c[2] * ks[w]);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          s[w][j][0] = fma2(k2[j][0], mk2(u, u), fma2(am1, s[w][j][0], s[w][j][0]));
          s[w][j][1] = fma2(k2[j][1], mk2(u, u), fma2(am1, s[w][j][1], s[w][j][1]));
        }
        if (r == 0) ys[b][tok][cl + w] = fmaf(c[4], u, c[3] * qs[w]);
      }
    };
    // (whole stages unrolled: the next tokens' operands are read ahead of the
    // chain through the state)
    if (n == TOK) {
#pragma unroll
      for (int tok = 0; tok < TOK; ++tok) token(tok);
    } else {
      for (int tok = 0; tok < n; ++tok) token(tok);
    }
    __syncthreads();
  }
  if (p.h_last) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float x[4] = {s[w][j][0].x, s[w][j][0].y, s[w][j][1].x, s[w][j][1].y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 32 * j + 4 * r + e;
          if (live[w] && row < K) p.h_last[so + (int64_t)row * p.V + w] = x[e];
        }
      }
  }
}

template <typename T>
cudaError_t recurrent_io(const GdrParams &p, cudaStream_t s) {
  const int64_t blocks = p.nseq * p.H * ((p.V + kCols - 1) / kCols);
  if (blocks >= (1ll << 31)) return cudaErrorNotSupported;
  const unsigned grid = (unsigned)blocks;
  if (p.K <= 32) gdr_recurrent_kernel<T, 1, 16><<<grid, 2 * kGroup, 0, s>>>(p);
  else if (p.K <= 64) gdr_recurrent_kernel<T, 2, 16><<<grid, 2 * kGroup, 0, s>>>(p);
  else if (p.K <= 128) gdr_recurrent_kernel<T, 4, 16><<<grid, 2 * kGroup, 0, s>>>(p);
  else gdr_recurrent_kernel<T, 8, 8><<<grid, 2 * kGroup, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_step(const GdrParams &p, cudaStream_t s) {
  return p.io == 1 ? step_io<__nv_bfloat16>(p, s) : step_io<float>(p, s);
}

cudaError_t launch_gdr_recurrent(const GdrParams &p, cudaStream_t s) {
  return p.io == 1 ? recurrent_io<__nv_bfloat16>(p, s) : recurrent_io<float>(p, s);
}

}  // namespace ssm
