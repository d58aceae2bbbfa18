// gdr_tc.cu -- the gated delta rule over prompts, 64 tokens a chunk, on the
// sm_100a tensor cores.
//
// Within a chunk that the state S enters, with a_t the decays, g_i the sum of
// log a over tokens 0 .. i, b_i the write strengths, k and q the scaled keys
// and queries:
//
//   (I + A) U = R,  A_ij = b_i e^(g_i - g_j) k_i.k_j (j < i),
//                   R_i = b_i (v_i - e^g_i S^T k_i),
//   y_i = scale (e^g_i S^T q_i + sum_{j<=i} e^(g_i - g_j) (q_i.k_j) U_j),
//   S  <- e^g_63 S + sum_j e^(g_63 - g_j) k_j U_j^T.
//
// One CTA per (sequence, value head, 128 value columns) walks the chunks.  A
// TMEM lane is a value column, so every product has M = 128 and its A operand
// (S, R, U, transposed) comes from TMEM, where the thread that owns the lane
// wrote it; tokens and key dimensions are columns:
//
//   KS = S^T K^T, QS = S^T Q^T        B = the keys / queries, K-major
//   G  = [K; Q] K^T                   (128 rows of keys and queries)
//   U  = R T^T,  T = (I + A)^-1       B = T
//   PU = U P^T,  P_ij = e^(g_i - g_j) q_i.k_j (j <= i)
//   dS = U'^T K, U'_j = e^(g_63 - g_j) U_j   B = the keys, MN-major
//
// Precision.  The state is kept and returned in float32, so what feeds it may
// not round to 16 bits: the products run on float16 pairs, x = hi + lo (22
// bits), two (KS, dS) or three (U) products for one.  y is returned in
// bfloat16: for QS and PU the hi parts alone do (2^-11 of a term beside the
// result's 2^-8).  float16 has the digits but not the range, so every operand
// is scaled by powers of two: a key or query by its own (its largest value
// comes to 1 .. 2, which keeps a bfloat16's 8 bits; the norm factor is applied
// to products in float32), and S, R, U each by one for the whole CTA and
// chunk, from bounds on measured maxima (below), so that the largest value
// stays below 2^15 and one 2^-18 of it still has 22 bits.  A lane whose values
// are not finite does not count toward the maxima.
//
// Warps (14):
//   12     TMA producer: K, Q ([64 x 64] slabs, 128-byte swizzle, three
//          stages), V ([64 x 128], two stages).
//   13     MMA issuer.
//   8-11   preparation of the next chunk: keys and queries to scaled float16 in
//          place, norms, gates (running sums in float64), the maximum of V,
//          then from G the matrices A and P, T by blocks (32 x 32 diagonal
//          blocks a column a lane by forward substitution, the block below
//          them -T22 A21 T11), T and P to float16 for the MMAs.
//   0-7    the chain: two warps per lane quarter, each with half of the columns:
//          R from KS and V; U and U' from the product with T; the state from
//          dS; then y of the chunk, under the next KS.
// The chain KS -> R -> U -> dS -> S is what bounds it: four products one behind
// the other and the elementwise work between them, each with its latency; G, QS, PU and all of the preparation run beside it.
//
// Every wait is bounded; one that runs out sets the status word, its role
// leaves, the others' waits run out in turn, and the CTA frees its TMEM.
#include <cuda_fp16.h>

#include "common.cuh"
#include "gdr.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "tma.h"

namespace ssm {
namespace {

using namespace sm100;

constexpr int kC = 64;    // tokens a chunk
constexpr int kV = 128;   // value columns a CTA
constexpr int kThreads = 448;
constexpr int kChain = 256, kPrep = 128;  // threads of the two groups
constexpr int kAm = 68;   // row stride of A / T in float32
constexpr long long kWaitLimit = 2000000000ll;  // cycles (about a second)

// TMEM columns.  dS lands where S's pieces are (they are rewritten from it),
// the product with T where KS was, U's hi parts where R's were.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColKS = 128, kColQS = 192, kColR = 256, kColU2 = 320, kColPU = 384,
                   kColG = 448;

template <int KD> struct __align__(1024) GdrSmem {
  uint8_t kq[3][KD / 64][128 * 128];  // [stage][slab]: rows 0-63 keys, 64-127 queries
  uint8_t T[2][2][kC * 128];          // [chunk parity][hi, lo]
  uint8_t P[2][kC * 128];
  __nv_bfloat16 v[2][kC][kV];
  float Am[kC][kAm];
  // of the chunk being prepared
  float ghi[kC], glo[kC], beta[kC], nk[kC], f31[kC / 2];
  // of a chunk, by parity: factors of the tokens ...
  float bv[2][kC], bk[2][kC], cu[2][kC], cqe[2][kC], cqp[2][kC];
  float gC[2];
  // ... and what the scales go by, a slot per warp
  float vmax[2][4], bvmax[2][2], bkmax[2][2], tmax[2][4];
  float rmax[2][8], umax[2][8], smax[2][8];
  float tpart[4];
  uint64_t fullk[3], empty[3], fullv[2], vempty[2], tready[2];
  uint64_t cready, gdone, ksdone, rready, udone, uready, supdone, sready, pudone, ofree;
  uint32_t taddr;
  int abort;
};
static_assert(sizeof(GdrSmem<128>) + 1024 <= 232448, "GdrSmem exceeds the shared memory of a CTA");

struct GdrTcParams {
  GdrParams p;
  int64_t vtiles;
  int *status;
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}
// Named barrier 1 over the preparation group; every thread gets the OR of v.
__device__ __forceinline__ bool prep_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// Instruction descriptor, kind::f16 with float16 A and B (formats 0) and a
// float32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// x = hi + lo in float16 pairs.
__device__ __forceinline__ void split_h2(f2 x, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  const float2 b = __half22float2(h);
  const f2 r = add2(x, mk2(-b.x, -b.y));
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = pack_h2(r.x, r.y);
}

// 2^e, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) {
  e = e < -126 ? -126 : e > 127 ? 127 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// The power of two that brings values up to `bound` below 2^15: its exponent,
// within +-100 (a bound of zero is no reason to scale).
__device__ __forceinline__ int scale_exp(float bound) {
  if (!(bound > 0.f)) return 0;
  const int e = 13 - ((int)(__float_as_uint(bound) >> 23) - 127);
  return e < -100 ? -100 : e > 100 ? 100 : e;
}
__device__ __forceinline__ float max_of(const float *s, int n) {
  float m = s[0];
  for (int i = 1; i < n; ++i) m = fmaxf(m, s[i]);
  return m;
}
// The warp's maximum of finite non-negative values; a lane's inf counts as 0.
__device__ __forceinline__ float warp_max(float m) {
  const uint32_t b = __float_as_uint(m);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, b < 0x7f800000u ? b : 0u));
}

template <typename S> __device__ __forceinline__ void set_abort(S &s, int *status, int code) {
  *(volatile int *)&s.abort = 1;
  if (status) atomicExch(status, code);
}
// A warp's wait: every lane polls (bounded), then the warp votes.
template <typename S>
__device__ __forceinline__ bool waitw(S &s, uint64_t *bar, uint32_t parity, int *status, int code) {
  const bool ok = mbar_wait(bar, parity, kWaitLimit);
  const bool fail = __any_sync(0xffffffffu, !ok);
  if (fail && (threadIdx.x & 31) == 0) set_abort(s, status, code);
  return !fail;
}

template <int KD>
__global__ void __launch_bounds__(kThreads, 1)
    gdr_tc_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mQ,
                  const __grid_constant__ CUtensorMap mV, const GdrTcParams tp) {
  constexpr int NP = KD / 64;        // slabs
  constexpr int KH = KD / 2;         // key dimensions of a chain warp's half
  constexpr int KS16 = KD / 16;      // K steps over the key dimension
  using Smem = GdrSmem<KD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const GdrParams &p = tp.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t vt = blockIdx.x % tp.vtiles, unit = blockIdx.x / tp.vtiles;
  const int64_t hd = unit % p.H, seq = unit / p.H;
  int64_t slot, t0, len;
  if (!gdr_sequence(p, seq, slot, t0, len)) return;
  const int64_t g = hd / (p.H / p.Hk);
  const int nch = (int)((len + kC - 1) / kC);
  const int64_t v0 = vt * kV;
  int *status = tp.status;
  const int64_t so = (slot * p.H + hd) * p.K * p.V + v0;  // the state's first value column

  // The chain's lanes: value column cv of the tile, columns of half ch.
  const int ch = warp >> 2;
  const int cv = 32 * (warp & 3) + lane;
  const bool live = v0 + cv < p.V;
  const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;

  if (nch == 0) {  // an empty sequence hands its state on
    if (warp < 8 && p.h_last && live) {
      for (int r = ch; r < p.K; r += 2) {
        const int64_t at = so + (int64_t)r * p.V + cv;
        p.h_last[at] = p.h0 ? p.h0[at] : 0.f;
      }
    }
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s.fullk[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.fullv[i], 1);
      mbar_init(&s.vempty[i], 8);
      mbar_init(&s.tready[i], 4);
    }
    mbar_init(&s.cready, 4);
    mbar_init(&s.gdone, 1);
    mbar_init(&s.ksdone, 1);
    mbar_init(&s.rready, 8);
    mbar_init(&s.udone, 1);
    mbar_init(&s.uready, 8);
    mbar_init(&s.supdone, 1);
    mbar_init(&s.sready, 8);
    mbar_init(&s.pudone, 1);
    mbar_init(&s.ofree, 8);
    s.abort = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(&s.taddr, kTmemCols);
    tmem_relinquish();
  }
  // T above its diagonal blocks is never written again
  if (warp >= 8 && warp < 12) {
    for (int i = tid - kChain; i < (int)sizeof(s.T) / 16; i += kPrep)
      reinterpret_cast<uint4 *>(&s.T[0][0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // the state's half row of this lane, and its maximum
  f2 st[KH / 2];
  if (warp < 8) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < KH; ++i) {
      const int r = ch * KH + i;
      const float x = p.h0 && live && r < p.K ? p.h0[so + (int64_t)r * p.V + cv] : 0.f;
      if (i & 1) st[i / 2].y = x; else st[i / 2].x = x;
      m = fmaxf(m, fabsf(x));
    }
    m = warp_max(m);
    if (lane == 0) s.smax[1][warp] = m;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.taddr;

  // S's pieces, hi and lo of each half within the half's own dS columns
  auto put_state = [&](int e) {
    const f2 sc = mk2(pow2i(e), pow2i(e));
#pragma unroll
    for (int i = 0; i < KH / 32; ++i) {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) split_h2(mul2(st[16 * i + j], sc), hi[j], lo[j]);
      tmem_st16(tb + lane_base + kColS + ch * KH + 16 * i, hi);
      tmem_st16(tb + lane_base + kColS + ch * KH + KH / 2 + 16 * i, lo);
    }
  };
  int eS = 0;
  if (warp < 8) {
    eS = scale_exp(max_of(s.smax[1], 8));
    put_state(eS);
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 12) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&mK);
      tma_prefetch_desc(&mQ);
      tma_prefetch_desc(&mV);
      int issued = 0;
      for (int c = 0; c < nch; ++c) {
        const int k3 = c % 3, t = (int)(t0 + (int64_t)c * kC);
        if (c >= 3 && !mbar_wait(&s.empty[k3], (c / 3 - 1) & 1, kWaitLimit)) {
          set_abort(s, status, 1);
          break;
        }
        mbar_expect_tx(&s.fullk[k3], NP * 128 * 128);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          tma_load_3d(s.kq[k3][n], &mK, &s.fullk[k3], 64 * n, (int)g, t);
          tma_load_3d(s.kq[k3][n] + kC * 128, &mQ, &s.fullk[k3], 64 * n, (int)g, t);
        }
        issued = c + 1;
        if (c >= 2 && !mbar_wait(&s.vempty[c & 1], ((c >> 1) - 1) & 1, kWaitLimit)) {
          set_abort(s, status, 2);
          break;
        }
        mbar_expect_tx(&s.fullv[c & 1], kC * kV * 2);
        tma_load_3d(s.v[c & 1], &mV, &s.fullv[c & 1], (int)v0, (int)hd, t);
      }
      // Leave no copy in flight: the last chunks issued have landed.
      for (int c = issued - 3; c < issued; ++c) {
        if (c < 0) continue;
        mbar_wait(&s.fullk[c % 3], (c / 3) & 1, kWaitLimit);
        if (c >= issued - 2 && !(*(volatile int *)&s.abort))
          mbar_wait(&s.fullv[c & 1], (c >> 1) & 1, kWaitLimit);
      }
    }
    __syncwarp();
  } else if (warp == 13) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t id64 = idesc_f16_f32(128, 64, false);
    const uint32_t idS = idesc_f16_f32(128, KD, true);
    uint64_t *last_bar = nullptr;
    uint32_t last_par = 0;
    auto commit = [&](uint64_t *bar, uint32_t par) {
      if (leader) mma_commit(bar);
      __syncwarp();
      last_bar = bar;
      last_par = par;
    };
    auto desc_k = [&](int c) { return smem_desc(smem_u32(s.kq[c % 3][0]), 16, 1024, kSwizzle128B); };
    // K step kk of a K-major operand of two slabs, in descriptor units
    auto koff = [](int kk) { return (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4); };
    auto gram = [&](int c) {
      tc_fence_after();
      if (leader) {
        const uint64_t d = desc_k(c);
#pragma unroll
        for (int kk = 0; kk < KS16; ++kk) mma_ss(tb + kColG, d + koff(kk), d + koff(kk), id64, kk > 0);
      }
      commit(&s.gdone, c & 1);
    };
    // TMEM column of K step kk of S's hi pieces (lo: KH / 2 further on)
    auto scol = [](int kk) { return kColS + (kk / (KH / 16)) * KH + (kk % (KH / 16)) * 8; };
    bool ok = waitw(s, &s.cready, 0, status, 3);
    if (ok) gram(0);
    for (int c = 0; ok && c < nch; ++c) {
      const uint32_t ph = c & 1, php = (c - 1) & 1;
      const uint64_t dk = desc_k(c), dq = dk + ((kC * 128) >> 4);
      if (c > 0 && !waitw(s, &s.sready, php, status, 4)) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int kk = 0; kk < KS16; ++kk)
            mma_ts(tb + kColKS, tb + scol(kk) + x * (KH / 2), dk + koff(kk), id64, x + kk > 0);
      }
      commit(&s.ksdone, ph);
      // QS and PU of the chunk before have been read
      if (c > 0 && !waitw(s, &s.ofree, php, status, 5)) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < KS16; ++kk)
          mma_ts(tb + kColQS, tb + scol(kk), dq + koff(kk), id64, kk > 0);
      }
      __syncwarp();
      // T and P of this chunk are there, so G of it has been read
      if (!waitw(s, &s.tready[ph], (c >> 1) & 1, status, 6)) break;
      if (c + 1 < nch) {
        if (!waitw(s, &s.cready, (c + 1) & 1, status, 7)) break;
        gram(c + 1);
      }
      if (!waitw(s, &s.rready, ph, status, 8)) break;
      tc_fence_after();
      if (leader) {  // hi hi, lo hi, hi lo
        const uint64_t th = smem_desc(smem_u32(s.T[ph][0]), 16, 1024, kSwizzle128B);
        const uint64_t tl = smem_desc(smem_u32(s.T[ph][1]), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int x = 0; x < 3; ++x)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tb + kColKS, tb + kColR + 32 * (kk >> 1) + 8 * (kk & 1) + (x == 1 ? 16 : 0),
                   (x == 2 ? tl : th) + 2 * kk, id64, x + kk > 0);
      }
      commit(&s.udone, ph);
      if (!waitw(s, &s.uready, ph, status, 9)) break;
      tc_fence_after();
      if (leader) {
        const uint64_t dm = smem_desc(smem_u32(s.kq[c % 3][0]), 128 * 128, 1024, kSwizzle128B);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tb + kColS, tb + kColU2 + 32 * (kk >> 1) + 8 * (kk & 1) + 16 * x, dm + kk * 128,
                   idS, x + kk > 0);
        mma_commit(&s.supdone);
        mma_commit(&s.empty[c % 3]);
        const uint64_t dp = smem_desc(smem_u32(s.P[ph]), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(tb + kColPU, tb + kColR + 32 * (kk >> 1) + 8 * (kk & 1), dp + 2 * kk, id64, kk > 0);
      }
      commit(&s.pudone, ph);
    }
    // Leave no MMA in flight before TMEM is freed.
    if (lane == 0 && last_bar) mbar_wait(last_bar, last_par, kWaitLimit);
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ preparation
    const int pt = tid - kChain, pw = warp - 8;  // pw 0, 1: keys; 2, 3: queries
    const int tok = pt & 63;
    const bool isk = pt < 64;
    __nv_bfloat16 dtr[2] = {}, ber[2] = {};
    // lane l of the last warp has tokens 2 l and 2 l + 1; their gates are
    // fetched a chunk ahead
    auto fetch = [&](int c) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t t = (int64_t)c * kC + 2 * lane + e;
        if (t < len) {
          if (p.dt) dtr[e] = static_cast<const __nv_bfloat16 *>(p.dt)[(t0 + t) * p.dt_row + hd];
          ber[e] = static_cast<const __nv_bfloat16 *>(p.beta)[(t0 + t) * p.beta_row + hd];
        }
      }
    };
    const float Ah = p.dt ? p.A[hd] : 0.f;
    const float bias = p.dt && p.dt_bias ? p.dt_bias[hd] : 0.f;
    if (pw == 3) fetch(0);
    float gtot = 1.f;
    for (int c = 0; c < nch; ++c) {
      const int par = c & 1;
      const int64_t left = len - (int64_t)c * kC;
      const int nv = (int)(left < kC ? left : kC);
      bool ok = true;
      if (pw == 3) {
        double gs[2];
        float be[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l2 = 0.f, b = 0.f;
          if (2 * lane + e < nv) {
            if (p.dt) {
              float d = __bfloat162float(dtr[e]) + bias;
              if (p.flags & SSM_DT_SOFTPLUS) d = softplus(d);
              l2 = d * Ah * kLog2e;
              if (l2 < -256.f) l2 = -256.f;  // zero either way; keeps the sums exact
            }
            b = __bfloat162float(ber[e]);
            if (p.flags & GDR_BETA_SIGMOID) b = 1.f / (1.f + ex2(-b * kLog2e));
          }
          gs[e] = (double)l2;
          be[e] = b;
        }
        if (c + 1 < nch) fetch(c + 1);
        double sum = gs[0] + gs[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const double o = __shfl_up_sync(0xffffffffu, sum, off);
          if (lane >= off) sum += o;
        }
        const double g1 = sum, g0 = sum - gs[1];
        s.ghi[2 * lane] = (float)g0;
        s.glo[2 * lane] = (float)(g0 - (double)(float)g0);
        s.ghi[2 * lane + 1] = (float)g1;
        s.glo[2 * lane + 1] = (float)(g1 - (double)(float)g1);
        s.beta[2 * lane] = be[0];
        s.beta[2 * lane + 1] = be[1];
        // the chunk's decay multiplies the state once a chunk: exact
        gtot = (float)exp2(__shfl_sync(0xffffffffu, g1, 31));
      }
      // keys and queries: float16 of value x 2^-e, e the row's own, in place
      ok = waitw(s, &s.fullk[c % 3], (c / 3) & 1, status, 10);
      float nf = 0.f;
      {
        uint8_t *base = &s.kq[c % 3][0][0];
        uint4 raw[NP * 8];
        __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int i = 0; i < NP * 8; ++i) {
          raw[i] = *reinterpret_cast<const uint4 *>(base + (i >> 3) * (128 * 128) + sw128(pt, i & 7));
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e])));
        }
        const float m = fmaxf(__low2float(m2), __high2float(m2));
        int e = (int)(__float_as_uint(m) >> 23);  // biased exponent of the row
        e = e < 1 ? 1 : e > 253 ? 253 : e;
        const bool on = tok < nv;
        const float f = on ? __uint_as_float((uint32_t)(254 - e) << 23) : 0.f;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NP * 8; ++i) {
          uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (!on) w[x] = 0u;  // rows behind the end may hold anything
            const f2 y = mul2(mk2(bf16lo(w[x]), bf16hi(w[x])), mk2(f, f));
            ss = fmaf(y.x, y.x, ss);
            ss = fmaf(y.y, y.y, ss);
            w[x] = pack_h2(y.x, y.y);
          }
          *reinterpret_cast<uint4 *>(base + (i >> 3) * (128 * 128) + sw128(pt, i & 7)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_smem();
        if (on) {
          nf = __uint_as_float((uint32_t)e << 23);  // 2^e, without the norm
          if (p.flags & GDR_QK_L2NORM) nf = ss > 0.f ? 1.f / sqrtf(ss + p.l2_eps * f * f) : 0.f;
          if (ss != ss) nf = ss;
        }
        if (isk) s.nk[tok] = nf;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.cready);
      // the largest finite value of V
      ok = ok && waitw(s, &s.fullv[par], (c >> 1) & 1, status, 11);
      float vm = 0.f;
      {
        __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
        const uint4 *vp = reinterpret_cast<const uint4 *>(&s.v[par][0][0]);
#pragma unroll
        for (int i = 0; i < kC * kV / 8 / kPrep; ++i) {
          const int at = pt + kPrep * i;
          if (at / (kV / 8) < nv) {
            const uint4 u = vp[at];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e])));
          }
        }
        vm = fmaxf(__low2float(m2), __high2float(m2));
        if (__float_as_uint(vm) >= 0x7f800000u) {  // an infinity among them: look again
          vm = 0.f;
          const __nv_bfloat16 *ve = &s.v[par][0][0];
          for (int i = 0; i < kC * kV / 8 / kPrep; ++i)
            for (int e = 0; e < 8; ++e) {
              const int at = (pt + kPrep * i) * 8 + e;
              const float x = at / kV < nv ? fabsf(__bfloat162float(ve[at])) : 0.f;
              if (x < __uint_as_float(0x7f800000u)) vm = fmaxf(vm, x);
            }
        }
        vm = warp_max(vm);
      }
      if (prep_any(!ok)) break;  // (and: gates and key factors are written)
      // G; with it the chain is done with the chunk two before, whose places
      // the factors, T and P take
      ok = waitw(s, &s.gdone, par, status, 12);
      tc_fence_after();
      const float ghi = s.ghi[tok], glo = s.glo[tok];
      const float eg = ex2(ghi + glo);
      const float e31 = ex2((ghi - s.ghi[31]) + (glo - s.glo[31]));  // of tokens behind the first 32
      float nb = 0.f;
      if (isk) {
        const float b = s.beta[tok];
        nb = nf * nf * b;
        const float bv = nf * b, bk = nb * eg;
        const float cu = ex2((s.ghi[63] - ghi) + (s.glo[63] - glo));
        s.bv[par][tok] = bv;
        s.bk[par][tok] = bk;
        s.cu[par][tok] = cu;
        if (tok < 32) s.f31[tok] = ex2((s.ghi[31] - ghi) + (s.glo[31] - glo));
        const float mv = warp_max(fabsf(bv)), mk = warp_max(fabsf(bk));
        if (lane == 0) {
          s.bvmax[par][pw] = mv;
          s.bkmax[par][pw] = mk;
        }
      } else {
        const float cq = p.scale * nf;
        s.cqp[par][tok] = cq;
        s.cqe[par][tok] = cq * eg;
      }
      if (lane == 0) s.vmax[par][pw] = vm;
      if (pw == 3 && lane == 0) s.gC[par] = gtot;
      prep_sync();  // f31
      // A (float32, to be inverted) and P (float16): this row's columns of
      // its own 32-token block, and of the first block below it
      const int blk = pw & 1;
      const uint32_t grow = tb + ((uint32_t)(32 * pw) << 16) + kColG;
      const float rowf = isk ? nb : 1.f;
#pragma unroll 1
      for (int J = 0; J < 4; ++J) {  // 16 columns
        float x[16];
        if ((J >> 1) <= blk) {
          uint32_t r[16];
          tmem_ld16(grow + 16 * J, r);
          tmem_ld_wait();
          if ((J >> 1) == blk) {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const int j = 16 * J + q;
              const float d = (ghi - s.ghi[j]) + (glo - s.glo[j]);
              const bool in = isk ? j < tok : j <= tok;
              x[q] = in ? __uint_as_float(r[q]) * (rowf * ex2(d)) : 0.f;
            }
          } else {
            const float f = rowf * e31;
#pragma unroll
            for (int q = 0; q < 16; ++q) x[q] = __uint_as_float(r[q]) * (f * s.f31[16 * J + q]);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q) x[q] = 0.f;
        }
        if (isk) {
          if ((J >> 1) <= blk) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4 *>(&s.Am[tok][16 * J + 4 * q]) =
                  make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<uint4 *>(s.P[par] + sw128(tok, 2 * J + q)) =
                make_uint4(pack_h2(x[8 * q], x[8 * q + 1]), pack_h2(x[8 * q + 2], x[8 * q + 3]),
                           pack_h2(x[8 * q + 4], x[8 * q + 5]), pack_h2(x[8 * q + 6], x[8 * q + 7]));
        }
      }
      tc_fence_before();
      float tm = 0.f;
      if (isk) {
        // the inverse of this warp's diagonal block, a column a lane
        __syncwarp();
        const int o = 32 * pw;
        f2 x[16];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          f2 a0 = mk2(lane == i ? 1.f : 0.f, 0.f), a1 = mk2(0.f, 0.f);
#pragma unroll
          for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
            const float4 a = *reinterpret_cast<const float4 *>(&s.Am[o + i][o + 4 * j4]);
            // (columns from i on hold zeros, or x not yet set is not read)
            if (4 * j4 + 1 < i) a0 = fma2(mk2(-a.x, -a.y), x[2 * j4], a0);
            else a0.x = fmaf(-a.x, x[2 * j4].x, a0.x);
            if (4 * j4 + 3 < i) a1 = fma2(mk2(-a.z, -a.w), x[2 * j4 + 1], a1);
            else if (4 * j4 + 2 < i) a1.x = fmaf(-a.z, x[2 * j4 + 1].x, a1.x);
          }
          a0 = add2(a0, a1);
          const float xi = a0.x + a0.y;
          tm = fmaxf(tm, fabsf(xi));
          if (i & 1) x[i / 2].y = xi; else x[i / 2].x = xi;
        }
        __syncwarp();  // every lane has read the block
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s.Am[o + 2 * i][o + lane] = x[i].x;
          s.Am[o + 2 * i + 1][o + lane] = x[i].y;
        }
      }
      prep_sync();
      {  // X = A21 T11, rows 8 pw .. + 8, a column a lane
        f2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = mk2(0.f, 0.f);
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {
          const f2 t01 = mk2(s.Am[4 * j4][lane], s.Am[4 * j4 + 1][lane]);
          const f2 t23 = mk2(s.Am[4 * j4 + 2][lane], s.Am[4 * j4 + 3][lane]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 a = *reinterpret_cast<const float4 *>(&s.Am[32 + 8 * pw + i][4 * j4]);
            acc[i] = fma2(mk2(a.x, a.y), t01, acc[i]);
            acc[i] = fma2(mk2(a.z, a.w), t23, acc[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s.Am[8 * pw + i][32 + lane] = acc[i].x + acc[i].y;
      }
      prep_sync();
      {  // T21 = -T22 X
        f2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = mk2(0.f, 0.f);
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {
          const f2 t01 = mk2(s.Am[4 * j4][32 + lane], s.Am[4 * j4 + 1][32 + lane]);
          const f2 t23 = mk2(s.Am[4 * j4 + 2][32 + lane], s.Am[4 * j4 + 3][32 + lane]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 a = *reinterpret_cast<const float4 *>(&s.Am[32 + 8 * pw + i][32 + 4 * j4]);
            acc[i] = fma2(mk2(a.x, a.y), t01, acc[i]);
            acc[i] = fma2(mk2(a.z, a.w), t23, acc[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = -(acc[i].x + acc[i].y);
          tm = fmaxf(tm, fabsf(t));
          s.Am[32 + 8 * pw + i][lane] = t;
        }
        tm = warp_max(tm);
        if (lane == 0) s.tmax[par][pw] = tm;
      }
      prep_sync();
      {  // T to float16 pairs: row pt / 2, half pt % 2 (above the diagonal blocks it stays zero)
        const int row = pt >> 1, hf = pt & 1;
        if (hf <= (row >> 5)) {
          const int eT = scale_exp(max_of(s.tmax[par], 4));
          const f2 sc = mk2(pow2i(eT < 0 ? eT : 0), pow2i(eT < 0 ? eT : 0));
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 a = *reinterpret_cast<const float4 *>(&s.Am[row][32 * hf + 8 * q]);
            const float4 b = *reinterpret_cast<const float4 *>(&s.Am[row][32 * hf + 8 * q + 4]);
            uint4 hi, lo;
            split_h2(mul2(mk2(a.x, a.y), sc), hi.x, lo.x);
            split_h2(mul2(mk2(a.z, a.w), sc), hi.y, lo.y);
            split_h2(mul2(mk2(b.x, b.y), sc), hi.z, lo.z);
            split_h2(mul2(mk2(b.z, b.w), sc), hi.w, lo.w);
            *reinterpret_cast<uint4 *>(s.T[par][0] + sw128(row, 4 * hf + q)) = hi;
            *reinterpret_cast<uint4 *>(s.T[par][1] + sw128(row, 4 * hf + q)) = lo;
          }
        }
      }
      fence_async_smem();
      if (prep_any(!ok)) break;
      if (lane == 0) mbar_arrive(&s.tready[par]);
    }
  } else {
    // ------------------------------------------------------------ the chain
    __nv_bfloat16 *yb = static_cast<__nv_bfloat16 *>(p.y) + (t0 * p.H + hd) * p.V + v0 + cv;
    const int64_t yrow = p.H * p.V;
    for (int c = 0; c < nch; ++c) {
      const int par = c & 1;
      const uint32_t ph = par;
      const int64_t left = len - (int64_t)c * kC;
      const int nv = (int)(left < kC ? left : kC);
      // R: the chunk's factors, KS and V
      if (!waitw(s, &s.tready[par], (c >> 1) & 1, status, 13)) break;
      if (c > 0 && !waitw(s, &s.sready, ph ^ 1, status, 14)) break;  // smax of every warp
      const float smax = max_of(s.smax[par ^ 1], 8);
      const float bvm = fmaxf(s.bvmax[par][0], s.bvmax[par][1]);
      const float bkm = fmaxf(s.bkmax[par][0], s.bkmax[par][1]);
      // |S^T k^| <= sum |k^| smax <= 2 KD smax
      const int eR = scale_exp(bvm * max_of(s.vmax[par], 4) + bkm * (2.f * KD) * smax);
      if (!waitw(s, &s.ksdone, ph, status, 15)) break;
      tc_fence_after();
      float m = 0.f;
      {
        const float fR = pow2i(eR), fK = -pow2i(-eS);
        const f2 fR2 = mk2(fR, fR), fK2 = mk2(fK, fK);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[16], hi[8], lo[8];
          tmem_ld16(tb + lane_base + kColKS + 32 * ch + 16 * i, r);
          const int j0 = 32 * ch + 16 * i;
          float vv[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) vv[q] = __bfloat162float(s.v[par][j0 + q][cv]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 bv = *reinterpret_cast<const float4 *>(&s.bv[par][j0 + 4 * q]);
            const float4 bk = *reinterpret_cast<const float4 *>(&s.bk[par][j0 + 4 * q]);
            f2 x[2];
            x[0] = mul2(mk2(bv.x, bv.y), mk2(vv[4 * q], vv[4 * q + 1]));
            x[1] = mul2(mk2(bv.z, bv.w), mk2(vv[4 * q + 2], vv[4 * q + 3]));
            x[0] = fma2(mul2(mk2(bk.x, bk.y), fK2),
                        mk2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])), x[0]);
            x[1] = fma2(mul2(mk2(bk.z, bk.w), fK2),
                        mk2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])), x[1]);
            x[0] = mul2(x[0], fR2);
            x[1] = mul2(x[1], fR2);
            if (nv < kC) {  // rows behind the end may hold anything
              const int j = j0 + 4 * q;
              if (j >= nv) x[0].x = 0.f;
              if (j + 1 >= nv) x[0].y = 0.f;
              if (j + 2 >= nv) x[1].x = 0.f;
              if (j + 3 >= nv) x[1].y = 0.f;
            }
            m = fmaxf(fmaxf(m, fabsf(x[0].x)), fabsf(x[0].y));
            m = fmaxf(fmaxf(m, fabsf(x[1].x)), fabsf(x[1].y));
            split_h2(x[0], hi[2 * q], lo[2 * q]);
            split_h2(x[1], hi[2 * q + 1], lo[2 * q + 1]);
          }
          tmem_st8(tb + lane_base + kColR + 32 * ch + 8 * i, hi);
          tmem_st8(tb + lane_base + kColR + 32 * ch + 16 + 8 * i, lo);
        }
      }
      m = warp_max(m);
      if (lane == 0) s.rmax[par][warp] = m;  // of R 2^eR
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.rready);
        mbar_arrive(&s.vempty[par]);
      }
      // U and U'
      if (!waitw(s, &s.rready, ph, status, 16)) break;  // rmax of every warp
      const float tmax = max_of(s.tmax[par], 4);
      int eT = scale_exp(tmax);
      eT = eT < 0 ? eT : 0;
      // |U| <= sum |T| |R| <= 64 tmax rmax
      const float rm = max_of(s.rmax[par], 8) * (tmax * pow2i(eT));
      int eU = scale_exp(64.f * rm);    // of U 2^(eR + eT)
      const float fU = pow2i(eU);
      eU += eR + eT;
      if (!waitw(s, &s.udone, ph, status, 17)) break;
      tc_fence_after();
      m = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t r[16], uh[8], hi[8], lo[8];
        tmem_ld16(tb + lane_base + kColKS + 32 * ch + 16 * i, r);
        tmem_ld_wait();
        const f2 fU2 = mk2(fU, fU);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 cu = *reinterpret_cast<const float4 *>(&s.cu[par][32 * ch + 16 * i + 4 * q]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f2 x = mul2(mk2(__uint_as_float(r[4 * q + 2 * e]), __uint_as_float(r[4 * q + 2 * e + 1])),
                        fU2);
            uh[2 * q + e] = pack_h2(x.x, x.y);
            x = mul2(x, e ? mk2(cu.z, cu.w) : mk2(cu.x, cu.y));
            m = fmaxf(fmaxf(m, fabsf(x.x)), fabsf(x.y));
            split_h2(x, hi[2 * q + e], lo[2 * q + e]);
          }
        }
        tmem_st8(tb + lane_base + kColR + 32 * ch + 8 * i, uh);
        tmem_st8(tb + lane_base + kColU2 + 32 * ch + 8 * i, hi);
        tmem_st8(tb + lane_base + kColU2 + 32 * ch + 16 + 8 * i, lo);
      }
      m = warp_max(m);
      if (lane == 0) s.umax[par][warp] = m;  // of U' 2^eU
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.uready);
      // the state
      if (!waitw(s, &s.uready, ph, status, 18)) break;  // umax of every warp
      const float gC = s.gC[par];
      const int eSo = eS;
      const float fD = pow2i(-eU);
      // |dS| <= sum |k^| |U'| <= 128 umax
      eS = scale_exp(fabsf(gC) * smax + 128.f * (max_of(s.umax[par], 8) * fD));
      if (!waitw(s, &s.supdone, ph, status, 19)) break;
      tc_fence_after();
      m = 0.f;
      {
        const f2 g2 = mk2(gC, gC), fD2 = mk2(fD, fD), fS2 = mk2(pow2i(eS), pow2i(eS));
        uint32_t hi[KH / 2], lo[KH / 2];
#pragma unroll
        for (int i = 0; i < KH / 16; ++i) {
          uint32_t r[16];
          tmem_ld16(tb + lane_base + kColS + ch * KH + 16 * i, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f2 &x = st[8 * i + j];
            x = fma2(x, g2, mul2(mk2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), fD2));
            m = fmaxf(fmaxf(m, fabsf(x.x)), fabsf(x.y));
            split_h2(mul2(x, fS2), hi[8 * i + j], lo[8 * i + j]);
          }
        }
        // (this warp's own dS columns, all read)
#pragma unroll
        for (int i = 0; i < KH / 32; ++i) {
          tmem_st16(tb + lane_base + kColS + ch * KH + 16 * i,
                    *reinterpret_cast<const uint32_t(*)[16]>(&hi[16 * i]));
          tmem_st16(tb + lane_base + kColS + ch * KH + KH / 2 + 16 * i,
                    *reinterpret_cast<const uint32_t(*)[16]>(&lo[16 * i]));
        }
      }
      m = warp_max(m);
      if (lane == 0) s.smax[par][warp] = m;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sready);
      // y, under the next chunk's KS
      if (!waitw(s, &s.pudone, ph, status, 20)) break;
      tc_fence_after();
      const f2 fQ2 = mk2(pow2i(-eSo), pow2i(-eSo)), fP2 = mk2(pow2i(-eU), pow2i(-eU));
      f2 o[16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t r[16], u[16];
        tmem_ld16(tb + lane_base + kColQS + 32 * ch + 16 * i, r);
        tmem_ld16(tb + lane_base + kColPU + 32 * ch + 16 * i, u);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 ce = *reinterpret_cast<const float4 *>(&s.cqe[par][32 * ch + 16 * i + 4 * q]);
          const float4 cp = *reinterpret_cast<const float4 *>(&s.cqp[par][32 * ch + 16 * i + 4 * q]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 4 * q + 2 * e;
            const f2 qs = mul2(mk2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), fQ2);
            const f2 pu = mul2(mk2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), fP2);
            o[8 * i + 2 * q + e] = fma2(e ? mk2(ce.z, ce.w) : mk2(ce.x, ce.y), qs,
                                        mul2(e ? mk2(cp.z, cp.w) : mk2(cp.x, cp.y), pu));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.ofree);
      if (live) {
        __nv_bfloat16 *yp = yb + ((int64_t)c * kC + 32 * ch) * yrow;
        const int n = nv - 32 * ch;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n) yp[j * yrow] = __float2bfloat16_rn((j & 1) ? o[j / 2].y : o[j / 2].x);
      }
    }
    if (p.h_last && live && !*(volatile int *)&s.abort) {
#pragma unroll
      for (int i = 0; i < KH; ++i) {
        const int r = ch * KH + i;
        if (r < p.K) p.h_last[so + (int64_t)r * p.V + cv] = (i & 1) ? st[i / 2].y : st[i / 2].x;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tb, kTmemCols);
}

bool encode(CUtensorMap *m, const void *ptr, int64_t dim, int64_t heads, int64_t rows, int64_t row,
            uint32_t box, CUtensorMapSwizzle sw) {
  const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)dim * 2, (uint64_t)row * 2};
  const uint32_t b[3] = {box, 1, kC};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, b, sw);
}

template <int KD>
cudaError_t launch(const GdrTcParams &q, const CUtensorMap &mK, const CUtensorMap &mQ,
                   const CUtensorMap &mV, unsigned blocks, cudaStream_t s) {
  const size_t smem = sizeof(GdrSmem<KD>) + 1024;
  // (set on every call: the attribute belongs to the current device)
  cudaError_t e = cudaFuncSetAttribute(gdr_tc_kernel<KD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  gdr_tc_kernel<KD><<<blocks, kThreads, smem, s>>>(mK, mQ, mV, q);
  return cudaGetLastError();
}

}  // namespace

bool gdr_tc_supported(const GdrParams &p) {
  // bf16; whole 16-byte steps for the TMA; 32-bit TMA coordinates
  return p.io == 1 && p.rows > 0 && p.nseq > 0 && p.K <= 128 && p.K % 8 == 0 && p.V % 8 == 0 && p.q_row % 8 == 0 &&
         p.k_row % 8 == 0 && p.v_row % 8 == 0 && p.rows + kC < (1ll << 31) &&
         p.nseq * p.H * ((p.V + kV - 1) / kV) < (1ll << 31);
}

cudaError_t launch_gdr_tc(const GdrParams &p, int *status, cudaStream_t s) {
  GdrTcParams q;
  q.p = p;
  q.vtiles = (p.V + kV - 1) / kV;
  q.status = status;
  CUtensorMap mK, mQ, mV;
  if (!encode(&mK, p.k, p.K, p.Hk, p.rows, p.k_row, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&mQ, p.q, p.K, p.Hk, p.rows, p.q_row, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&mV, p.v, p.V, p.H, p.rows, p.v_row, kV, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const unsigned blocks = (unsigned)(p.nseq * p.H * q.vtiles);
  return p.K <= 64 ? launch<64>(q, mK, mQ, mV, blocks, s) : launch<128>(q, mK, mQ, mV, blocks, s);
}

}  // namespace ssm
