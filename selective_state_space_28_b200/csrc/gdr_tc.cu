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
// Two kernels.  The first is parallel over chunks: for each and each value head
// it makes what needs no state, T = (I + A)^-1 diag(b), P_ij = e^(g_i - g_j)
// q_i.k_j (j <= i) and the tokens' factors, and leaves them in the workspace as
// the second one's shared-memory image (26 KB), with the chunk's scaled keys for
// each key head.  The second walks the chunks, one CTA per (sequence, value
// head, 128 value columns).  A TMEM lane is a value column, so every product has
// M = 128 and its A operand (S, R, U, transposed) comes from TMEM, where the
// thread that owns the lane wrote it; tokens and key dimensions are columns:
//
//   KS = S^T K^T                      B = the keys, K-major
//   U  = R T^T, R = v - e^g KS        B = T
//   Y  = S^T (e^g Q)^T + U P^T        B = the queries with their decays, and P
//   dS = U'^T K, U'_j = e^(g_63 - g_j) U_j   B = the keys, MN-major
//
// The chain KS -> R -> U -> U' -> dS -> S bounds it: three products one behind
// the other and the elementwise work between them, each with its latency
// (commit, wake-up, TMEM loads and stores).  Y and the next chunk's conversion
// run beside it; the state goes in two halves of key dimensions, so that KS of
// one half runs under the elementwise work of the other.  8 x 2048 tokens of 32
// heads, 128 x 128: 117 us + 200 us, 5200 cycles a chunk, 1600 of them the
// chain's products.
//
// Precision.  The state is kept and returned in float32, so what feeds it may
// not round to 16 bits: the products run on float16 pairs, x = hi + lo (22
// bits), two (KS, dS) or three (U) products for one.  y is returned in
// bfloat16: for Y the hi parts alone do (2^-11 of a term beside the
// result's 2^-8).  float16 has the digits but not the range, so every operand
// is scaled by powers of two: a key or query by its own (its norm comes to
// 1 .. 2; a bfloat16's 8 bits stay exact down to 2^-17 of that), the norm
// factors being applied in float32, and S, R, U each by one for 32 value
// columns and a chunk, from bounds on the measured largest S and v, so that the largest
// value stays below 2^15 and one 2^-18 of it still has 22 bits.  A warp's
// lanes that are not finite do not count toward the maxima.
//
// Few long sequences are cut into segments (segments_of).
//
// Every wait is bounded; one that runs out sets the status word, its warp
// waits no more, the others' waits run out in turn, and the CTA frees its TMEM.
#include <cuda_fp16.h>

#include <atomic>

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
constexpr long long kWaitLimit = 2000000000ll;  // cycles (about a second)
constexpr int kAm = 68;   // row stride of A / T in float32 (a row a lane: no bank conflicts)

// What the first kernel leaves for a chunk and head.
struct Rec {
  uint8_t T[2][kC * 128];  // hi, lo: 64 x 64 float16, 128-byte swizzled rows
  uint8_t P[kC * 128];
  float ek[kC], cu[kC], cq[kC];  // factors of KS (negative), U' and y
  float fq[kC];                  // of queries: powers of two and decays
  // e^g_63; bounds of ek |k| and of T's rows (scaled); T's exponent; the largest
  // write strength, at least 1, of a chunk that contracts the state, or 0
  float gC, ekn, tn, eT, con;
  float expired;  // a wait ran out
  float pad[10];
};
// and, for a chunk and key head, the keys as scaled float16: KD / 64 slabs of
// 64 x 64, 128-byte swizzled rows.
constexpr size_t kSlab = kC * 128;
constexpr size_t kRecT = 2 * kC * 128;
static_assert(sizeof(Rec) == 25664 && sizeof(Rec) % 16 == 0, "a record is copied in 16-byte units");

struct GdrTcParams {
  GdrParams p;
  int64_t vtiles;
  int64_t chunks;  // of a sequence (dense), or 0: packed
  int64_t share;   // value heads that the first kernel makes the records of together
  int64_t units;   // such groups of records
  uint8_t *rec;   // [slot][head]
  uint8_t *keys;  // [slot][key head][slab]
  int *status;
  // A sequence cut into segments (see segments_of): how many, which pass, and
  // the states entering segments 1 .. and the maps of segments 1 .. nseg - 2,
  // [segment][sequence][head][key side first].
  int nseg;
  float *seg_state, *seg_map;
};

// The record of the chunk that starts at row t0 of sequence `seq`, its chunk c.
// Packed, a sequence's first chunk has one of its own, number rows / 64 + seq, and
// a later chunk the number t0 / 64 - 1, whatever the order of the sequences: the 64
// rows before such a chunk are its own sequence's, so that among sequences that are
// apart no two such chunks start within the same 64 rows.
__device__ __forceinline__ int64_t record_slot(const GdrTcParams &tp, int64_t seq, int64_t t0, int64_t c) {
  return tp.chunks ? seq * tp.chunks + c : c == 0 ? tp.p.rows / kC + seq : t0 / kC - 1;
}

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
// Named barrier over the two chain warps of one lane quarter.
__device__ __forceinline__ void pair_sync(int quarter) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
}
// Untiled copies, sizes and addresses in 16-byte units.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
               : "memory");
}
template <int N> __device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

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
// x = hi + lo in float16 pairs (x - hi by a multiply-add that takes float16
// factors: at full rate, where a conversion back and a packed sum take three
// times as long).
__device__ __forceinline__ void split_h2(f2 x, uint32_t &hi, uint32_t &lo) {
  hi = pack_h2(x.x, x.y);
  float a, b;
  asm("{\n\t.reg .f16 h0, h1, m;\n\tmov.b32 {h0, h1}, %2;\n\tmov.b16 m, 0xbc00;\n\t"
      "fma.rn.f32.f16 %0, h0, m, %3;\n\tfma.rn.f32.f16 %1, h1, m, %4;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(hi), "f"(x.x), "f"(x.y));
  lo = pack_h2(a, b);
}
// max(|a|, |b|) of float16 pairs (the sign bits are not part of the result).
__device__ __forceinline__ uint32_t maxabs_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t maxabs_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two bfloat16 times a bfloat16, plus c, in float32.
__device__ __forceinline__ f2 fma_bf16x2(uint32_t x, uint32_t y, f2 c) {
  f2 d;
  asm("{\n\t.reg .b16 x0, x1, y0, y1;\n\tmov.b32 {x0, x1}, %2;\n\tmov.b32 {y0, y1}, %3;\n\t"
      "fma.rn.f32.bf16 %0, x0, y0, %4;\n\tfma.rn.f32.bf16 %1, x1, y1, %5;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(x), "r"(y), "f"(c.x), "f"(c.y));
  return d;
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
// The warp's maximum of finite non-negative values; a lane's inf counts as 0.
__device__ __forceinline__ float warp_max(float m) {
  const uint32_t b = __float_as_uint(m);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, b < 0x7f800000u ? b : 0u));
}


// ---------------------------------------------------------- what needs no state
constexpr int kPrepThreads = 128;
constexpr int kSearched = 1024;  // packed sequences looked through for a record's (more: bisected)

template <int KD> struct __align__(1024) PrepSmem {
  union {
    uint8_t kq[KD / 64][128 * 128];  // [slab]: rows 0-63 keys, 64-127 queries
    struct {                         // once their products are there
      union {
        float Am[kC][kAm];  // A, then T
        uint8_t T[kRecT];
      };
      __align__(16) uint8_t rest[sizeof(Rec) - kRecT];
    };
  };
  f2 g[2][kC];  // running sum of log2 of the decays, hi and lo; a head's and the next's
  float beta[2][kC], f[kC], h[kC], qq[kC], bv[kC];
  float ekn[2], tn[4];
  int found[2][4];
  uint64_t full, done;
  uint32_t taddr;
};

// C (+)= A B in float32 on the tensor cores' tf32: both operands as hi + lo,
// three products.  C [16 x 8], A [16 x 8] rows and B [8 x 8] in mma.m16n8k8's
// lane layout.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;  // 11 bits, to nearest
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// out [16 MT x 8] = a [16 MT x 8 KT] b [8 KT x 8], rows of kAm floats.
// k starts at step k0 (b holds zeros before it); LOWER: a is lower triangular.
template <int MT, int KT, bool LOWER>
__device__ __forceinline__ void small_product(const float *a, const float *b, int k0, float (&out)[MT][4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[m][e] = 0.f;
#pragma unroll 2
  for (int k = k0; k < KT; ++k) {
    uint32_t bh[2], bl[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) split_tf32(b[(8 * k + t + 4 * e) * kAm + r], bh[e], bl[e]);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (LOWER && k >= 2 * m + 2) continue;
      uint32_t ah[4], al[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        split_tf32(a[(16 * m + r + 8 * (e & 1)) * kAm + 8 * k + t + 4 * (e >> 1)], ah[e], al[e]);
      mma_tf32(out[m], al, bh);
      mma_tf32(out[m], ah, bl);
      mma_tf32(out[m], ah, bh);
    }
  }
}
template <int MT>
__device__ __forceinline__ void put_product(float *o, const float (&c)[MT][4], float sign) {
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      *reinterpret_cast<float2 *>(&o[(16 * m + r + 8 * e) * kAm + 2 * t]) =
          make_float2(sign * c[m][2 * e], sign * c[m][2 * e + 1]);
}

// CTAs of 128 threads, six to an SM, each over (chunk, value head) units.  Row pt
// of [K; Q] [K]^T is thread pt's (TMEM lane pt): keys' rows make A, queries' P.
// The inverse goes by blocks: the four 16 x 16 diagonal blocks by forward
// substitution, a column a lane; then twice -T22 A21 T11 for the block below two
// of them, the products as float32 on mma (a multiply-add version read its
// operands from shared memory four times as often, which bound the kernel: 4200
// cycles a unit of SM time).  Bound by issue: 8700 warp instructions a unit, half
// of the slots taken; barriers and instruction fetch are the largest stalls.
template <int KD>
__global__ void __launch_bounds__(kPrepThreads, 6)
    gdr_prep_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mQ,
                    const GdrTcParams tp) {
  constexpr int NP = KD / 64;
  using Smem = PrepSmem<KD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const GdrParams &p = tp.p;
  const int pt = threadIdx.x, pw = pt >> 5, lane = pt & 31;
  // (cleared before a CTA of the next kernel can start; what runs out here is
  // left in the records)
  if (blockIdx.x == 0 && pt == 0) *tp.status = 0;
  __threadfence();
  pdl_launch_dependents();
  if (pt == 0) {
    mbar_init(&s.full, 1);
    mbar_init(&s.done, 1);
    fence_mbar_init();
  }
  if (pw == 1) {
    tmem_alloc(&s.taddr, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.taddr;
  uint32_t ph = 0, round = 0;
  bool ok = true;
  for (int64_t unit = blockIdx.x; unit < tp.units; unit += gridDim.x) {
    // the sequence and chunk of this record
    const int64_t groups = p.H / tp.share, rs = unit / groups, hd0 = unit % groups * tp.share;
    int64_t seq, c, slot, t0, len;
    if (tp.chunks) {
      seq = rs / tp.chunks;
    } else {
      if (rs >= p.rows / kC) {  // a first chunk
        seq = rs - p.rows / kC;
      } else if (p.nseq <= kSearched) {
        // (among all: bounds that are out of order and sequences that are skipped
        // leave the others right)
        round ^= 1;
        int at = -1;
        for (int64_t i = pt; i < p.nseq; i += kPrepThreads) {
          const int64_t b = p.cu[i], e = p.cu[i + 1], first = b / kC;
          if (b < 0 || e <= b || e > p.rows || first > rs || rs >= first + (e - b - 1) / kC) continue;
          if (!p.slots || (p.slots[i] >= 0 && p.slots[i] < p.state_rows)) at = (int)i;
        }
        at = __reduce_max_sync(0xffffffffu, at);
        if (lane == 0) s.found[round][pw] = at;
        __syncthreads();
        const int(&f)[4] = s.found[round];
        seq = max(max(f[0], f[1]), max(f[2], f[3]));
      } else {
        int64_t lo = 0, hi = p.nseq - 1;
        while (lo < hi) {
          const int64_t mid = (lo + hi + 1) >> 1;
          if (p.cu[mid] / kC <= rs) lo = mid;
          else hi = mid - 1;
        }
        seq = p.cu[lo] / kC <= rs ? lo : -1;
      }
      if (seq < 0) continue;
    }
    if (!gdr_sequence(p, seq, slot, t0, len)) continue;
    c = tp.chunks ? rs - seq * tp.chunks : rs >= p.rows / kC ? 0 : rs - t0 / kC + 1;
    if (c < 0 || c * kC >= len) continue;
    const int64_t left = len - c * kC;
    const int nv = (int)(left < kC ? left : kC);
    t0 += c * kC;
    const int64_t g = hd0 / (p.H / p.Hk);

    if (pt == 0) {
      // (the records before have left the shared memory)
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      mbar_expect_tx(&s.full, NP * 128 * 128);
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        tma_load_3d(s.kq[n], &mK, &s.full, 64 * n, (int)g, (int)t0);
        tma_load_3d(s.kq[n] + kC * 128, &mQ, &s.full, 64 * n, (int)g, (int)t0);
      }
    }
    __syncwarp();
    // the gates of a head, by the last warp: lane l has tokens 2 l and 2 l + 1
    int64_t g63x = 0;
    float con = 0.f;
    auto gates = [&](int64_t hd, int buf) {
      float dtv[2] = {}, be[2] = {};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (2 * lane + e < nv) {
          const int64_t at = t0 + 2 * lane + e;
          if (p.dt) dtv[e] = ld(static_cast<const __nv_bfloat16 *>(p.dt) + at * p.dt_row + hd);
          be[e] = ld(static_cast<const __nv_bfloat16 *>(p.beta) + at * p.beta_row + hd);
        }
      }
      const float Ah = p.dt ? p.A[hd] : 0.f;
      const float bias = p.dt && p.dt_bias ? p.dt_bias[hd] : 0.f;
      // log2 of the decays summed in fixed point, 2^-44 a unit: exact, and the
      // sums of 64 fit (each at least -256: zero either way)
      int64_t gs[2];
      bool fine = (p.flags & GDR_QK_L2NORM) != 0;
      float bmax = 1.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l2 = 0.f, b = 0.f;
        if (2 * lane + e < nv) {
          if (p.dt) {
            float d = dtv[e] + bias;
            if (p.flags & SSM_DT_SOFTPLUS) d = softplus(d);
            l2 = d * Ah * kLog2e;
          }
          b = (p.flags & GDR_BETA_SIGMOID) ? 1.f / (1.f + ex2(-be[e] * kLog2e)) : be[e];
          if (l2 != l2) b = l2;  // (not a number: seen in everything written)
          l2 = fmaxf(l2, -256.f);
        }
        gs[e] = __float2ll_rn(fminf(l2, 256.f) * 17592186044416.f);
        s.beta[buf][2 * lane + e] = b;
        fine = fine && l2 <= 0.f && b >= 0.f && b <= 2.f;
        bmax = fmaxf(bmax, b);
      }
      fine = __all_sync(0xffffffffu, fine);
      con = fine ? warp_max(bmax) : 0.f;
      int64_t sum = gs[0] + gs[1];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
      }
      g63x = __shfl_sync(0xffffffffu, sum, 31);
      // hi: multiples of 2^-10 (24 bits); lo: the rest below, in 2^-34
      auto parts = [](int64_t g) {
        return mk2((float)(int)(g >> 34) * 0.0009765625f,
                   (float)(int)((g & ((1ll << 34) - 1)) >> 10) * 5.8207660913467407e-11f);
      };
      s.g[buf][2 * lane] = parts(sum - gs[1]);
      s.g[buf][2 * lane + 1] = parts(sum);
    };
    if (pw == 3) gates(hd0, 0);
    ok = mbar_wait(&s.full, ph, kWaitLimit) && ok;
    if (pw == 0) {
      if (elect_one()) {
        const uint64_t d = smem_desc(smem_u32(s.kq[0]), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk) {
          const uint64_t o = (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4);
          mma_ss(tb, d + o, d + o, idesc_bf16_f32(128, 64, false, false), kk > 0);
        }
        mma_commit(&s.done);
      }
      __syncwarp();
    }
    {  // |q|^2, two threads a query (|k|^2 is on G's diagonal)
      const int row = pt >> 1, hf = pt & 1;
      f2 a = mk2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < KD / 16; ++i) {
        // (the halves' accesses lie in different banks)
        const int ch = NP == 2 ? 8 * hf + (i ^ (4 * hf)) : hf * (KD / 16) + i;
        const uint4 u = *reinterpret_cast<const uint4 *>(&s.kq[ch >> 3][0] + sw128(kC + row, ch & 7));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) a = fma_bf16x2(w[e], w[e], a);
      }
      float n2 = a.x + a.y;
      n2 += __shfl_xor_sync(0xffffffffu, n2, 1);
      if (hf == 0) s.qq[row] = n2;
    }
    ok = mbar_wait(&s.done, ph, kWaitLimit) && ok;
    ph ^= 1;
    tc_fence_after();
    __syncthreads();  // the gates, |q|^2; every thread is done with the rows

    const int tok = pt & 63;
    const bool isk = pt < 64, on = tok < nv;
    const uint32_t grow = tb + ((uint32_t)(32 * pw) << 16);
    // of G this row's columns of its own 32-token block; own: of its 16-token block
    const int blk = pw & 1;
    const bool up = lane >= 16;  // the second of the two 16-token blocks
    float n2, f = 0.f, nf = 0.f;
    for (int hj = 0; hj < tp.share; ++hj) {  // the value heads that share these keys
      const int64_t hd = hd0 + hj;
      const int gb = hj & 1;
      uint32_t r0[16], own[16];
      {
        uint32_t r1[16];
        tmem_ld16(grow + 32 * blk, r0);
        tmem_ld16(grow + 32 * blk + 16, r1);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q) own[q] = up ? r1[q] : r0[q];
      }
      if (hj == 0) {
        if (isk) {
          uint32_t t[8];  // own[lane & 15], bit by bit of the index
#pragma unroll
          for (int q = 0; q < 8; ++q) t[q] = lane & 8 ? own[q + 8] : own[q];
#pragma unroll
          for (int q = 0; q < 4; ++q) t[q] = lane & 4 ? t[q + 4] : t[q];
#pragma unroll
          for (int q = 0; q < 2; ++q) t[q] = lane & 2 ? t[q + 2] : t[q];
          n2 = __uint_as_float(lane & 1 ? t[1] : t[0]);
        } else {
          n2 = s.qq[tok];
        }
        // the row's power of two f = 2^-e, |row| f in 1 .. 2; its norm factor beside
        // rows scaled so
        int e = ((int)((__float_as_uint(n2) >> 23) & 255u) - 127) >> 1;
        e = !(n2 > 0.f) ? 0 : e < -60 ? -60 : e > 60 ? 60 : e;
        if (on) {
          f = pow2i(-e);
          nf = pow2i(e);
          if (p.flags & GDR_QK_L2NORM) {
            const float a = n2 + p.l2_eps, r = rsqrtf(a);
            // (one Newton step on the hardware's; infinite norms give 0)
            nf = n2 == 0.f || !(r > 0.f) ? 0.f : nf * (r * fmaf(-0.5f * a * r, r, 1.5f));
          }
          if (n2 != n2) nf = n2;
        }
      }
      if (hj > 0) {  // the head's before has left the shared memory
        if (pt == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncthreads();
      }
      const f2(&sg)[kC] = s.g[gb];
      const f2 gi = sg[tok], g63 = sg[63], gend = sg[tok | 15];
      const float eg = ex2(gi.x + gi.y);
      float *fac = reinterpret_cast<float *>(s.rest + (offsetof(Rec, ek) - kRecT));
      float rowf = f;
      if (isk) {
        const float b = s.beta[gb][tok];
        rowf = nf * nf * b * f;
        s.bv[tok] = nf * b;
        fac[0 * kC + tok] = -nf * eg;                              // ek
        fac[1 * kC + tok] = ex2((g63.x - gi.x) + (g63.y - gi.y));  // cu
        s.f[tok] = f;
        s.h[tok] = f * ex2((gend.x - gi.x) + (gend.y - gi.y));
        const float m = warp_max(2.f * nf * eg);
        if (lane == 0) s.ekn[pw] = m;
      } else {
        fac[2 * kC + tok] = p.scale * nf;  // cq
        fac[3 * kC + tok] = f * eg;        // fq
      }
      __syncthreads();  // f, h
      if (hd % (p.H / p.Hk) == 0) {  // the keys, scaled; rows behind the end may hold anything
        uint8_t *out = tp.keys + (rs * p.Hk + g) * (int64_t)(NP * kSlab);
#pragma unroll
        for (int i = 0; i < NP * 4; ++i) {
          const int at = (i & 3) * kPrepThreads + pt;  // 16 bytes of the slab: any swizzle
          const uint4 u = *reinterpret_cast<const uint4 *>(&s.kq[i >> 2][16 * at]);
          const float fr = s.f[at >> 3];
          const uint32_t f2x = __byte_perm(__float_as_uint(fr), 0, 0x3232);  // (a power of two: exact)
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2 y = fma_bf16x2(w[e], f2x, mk2(0.f, 0.f));
            w[e] = (at >> 3) < nv ? pack_h2(y.x, y.y) : 0u;
          }
          *reinterpret_cast<uint4 *>(out + (i >> 2) * kSlab + 16 * at) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncthreads();  // A and P take the keys' place
      }

      // A and P, 16 columns at a time.  In the row's own 16-token block the decays
      // are taken element by element; in blocks before it they go by way of the
      // block's last token, e^(g_i - g_j) = e^(g_i - g_end) e^(g_end - g_j), no factor
      // above 1.
      uint8_t *P = s.rest;  // (16-byte aligned; the copy to a swizzled place keeps the chunk order)
      const bool part = nv < kC;
      auto put = [&](int J, const f2(&x)[8]) {
        f2 z[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) z[q] = part && !on ? mk2(0.f, 0.f) : x[q];  // (may hold anything)
        if (isk) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4 *>(&s.Am[tok][16 * J + 4 * q]) =
                make_float4(z[2 * q].x, z[2 * q].y, z[2 * q + 1].x, z[2 * q + 1].y);
        } else {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            *reinterpret_cast<uint4 *>(P + sw128(tok, 2 * J + q)) =
                make_uint4(pack_h2(z[4 * q].x, z[4 * q].y), pack_h2(z[4 * q + 1].x, z[4 * q + 1].y),
                           pack_h2(z[4 * q + 2].x, z[4 * q + 2].y), pack_h2(z[4 * q + 3].x, z[4 * q + 3].y));
        }
      };
      auto before = [&](int J, const uint32_t(&r)[16], f2(&x)[8]) {  // a block before the row's own
        const f2 ge = sg[16 * J + 15];
        const float fr = rowf * ex2((gi.x - ge.x) + (gi.y - ge.y));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 h = *reinterpret_cast<const float4 *>(&s.h[16 * J + 4 * q]);
          x[2 * q] = mul2(mul2(mk2(h.x, h.y), mk2(fr, fr)),
                          mk2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])));
          x[2 * q + 1] = mul2(mul2(mk2(h.z, h.w), mk2(fr, fr)),
                              mk2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])));
        }
      };
      {
        f2 x[8];
        float o[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int j = (tok & ~15) + q;
          const f2 gj = sg[j];
          const f2 d = add2(gi, mk2(-gj.x, -gj.y));
          const bool in = isk ? j < tok : j <= tok;
          o[q] = in ? __uint_as_float(own[q]) * (rowf * s.f[j] * ex2(d.x + d.y)) : 0.f;
        }
        before(2 * blk, r0, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = up ? x[q] : mk2(o[2 * q], o[2 * q + 1]);
        put(2 * blk, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = up ? mk2(o[2 * q], o[2 * q + 1]) : mk2(0.f, 0.f);
        put(2 * blk + 1, x);
      }
#pragma unroll 1
      for (int J = 0; J < 2; ++J) {
        f2 x[8];
        if (blk) {
          tmem_ld16(grow + 16 * J, r0);
          tmem_ld_wait();
          before(J, r0, x);
          put(J, x);
        } else if (!isk) {  // above P's diagonal blocks
#pragma unroll
          for (int q = 0; q < 8; ++q) x[q] = mk2(0.f, 0.f);
          put(2 + J, x);
        }
      }
      tc_fence_before();
      // the chunk's decay multiplies the state once a chunk: exact (while the other
      // warps invert)
      double gtot = 0.;
      const float con0 = con;
      if (pw == 3) {
        gtot = exp2((double)g63x * 0x1p-44);
        if (hj + 1 < tp.share) gates(hd + 1, gb ^ 1);
      }
      if (isk) {
        // the inverses of this warp's two diagonal blocks, a column a lane
        __syncwarp();
        const int o = 32 * pw + (lane & 16), col = lane & 15;
        f2 x[8];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f2 a0 = mk2(col == i ? 1.f : 0.f, 0.f), a1 = mk2(0.f, 0.f);
#pragma unroll
          for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
            const float4 a = *reinterpret_cast<const float4 *>(&s.Am[o + i][o + 4 * j4]);
            // (columns from i on hold zeros; x not yet set is not read)
            if (4 * j4 + 1 < i) a0 = fma2(mk2(-a.x, -a.y), x[2 * j4], a0);
            else a0.x = fmaf(-a.x, x[2 * j4].x, a0.x);
            if (4 * j4 + 3 < i) a1 = fma2(mk2(-a.z, -a.w), x[2 * j4 + 1], a1);
            else if (4 * j4 + 2 < i) a1.x = fmaf(-a.z, x[2 * j4 + 1].x, a1.x);
          }
          a0 = add2(a0, a1);
          const float xi = a0.x + a0.y;
          if (i & 1) x[i / 2].y = xi; else x[i / 2].x = xi;
        }
        __syncwarp();  // every lane has read the blocks
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s.Am[o + 2 * i][o + col] = x[i].x;
          s.Am[o + 2 * i + 1][o + col] = x[i].y;
        }
      }
      __syncthreads();
      {  // below the diagonal blocks of 16: half pw & 1 of the columns of pair pw / 2
        const int o = 32 * (pw >> 1), n = 8 * (pw & 1);
        float *scratch = &s.Am[16 * (pw >> 1)][32 + n];  // (of the block above the diagonal)
        float c1[1][4], c2[1][4];
        small_product<1, 2, false>(&s.Am[o + 16][o], &s.Am[o][o + n], pw & 1, c1);
        put_product<1>(scratch, c1, 1.f);
        __syncwarp();
        small_product<1, 2, true>(&s.Am[o + 16][o + 16], scratch, 0, c2);
        __syncthreads();  // A21 has been read
        put_product<1>(&s.Am[o + 16][o + n], c2, -1.f);
      }
      __syncthreads();
      {  // and of 32: eight columns a warp
        float *scratch = &s.Am[0][32 + 8 * pw];
        float c1[2][4], c2[2][4];
        small_product<2, 4, false>(&s.Am[32][0], &s.Am[0][8 * pw], pw, c1);
        put_product<2>(scratch, c1, 1.f);
        __syncwarp();
        small_product<2, 4, true>(&s.Am[32][32], scratch, 0, c2);
        __syncthreads();
        put_product<2>(&s.Am[32][8 * pw], c2, -1.f);
      }
      __syncthreads();
      // T diag(b) to float16 pairs: row pt % 64, half pt / 64 (of the first rows
      // the second half is zero)
      const int hf = pw >> 1;
      const bool have = pw != 2;
      f2 t[16];
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (have) a = *reinterpret_cast<const float4 *>(&s.Am[tok][32 * hf + 4 * q]);
        const float4 b = *reinterpret_cast<const float4 *>(&s.bv[32 * hf + 4 * q]);
        t[2 * q] = mul2(mk2(a.x, a.y), mk2(b.x, b.y));
        t[2 * q + 1] = mul2(mk2(a.z, a.w), mk2(b.z, b.w));
        sum += (fabsf(t[2 * q].x) + fabsf(t[2 * q].y)) + (fabsf(t[2 * q + 1].x) + fabsf(t[2 * q + 1].y));
      }
      sum = warp_max(sum);
      if (lane == 0) s.tn[pw] = sum;
      __syncthreads();  // T takes A's place
      // (a bound of the rows' sums: the largest of each half)
      const float tn = fmaxf(s.tn[0], s.tn[1]) + fmaxf(s.tn[2], s.tn[3]);
      // T goes as it is where its digits and range are float16's (the second kernel
      // need not take a scale back), by a power of two where it is larger or, as
      // strengths below 1/16 make it, smaller
      int eT = scale_exp(tn);
      eT = eT < 0 || tn < 0.0625f ? eT : 0;
      const f2 sc = mk2(pow2i(eT), pow2i(eT));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 hi = make_uint4(0u, 0u, 0u, 0u), lo = hi;
        if (have) {
          split_h2(mul2(t[4 * q], sc), hi.x, lo.x);
          split_h2(mul2(t[4 * q + 1], sc), hi.y, lo.y);
          split_h2(mul2(t[4 * q + 2], sc), hi.z, lo.z);
          split_h2(mul2(t[4 * q + 3], sc), hi.w, lo.w);
        }
        *reinterpret_cast<uint4 *>(s.T + sw128(tok, 4 * hf + q)) = hi;
        *reinterpret_cast<uint4 *>(s.T + kC * 128 + sw128(tok, 4 * hf + q)) = lo;
      }
      if (pw == 3 && lane == 0) {
        fac[4 * kC] = (float)gtot;
        fac[4 * kC + 1] = fmaxf(s.ekn[0], s.ekn[1]);
        fac[4 * kC + 2] = tn * sc.x;
        fac[4 * kC + 3] = (float)eT;
        fac[4 * kC + 4] = con0;
        fac[4 * kC + 5] = ok ? 0.f : 1.f;
      }
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (pt == 0) {
        uint8_t *out = tp.rec + (rs * p.H + hd) * (int64_t)sizeof(Rec);
        bulk_store(out, s.T, kRecT);
        bulk_store(out + kRecT, s.rest, sizeof(Rec) - kRecT);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
  }
  if (pt == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncthreads();
  if (pw == 1) tmem_dealloc(tb, 64);
}

// ------------------------------------------------------------- the chain
// Warps (20):
//   0-7    the chain: two warps per lane quarter, each with half of the columns
//          (tokens of R and U, key dimensions of S): R from KS and V; U' from
//          the product with T; the state from dS.
//   8-11   queries to scaled float16, in place, and the chunk's bounds, a chunk
//          ahead.
//   12-15  y from Y, a chunk behind.
//   16     copies of the scaled keys and of Q ([64 x 64] slabs, 128-byte swizzle,
//          three stages).
//   17     MMA issuer.
//   18     copies of the records (three stages).
//   19     copies of V ([64 x 128], two stages).
constexpr int kThreads = 640;
constexpr int kSorted = 256;  // packed sequences that are put in order
// Registers a thread of the groups; together the launch's 640 x 96.
constexpr int kRegChain = 168, kRegSide = 56, kRegIssue = 32;
static_assert(256 * kRegChain + 256 * kRegSide + 128 * kRegIssue <= kThreads * 96, "register split");

// TMEM columns.  dS lands where S's pieces are (they are rewritten from it),
// the product with T where KS was, U's hi parts where R's pieces were.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColKS = 128, kColR = 192, kColU2 = 256, kColY = 320;  // Y: two

template <int KD> struct __align__(1024) GdrSmem {
  uint8_t kq[3][KD / 64][128 * 128];  // [stage][slab]: rows 0-63 keys, 64-127 queries
  __nv_bfloat16 v[2][kC][kV];
  struct __align__(1024) { Rec r; } rec[3];
  __align__(128) __nv_bfloat16 y[4][2][kC / 2][32];  // two halves of a chunk's y, a warp's 32 columns
  // maxima, by lane quarter (and half); of a chunk's y, the scale, and a warp's
  // factors with it
  float smax[4][2], ysc[3][4], yfac[4][kC];
  float4 bound[3][4];  // of a chunk, by lane quarter: see the chain
  uint64_t fullk[3], conv[3], empty[3], fullr[3], rfree[3], yfree[2], fullv[2], vfree[2], sready[2];
  uint64_t ksdone, rready, udone, uready, supdone, pudone;
  uint32_t taddr;
};
static_assert(sizeof(GdrSmem<128>) + 1024 + 4 * (kSorted + 4) <= 232448, "GdrSmem exceeds the shared memory of a CTA");

// A warp's wait (bounded).  After one that ran out the warp goes on without
// waiting, so that barriers stay matched.
struct Waiter {
  int *status;
  bool dead;
  __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity, int code) {
    if (dead) return;
    if (__any_sync(0xffffffffu, !mbar_wait(bar, parity, kWaitLimit))) expired(code);
  }
  __device__ __forceinline__ void expired(int code) {
    dead = true;
    if (status && (threadIdx.x & 31) == 0) atomicExch(status, code);
  }
};

template <int KD, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    gdr_tc_kernel(const __grid_constant__ CUtensorMap mQ,
                  const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mY,
                  const GdrTcParams tp) {
  constexpr int NP = KD / 64;        // slabs
  constexpr int KH = KD / 2;         // key dimensions of a chain warp's half
  constexpr int KS16 = KD / 16;      // K steps over the key dimension
  using Smem = GdrSmem<KD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem &s = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const GdrParams &p = tp.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the CTA's sequence, head, segment and value columns
  const int64_t per = PASS == 0 ? tp.vtiles
                      : PASS == 1 ? tp.vtiles + (tp.nseg - 2) * (tp.vtiles + 1)
                                     : (tp.nseg - 1) * tp.vtiles;
  const int64_t unit = blockIdx.x / per;
  int64_t vt = blockIdx.x % per;
  int seg = 0;
  bool map = false;  // the segment's map: from the identity, without values
  if (PASS == 2) {
    seg = 1 + (int)(vt / tp.vtiles);
    vt %= tp.vtiles;
  } else if (PASS == 1 && vt >= tp.vtiles) {
    vt -= tp.vtiles;
    seg = 1 + (int)(vt / (tp.vtiles + 1));
    vt %= tp.vtiles + 1;
    map = vt == tp.vtiles;
    if (map) vt = 0;
  }
  const bool outs = PASS != 1 || seg == 0;  // y is wanted
  const int64_t hd = unit % p.H;
  int64_t seq = unit / p.H;
  // Packed sequences start in the order of their lengths, the longest first: CTAs
  // are taken up in order, and one that starts late and runs long keeps the
  // others' SMs waiting (24 sequences of 1 to 2601 tokens, 16 heads: 248 -> 194 us).
  if (PASS == 0 && p.cu && p.nseq > 1 && p.nseq <= kSorted) {
    __shared__ int lens[kSorted], pick;
    const int n = (int)p.nseq;
    if (tid < n) lens[tid] = p.cu[tid + 1] - p.cu[tid];
    __syncthreads();
    if (tid < n) {
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += lens[i] > lens[tid] || (lens[i] == lens[tid] && i < tid);
      if (rank == (int)seq) pick = tid;
    }
    __syncthreads();
    seq = pick;
  }
  int64_t slot, t0, len;
  if (!gdr_sequence(p, seq, slot, t0, len)) {
    pdl_wait();  // (no CTA ends before the kernels ahead have)
    return;
  }
  const int64_t g = hd / (p.H / p.Hk);
  int64_t c0 = 0;  // the segment's first chunk
  if (PASS) {
    const int64_t all = (len + kC - 1) / kC, c1 = all * (seg + 1) / tp.nseg;
    c0 = all * seg / tp.nseg;
    t0 += c0 * kC;
    len = (c1 * kC < len ? c1 * kC : len) - c0 * kC;
  }
  const int nch = (int)((len + kC - 1) / kC);
  // the records of the first chunk here and, one behind the other, of the rest
  const int64_t slot0 = record_slot(tp, seq, t0, c0), slot1 = record_slot(tp, seq, t0 + kC, c0 + 1);
  const int64_t v0 = vt * kV;
  const int64_t cols = map ? p.K : p.V;
  // where the state comes from and goes to: its first value column here
  const int64_t per_seg = p.nseq * p.H * p.K;
  const float *src = p.h0 ? p.h0 + (slot * p.H + hd) * p.K * p.V + v0 : nullptr;
  float *dst = p.h_last ? p.h_last + (slot * p.H + hd) * p.K * p.V + v0 : nullptr;
  if (PASS == 1) {
    if (seg > 0) src = nullptr;
    dst = map ? tp.seg_map + ((seg - 1) * per_seg + unit * p.K) * p.K
              : tp.seg_state + (seg * per_seg + unit * p.K) * p.V + v0;
  } else if (PASS == 2) {
    src = tp.seg_state + ((seg - 1) * per_seg + unit * p.K) * p.V + v0;
    if (seg < tp.nseg - 1) dst = nullptr;
  }

  // Chain and output warps: value column cv of the tile; chain: half ch.
  const int quarter = warp & 3, ch = warp >> 2;
  const int cv = 32 * quarter + lane;
  const bool live = v0 + cv < cols;
  const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
  const float kNorm = KD == 128 ? 11.32f : 8.f;  // sqrt(KD): |S^T k| <= |k| sqrt(KD) max |S|
  auto start = [&](int r) {  // the state's row r of this lane's column
    if (!live || r >= p.K) return 0.f;
    return map ? (r == cv ? 1.f : 0.f) : src ? src[(int64_t)r * p.V + cv] : 0.f;
  };

  if (nch == 0) {  // an empty sequence or segment hands its state on
    pdl_wait();
    if (warp < 8 && dst && live) {
      for (int r = ch; r < p.K; r += 2) dst[(int64_t)r * cols + cv] = start(r);
    }
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s.fullk[i], 1);
      mbar_init(&s.conv[i], 4);
      mbar_init(&s.empty[i], 1);
      mbar_init(&s.fullr[i], 1);
      mbar_init(&s.rfree[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.yfree[i], 4);
      mbar_init(&s.fullv[i], 1);
      mbar_init(&s.vfree[i], 8);
      mbar_init(&s.sready[i], 4);
    }
    mbar_init(&s.ksdone, 1);
    mbar_init(&s.rready, 8);
    mbar_init(&s.udone, 1);
    mbar_init(&s.uready, 8);
    mbar_init(&s.supdone, 1);
    mbar_init(&s.pudone, 1);
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&s.taddr, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.taddr;
  Waiter wait{tp.status, false};

  if (warp >= 16) {
    reg_dealloc<kRegIssue>();
    if (warp == 16 && lane == 0) {
      // ---------------------------------------------------------- keys and queries
      tma_prefetch_desc(&mQ);
      const int64_t step = p.Hk * (int64_t)(NP * kSlab);
      const uint8_t *keys = tp.keys + slot0 * step + g * (int64_t)(NP * kSlab);
      pdl_wait();  // the first kernel's work
      int c = 0;
      for (; c < nch; ++c) {
        const int k3 = c % 3, t = (int)(t0 + (int64_t)c * kC);
        if (c >= 3 && !mbar_wait(&s.empty[k3], (c / 3 - 1) & 1, kWaitLimit)) break;
        mbar_expect_tx(&s.fullk[k3], NP * 128 * 128);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          bulk_load(s.kq[k3][n], keys + n * kSlab, kSlab, &s.fullk[k3]);
          tma_load_3d(s.kq[k3][n] + kC * 128, &mQ, &s.fullk[k3], 64 * n, (int)g, t);
        }
        keys += c ? step : (slot1 - slot0) * step;
      }
      if (c < nch && tp.status) atomicExch(tp.status, 2);
      // Leave no copy in flight: the last chunks issued have landed.
      for (int i = c > 3 ? c - 3 : 0; i < c; ++i) mbar_wait(&s.fullk[i % 3], (i / 3) & 1, kWaitLimit);
    } else if (warp == 18 && lane == 0) {
      // ---------------------------------------------------------- records
      const int64_t step = p.H * (int64_t)sizeof(Rec);
      const uint8_t *rec = tp.rec + slot0 * step + hd * (int64_t)sizeof(Rec);
      pdl_wait();  // the first kernel's work
      int c = 0;
      for (; c < nch; ++c) {
        const int r3 = c % 3;
        if (c >= 3 && !mbar_wait(&s.rfree[r3], (c / 3 - 1) & 1, kWaitLimit)) break;
        mbar_expect_tx(&s.fullr[r3], (uint32_t)sizeof(Rec));
        bulk_load(&s.rec[r3].r, rec, sizeof(Rec), &s.fullr[r3]);
        rec += c ? step : (slot1 - slot0) * step;
      }
      if (c < nch && tp.status) atomicExch(tp.status, 2);
      for (int i = c > 3 ? c - 3 : 0; i < c; ++i) mbar_wait(&s.fullr[i % 3], (i / 3) & 1, kWaitLimit);
    } else if (warp == 19 && lane == 0) {
      // ---------------------------------------------------------- values
      tma_prefetch_desc(&mV);
      int c = 0;
      for (; c < nch; ++c) {
        const int r2 = c & 1;
        if (c >= 2 && !mbar_wait(&s.vfree[r2], ((c >> 1) - 1) & 1, kWaitLimit)) break;
        mbar_expect_tx(&s.fullv[r2], kC * kV * 2);
        tma_load_3d(s.v[r2], &mV, &s.fullv[r2], (int)v0, (int)hd, (int)(t0 + (int64_t)c * kC));
      }
      if (c < nch && tp.status) atomicExch(tp.status, 2);
      for (int i = c > 2 ? c - 2 : 0; i < c; ++i) mbar_wait(&s.fullv[i & 1], (i >> 1) & 1, kWaitLimit);
    } else if (warp == 17) {
      // ---------------------------------------------------------- MMA issuer
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
      // K step kk of a K-major operand of two slabs, in descriptor units
      auto koff = [](int kk) { return (uint64_t)(((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4); };
      // TMEM column of K step kk of S's, R's, U's hi pieces: 32 columns hold hi
      // and, 16 further on, lo of 32 values
      auto rcol = [](int kk) { return 32 * (kk >> 1) + 8 * (kk & 1); };
      for (int c = 0; c < nch; ++c) {
        const uint32_t ph = c & 1, ycol = tb + kColY + 64 * ph;
        const uint64_t dk = smem_desc(smem_u32(s.kq[c % 3][0]), 16, 1024, kSwizzle128B);
        const uint64_t dq = dk + ((kC * 128) >> 4);
        const uint64_t dm = smem_desc(smem_u32(s.kq[c % 3][0]), 128 * 128, 1024, kSwizzle128B);
        const uint64_t th = smem_desc(smem_u32(s.rec[c % 3].r.T[0]), 16, 1024, kSwizzle128B);
        const uint64_t tl = smem_desc(smem_u32(s.rec[c % 3].r.T[1]), 16, 1024, kSwizzle128B);
        const uint64_t dp = smem_desc(smem_u32(s.rec[c % 3].r.P), 16, 1024, kSwizzle128B);
        auto ready = [&](int i) {  // keys, queries and record of chunk i
          wait(&s.fullk[i % 3], (i / 3) & 1, 3);
          wait(&s.fullr[i % 3], (i / 3) & 1, 3);
          wait(&s.conv[i % 3], (i / 3) & 1, 3);
        };
        if (c == 0) ready(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // a half of the state at a time
          wait(&s.sready[h], ph, 4);
          if (wait.dead) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int kk = h * (KS16 / 2); kk < (h + 1) * (KS16 / 2); ++kk)
                mma_ts(tb + kColKS, tb + kColS + rcol(kk) + x * 16, dk + koff(kk), id64, h + x + kk > 0);
          }
          __syncwarp();
        }
        if (wait.dead) break;
        commit(&s.ksdone, ph);
        // y of the chunk two before has been read
        if (c > 1) wait(&s.yfree[ph], ((c >> 1) - 1) & 1, 5);
        wait(&s.rready, ph, 7);
        if (wait.dead) break;
        tc_fence_after();
        if (leader) {  // hi hi, lo hi, hi lo
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tb + kColKS, tb + kColR + rcol(kk) + (x == 1 ? 16 : 0),
                     (x == 2 ? tl : th) + 2 * kk, id64, x + kk > 0);
        }
        commit(&s.udone, ph);
        if (leader && outs) {
#pragma unroll
          for (int kk = 0; kk < KS16; ++kk)
            mma_ts(ycol, tb + kColS + rcol(kk), dq + koff(kk), id64, kk > 0);
        }
        __syncwarp();
        if (c + 1 < nch) ready(c + 1);
        wait(&s.uready, ph, 8);
        if (wait.dead) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(tb + kColS, tb + kColU2 + rcol(kk) + 16 * x, dm + kk * 128, idS, x + kk > 0);
          mma_commit(&s.supdone);
          mma_commit(&s.empty[c % 3]);
          if (outs) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(ycol, tb + kColR + rcol(kk), dp + 2 * kk, id64, 1);
          }
        }
        commit(&s.pudone, ph);
      }
      // Leave no MMA in flight before TMEM is freed.
      if (lane == 0 && last_bar) mbar_wait(last_bar, last_par, kWaitLimit);
      __syncwarp();
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ y
    reg_dealloc<kRegSide>();
    __nv_bfloat16 *yb = static_cast<__nv_bfloat16 *>(p.y) + (t0 * p.H + hd) * p.V + v0 + cv;
    const int64_t yrow = p.H * p.V;
    for (int c = 0; c < nch; ++c) {
      const int par = c & 1;
      const int64_t left = len - (int64_t)c * kC;
      const int nv = (int)(left < kC ? left : kC);
      const Rec &rc = s.rec[c % 3].r;
      wait(&s.fullr[c % 3], (c / 3) & 1, 9);
      wait(&s.pudone, par, 10);
      tc_fence_after();
      // this warp's factors of the tokens
      float *yf = s.yfac[quarter];
#pragma unroll
      for (int e = 0; e < 2; ++e) yf[lane + 32 * e] = rc.cq[lane + 32 * e] * s.ysc[c % 3][quarter];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.rfree[c % 3]);
      if (!outs) {
        if (lane == 0) mbar_arrive(&s.yfree[par]);
        continue;
      }
      // a whole chunk leaves by TMA (columns behind V are not written), the
      // last one's rows one by one
      const bool whole = nv == kC;
      __nv_bfloat16 *yp = yb + (int64_t)c * kC * yrow;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        uint32_t r[16], out[8];
        tmem_ld16(tb + lane_base + kColY + 64 * par + 16 * i, r);
        if (whole && !(i & 1)) {  // the half two before has left
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
        }
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 f = *reinterpret_cast<const float4 *>(&yf[16 * i + 4 * q]);
          const f2 o0 = mul2(mk2(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1])), mk2(f.x, f.y));
          const f2 o1 = mul2(mk2(__uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3])), mk2(f.z, f.w));
          out[2 * q] = pack_bf16x2(o0.x, o0.y);
          out[2 * q + 1] = pack_bf16x2(o1.x, o1.y);
        }
        if (whole) {
          uint16_t *sy = reinterpret_cast<uint16_t *>(&s.y[quarter][i >> 1][16 * (i & 1)][lane]);
#pragma unroll
          for (int j = 0; j < 16; ++j) sy[32 * j] = (uint16_t)(out[j / 2] >> (16 * (j & 1)));
          if (i & 1) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0 && v0 + 32 * quarter < p.V) {
              tma_store_3d(&mY, s.y[quarter][i >> 1], (int)v0 + 32 * quarter, (int)hd,
                           (int)(t0 + (int64_t)c * kC + 16 * (i - 1)));
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        } else if (live) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (16 * i + j < nv) *reinterpret_cast<uint16_t *>(yp) = (uint16_t)(out[j / 2] >> (16 * (j & 1)));
            yp += yrow;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.yfree[par]);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ conversion
    reg_dealloc<kRegSide>();
    const int tok = (tid - 256) >> 1, hf = tid & 1;  // two threads a query
    for (int c = 0; c < nch; ++c) {
      const int64_t left = len - (int64_t)c * kC;
      const Rec &rc = s.rec[c % 3].r;
      wait(&s.fullr[c % 3], (c / 3) & 1, 11);
      const float f = rc.fq[tok];
      wait(&s.fullk[c % 3], (c / 3) & 1, 12);
      const bool on = tok < left;  // rows behind the end may hold anything
#pragma unroll
      for (int i = 0; i < NP * 4; ++i) {
        // (the halves' accesses lie in different banks)
        const int at = NP == 2 ? (i ^ (4 * hf)) : i + 4 * hf;
        uint4 *qp = reinterpret_cast<uint4 *>(&s.kq[c % 3][NP == 2 ? hf : 0][0] + sw128(kC + tok, at));
        const uint4 u = *qp;
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const f2 y = mul2(mk2(bf16lo(w[x]), bf16hi(w[x])), mk2(f, f));
          w[x] = on ? pack_h2(y.x, y.y) : 0u;
        }
        *qp = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_async_smem();
      {  // the largest finite value of this warp's quarter of V
        wait(&s.fullv[c & 1], (c >> 1) & 1, 18);
        const uint4 *vp = reinterpret_cast<const uint4 *>(&s.v[c & 1][lane >> 2][32 * quarter + 8 * (lane & 3)]);
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (8 * i + (lane >> 2) < left) {
            const uint4 u = vp[i * (8 * kV / 8)];
            m = maxabs_bf2(maxabs_bf2(m, u.x), maxabs_bf2(u.y, maxabs_bf2(u.z, u.w)));
          }
        }
        float mx = fmaxf(fabsf(bf16lo(m)), fabsf(bf16hi(m)));
        if (mx >= __uint_as_float(0x7f800000u)) {  // an infinity among them: look again
          mx = 0.f;
          const __nv_bfloat16 *ve = reinterpret_cast<const __nv_bfloat16 *>(vp);
          for (int i = 0; i < 8; ++i)
            for (int e = 0; e < 8; ++e) {
              const float x = fabsf(__bfloat162float(ve[i * 8 * kV + e]));
              if (8 * i + (lane >> 2) < left && x < __uint_as_float(0x7f800000u)) mx = fmaxf(mx, x);
            }
        }
        mx = map ? 0.f : warp_max(mx);
        // From m, the largest value of the state entering the chunk, a bound of the
        // state leaving it, z + w m = n, which is one of its columns' lengths |S|, and
        // from such an n of the chunk before, bounds of this chunk's R and U, x + y n.
        // With keys of length at most 1, write strengths b in 0 .. 2 and no growth,
        // I - b k k^T lengthens nothing: |S| <= e^g sqrt(K) m + 64 b |v| column by
        // column, |R| <= |v| + |S| and |U| <= b (|v| + |S|).  Else step by step:
        // |R| <= |v| + |ek k| |S|, |U| <= (T's row sums) |R|, |dS| <= sum |k| |U'|
        // <= 128 |U|, |S| <= sqrt(K) m before.
        const float b = rc.con;
        if (lane == 0 && rc.expired != 0.f) atomicExch(tp.status, 1);
        float4 f = make_float4(65.f * b * b * mx, b, 65.f * b * b * mx, b * kNorm * rc.gC);
        if (!(b > 0.f)) {
          const float tn = rc.tn * pow2i(-(int)rc.eT), t1 = fmaxf(1.f, tn), en = rc.ekn;
          f = make_float4(t1 * mx, t1 * en, 128.f * tn * mx, kNorm * fmaf(128.f * tn, en, fabsf(rc.gC)));
        }
        if (lane == 0) s.bound[c % 3][quarter] = f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.conv[c % 3]);
    }
  } else {
    // ------------------------------------------------------------ the chain
    reg_alloc<kRegChain>();
    if (PASS == 2) pdl_wait();  // the states entering the segments
    f2 st[KH / 2];  // the half row of this lane, scaled by 2^eS
    float m = 0.f;
    if (src) {  // (loads without branches between them: all in flight together)
      const float *sp = src + (live ? cv : 0);
      float x[KH];
#pragma unroll
      for (int i = 0; i < KH; ++i) {
        const int64_t r = ch * KH + i;
        x[i] = sp[(r < p.K ? r : 0) * p.V];
      }
#pragma unroll
      for (int i = 0; i < KH; ++i) {
        if (!live || ch * KH + i >= p.K) x[i] = 0.f;
        m = fmaxf(m, fabsf(x[i]));
      }
#pragma unroll
      for (int i = 0; i < KH / 2; ++i) st[i] = mk2(x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < KH / 2; ++i) st[i] = mk2(start(ch * KH + 2 * i), start(ch * KH + 2 * i + 1));
      m = map ? 1.f : 0.f;
    }
    m = warp_max(m);
    if (lane == 0) s.smax[quarter][ch] = m;
    pair_sync(quarter);
    float smax = fmaxf(s.smax[quarter][0], s.smax[quarter][1]);
    // One scale 2^e a chunk for S, R and U, from the bounds beside the conversion.
    wait(&s.conv[0], 0, 13);
    int eS = scale_exp(fmaxf(smax, fmaf(s.bound[0][quarter].y, kNorm * smax, s.bound[0][quarter].x)));
    // S's pieces, hi and lo of 32 values within their own dS columns
    const uint32_t mycol = tb + lane_base + kColS + ch * KH;
    {
      const f2 sc = mk2(pow2i(eS), pow2i(eS));
#pragma unroll
      for (int i = 0; i < KH / 32; ++i) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          st[16 * i + j] = mul2(st[16 * i + j], sc);
          split_h2(st[16 * i + j], hi[j], lo[j]);
        }
        tmem_st16(mycol + 32 * i, hi);
        tmem_st16(mycol + 32 * i + 16, lo);
      }
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.sready[ch]);

    // The values of a chunk that is converted (and so has its V and record), two
    // tokens a register.
    uint32_t vv[16];
    auto values = [&](int c) {
      const int64_t left = len - (int64_t)c * kC - 32 * ch;
      const uint16_t *vp = reinterpret_cast<const uint16_t *>(&s.v[c & 1][32 * ch][cv]);
#pragma unroll
      for (int q = 0; q < 16; ++q)
        vv[q] = (uint32_t)vp[2 * q * kV] | ((uint32_t)vp[(2 * q + 1) * kV] << 16);
      if (left < 32 || map) {  // rows behind the end may hold anything
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (map || 2 * q >= left) vv[q] = 0u;
          else if (2 * q + 1 >= left) vv[q] &= 0xffffu;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.vfree[c & 1]);
    };
    values(0);
    for (int c = 0; c < nch; ++c) {
      const uint32_t ph = c & 1;
      const Rec &rc = s.rec[c % 3].r;
      // While KS runs: the factors of R, and the next chunk's scale (U' takes it
      // already, so that dS comes out in it) from a bound of its state.
      const bool more = c + 1 < nch;
      f2 nb[16];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 ek = *reinterpret_cast<const float4 *>(&rc.ek[32 * ch + 4 * q]);
        nb[2 * q] = mk2(ek.x, ek.y);
        nb[2 * q + 1] = mk2(ek.z, ek.w);
      }
      if (more) wait(&s.conv[(c + 1) % 3], ((c + 1) / 3) & 1, 17);
      const float4 bn = s.bound[c % 3][quarter], bx = s.bound[more ? (c + 1) % 3 : c % 3][quarter];
      const float gC = rc.gC;
      const int eT = (int)rc.eT;
      const uint32_t sv = __byte_perm(__float_as_uint(pow2i(eS)), 0, 0x3232);  // 2^eS in bfloat16, twice
      pair_sync(quarter);
      if (c > 0) smax = pow2i(-eS) * fmaxf(s.smax[quarter][0], s.smax[quarter][1]);
      const float bS = fmaf(bn.w, smax, bn.z);
      const int eN = scale_exp(more ? fmaxf(bS, fmaf(bx.y, bS, bx.x)) : bS);
      if (ch == 0 && lane == 0) s.ysc[c % 3][quarter] = pow2i(-eS);
      // R
      wait(&s.ksdone, ph, 14);
      tc_fence_after();
      {
        uint32_t r0[16], r1[16], hi[16], lo[16];
        tmem_ld16(tb + lane_base + kColKS + 32 * ch, r0);
        tmem_ld16(tb + lane_base + kColKS + 32 * ch + 16, r1);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint32_t a = q < 8 ? r0[2 * q] : r1[2 * q - 16], b = q < 8 ? r0[2 * q + 1] : r1[2 * q - 15];
          f2 x = mul2(nb[q], mk2(__uint_as_float(a), __uint_as_float(b)));
          split_h2(fma_bf16x2(vv[q], sv, x), hi[q], lo[q]);
        }
        tmem_st16(tb + lane_base + kColR + 32 * ch, hi);
        tmem_st16(tb + lane_base + kColR + 32 * ch + 16, lo);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.rready);
      {
        const f2 fU = mk2(pow2i(eN - eS - eT), pow2i(eN - eS - eT));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 cu = *reinterpret_cast<const float4 *>(&rc.cu[32 * ch + 4 * q]);
          nb[2 * q] = mul2(mk2(cu.x, cu.y), fU);
          nb[2 * q + 1] = mul2(mk2(cu.z, cu.w), fU);
        }
      }
      const float un = pow2i(-eT);  // 1 but for very large or small T
      // U and U'
      wait(&s.udone, ph, 15);
      tc_fence_after();
      {
        uint32_t r0[16], r1[16], uh[16], hi[16], lo[16];
        tmem_ld16(tb + lane_base + kColKS + 32 * ch, r0);
        tmem_ld16(tb + lane_base + kColKS + 32 * ch + 16, r1);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint32_t a = q < 8 ? r0[2 * q] : r1[2 * q - 16], b = q < 8 ? r0[2 * q + 1] : r1[2 * q - 15];
          const f2 y = mk2(__uint_as_float(a), __uint_as_float(b));
          uh[q] = eT == 0 ? pack_h2(y.x, y.y) : pack_h2(y.x * un, y.y * un);
          split_h2(mul2(y, nb[q]), hi[q], lo[q]);
        }
        tmem_st16(tb + lane_base + kColU2 + 32 * ch, hi);
        tmem_st16(tb + lane_base + kColU2 + 32 * ch + 16, lo);
        tmem_st16(tb + lane_base + kColR + 32 * ch, uh);  // (K step columns as R's hi parts)
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.uready);
      // While dS runs: the next chunk's values.
      if (more) values(c + 1);
      // the state
      wait(&s.supdone, ph, 16);
      tc_fence_after();
      {
        const float gn = gC * pow2i(eN - eS);  // (the difference beyond the range: all or nothing is left)
        const f2 g2 = mk2(gn, gn);
        eS = eN;
        uint32_t mh = 0u;
#pragma unroll
        for (int i = 0; i < KH / 32; ++i) {
          uint32_t r[2][16];
          tmem_ld16(mycol + 32 * i, r[0]);
          tmem_ld16(mycol + 32 * i + 16, r[1]);
          tmem_ld_wait();
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            f2 &w = st[16 * i + j];
            const uint32_t a = r[j >> 3][2 * (j & 7)], b = r[j >> 3][2 * (j & 7) + 1];
            w = fma2(w, g2, mk2(__uint_as_float(a), __uint_as_float(b)));
            split_h2(w, hi[j], lo[j]);
            mh = maxabs_h2(mh, hi[j]);
          }
          tmem_st16(mycol + 32 * i, hi);
          tmem_st16(mycol + 32 * i + 16, lo);
        }
        const uint32_t a = mh & 0x7fffu, b = (mh >> 16) & 0x7fffu;  // float16 order is that of the bits
        mh = a > b ? a : b;
        // (hi may lie half a step, 2^-11, below the value)
        m = mh < 0x7c00u ? 1.001f * __half2float(__ushort_as_half((unsigned short)mh)) : 0.f;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.sready[ch]);
      m = warp_max(m);
      if (lane == 0) s.smax[quarter][ch] = m;
    }
    if (dst && live && !wait.dead) {
      const float un = pow2i(-eS);
#pragma unroll
      for (int i = 0; i < KH; ++i) {
        const int r = ch * KH + i;
        if (r < p.K) dst[(int64_t)r * cols + cv] = un * ((i & 1) ? st[i / 2].y : st[i / 2].x);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc(tb, kTmemCols);
}

// ---------------------------------------------------------------- segments
// The state entering segment i + 1 from the one entering segment i: S <- M S +
// N, N the segment's own state from zeros (in the place of the result), M its
// map.  One CTA per (sequence, head, 16 value columns), over the segments in
// turn, a warp 16 key rows; the products as float32 on mma, each step's summed by
// itself and added with rounding (mma's own sums are cut off, which without decay,
// where most of M is 1 on the diagonal, came to 2e-5 of the state).  A lane takes four
// neighbouring columns of M for the four k of two steps (the sum's order is
// free), so M comes in 16-byte loads, the next segment's under this one's.
constexpr int kCarryCols = 16, kCarryRow = 18;  // (18: no bank conflicts)
__global__ void __launch_bounds__(256) gdr_carry_kernel(const GdrTcParams tp) {
  __shared__ __align__(16) float S[2][128][kCarryRow];
  const GdrParams &p = tp.p;
  const int K = (int)p.K, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int64_t tiles = (p.V + kCarryCols - 1) / kCarryCols;
  const int64_t unit = blockIdx.x / tiles, v0 = (blockIdx.x % tiles) * kCarryCols;
  const int64_t per_seg = p.nseq * p.H * p.K;
  pdl_launch_dependents();
  pdl_wait();
  const int k0 = 16 * warp + r;  // rows k0 and k0 + 8, columns v0 + 2 t (+ 8) and the next
  float *at = tp.seg_state + unit * p.K * p.V + v0;
  const float *m = tp.seg_map + unit * p.K * p.K;
  float4 a[8][2];
  auto fetch = [&]() {
#pragma unroll
    for (int b = 0; b < 8; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = k0 + 8 * e, col = 16 * b + 4 * t;  // (K is a multiple of 8)
        a[b][e] = row < K && col < K ? *reinterpret_cast<const float4 *>(m + (int64_t)row * K + col)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    m += per_seg * p.K;
  };
  float c[2][4];
  auto get = [&](float (&c)[2][4]) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = k0 + 8 * (e >> 1), col = 8 * n + 2 * t + (e & 1);
        c[n][e] = row < K && v0 + col < p.V ? at[(int64_t)row * p.V + col] : 0.f;
      }
  };
  fetch();
  get(c);
  for (int i = 1; i < tp.nseg - 1; ++i) {
    float(*buf)[kCarryRow] = S[i & 1];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float2 *>(&buf[k0 + 8 * e][8 * n + 2 * t]) = make_float2(c[n][2 * e], c[n][2 * e + 1]);
    at += per_seg * p.V;
    float4 w[8][2];
#pragma unroll
    for (int b = 0; b < 8; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) w[b][e] = a[b][e];
    if (i + 1 < tp.nseg - 1) fetch();
    get(c);  // N
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (16 * b >= K) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // k of this step: 16 b + 4 t + 2 h and the next
        uint32_t ah[4], al[4];
        split_tf32(h ? w[b][0].z : w[b][0].x, ah[0], al[0]);
        split_tf32(h ? w[b][1].z : w[b][1].x, ah[1], al[1]);
        split_tf32(h ? w[b][0].w : w[b][0].y, ah[2], al[2]);
        split_tf32(h ? w[b][1].w : w[b][1].y, ah[3], al[3]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t bh[2], bl[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) split_tf32(buf[16 * b + 4 * t + 2 * h + e][8 * n + r], bh[e], bl[e]);
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_tf32(d, al, bh);
          mma_tf32(d, ah, bl);
          mma_tf32(d, ah, bh);
#pragma unroll
          for (int e = 0; e < 4; ++e) c[n][e] += d[e];
        }
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = k0 + 8 * (e >> 1), col = 8 * n + 2 * t + (e & 1);
        if (row < K && v0 + col < p.V) at[(int64_t)row * p.V + col] = c[n][e];
      }
  }
}

// How many segments a sequence is cut into.  Uncut, a call takes its longest
// sequence's chunks one behind the other, 2.75 us each (K = V = 128), on one SM
// per head and 128 value columns.  Cut into n >= 3: a first pass runs segment 0,
// and of segments 1 .. n - 2 the state from zeros and the map of an entering
// state (the same kernel, from the identity and without values); the carry
// joins them; a second pass runs segments 1 .. n - 1 from their states.  That
// is 2 / n of the chunks, about 1.3 us a carry and 20 us of launches, as long
// as each pass finds an SM for every CTA.  Only where no map can grow, and so lose
// the digits of what it leaves as it is: keys of length at most 1, written with
// strengths of a sigmoid (and no decay above 1).
int segments_of(const GdrParams &p) {
  const int64_t vt = (p.V + kV - 1) / kV, base = p.nseq * p.H * vt, sms = device_sm_count();
  const uint32_t bounded = GDR_QK_L2NORM | GDR_BETA_SIGMOID;
  if ((p.flags & bounded) != bounded || base * 3 > sms) return 1;
  const int64_t chunks = p.rows / kC / p.nseq;
  int best = 1;
  double least = 0.9 * 2.75 * (double)chunks;
  for (int n = 3; n <= 16; ++n) {
    const int64_t first = p.nseq * p.H * (vt + (n - 2) * (vt + 1));
    if (first > sms || base * (n - 1) > sms) break;
    const double t = 2.75 * 2. * (double)((chunks + n - 1) / n) + 1.3 * (n - 2) + 20.;
    if (t < least) {
      least = t;
      best = n;
    }
  }
  return best;
}

bool encode(CUtensorMap *m, const void *ptr, int64_t dim, int64_t heads, int64_t rows, int64_t row,
            uint32_t box, CUtensorMapSwizzle sw, uint32_t tokens = kC) {
  const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)dim * 2, (uint64_t)row * 2};
  const uint32_t b[3] = {box, 1, tokens};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, b, sw);
}

// Records of a call: of every chunk (packed: see record_slot).
int64_t slots_of(const GdrParams &p) {
  return p.cu ? p.rows / kC + p.nseq : p.nseq * ((p.L + kC - 1) / kC);
}

// Lets `kernel` use `bytes` of shared memory: an attribute of the current
// device, set once for each (setting it costs a microsecond a call).
template <auto kernel> cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <int KD, int PASS>
cudaError_t launch_pass(const GdrTcParams &q, int64_t blocks, const CUtensorMap &mQ, const CUtensorMap &mV,
                        const CUtensorMap &mY, cudaStream_t s) {
  const size_t smem = sizeof(GdrSmem<KD>) + 1024;
  const cudaError_t e = allow_smem<gdr_tc_kernel<KD, PASS>>(smem);
  if (e != cudaSuccess) return e;
  return launch_dependent(gdr_tc_kernel<KD, PASS>, dim3((unsigned)blocks), dim3(kThreads), smem, s, mQ, mV,
                          mY, q);
}

template <int KD>
cudaError_t launch(const GdrTcParams &q, const CUtensorMap &mK, const CUtensorMap &mQ,
                   const CUtensorMap &mV, const CUtensorMap &mY, cudaStream_t s) {
  const size_t prep = sizeof(PrepSmem<KD>) + 1024;
  cudaError_t e = allow_smem<gdr_prep_kernel<KD>>(prep);
  if (e != cudaSuccess) return e;
  const int64_t most = 6ll * device_sm_count();
  gdr_prep_kernel<KD><<<(unsigned)(q.units < most ? q.units : most), kPrepThreads, prep, s>>>(mK, mQ, q);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t units = q.p.nseq * q.p.H;
  if (q.nseg == 1) return launch_pass<KD, 0>(q, units * q.vtiles, mQ, mV, mY, s);
  e = launch_pass<KD, 1>(q, units * (q.vtiles + (q.nseg - 2) * (q.vtiles + 1)), mQ, mV, mY, s);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (q.p.V + kCarryCols - 1) / kCarryCols;
  e = launch_dependent(gdr_carry_kernel, dim3((unsigned)(units * tiles)), dim3(256), 0, s, q);
  if (e != cudaSuccess) return e;
  return launch_pass<KD, 2>(q, units * (q.nseg - 1) * q.vtiles, mQ, mV, mY, s);
}

// Whether the token-by-token kernel is the faster one: sequences so short that a
// chunk is mostly padding, and few enough heads.  Measured (K = 128): that one
// takes 5.5 us and 0.24 us a token for up to 124 CTAs of 32 value columns (L =
// 16: 8.9 us, L = 64: 20.5), this one 4 us and 13 us for every 148 CTAs of 128
// (17 us up to L = 64 with 4 heads, 31 us with 256).  Packed sequences may be as
// long as all rows.
bool few_tokens(const GdrParams &p) {
  const int64_t longest = p.cu ? p.rows : p.L, sms = device_sm_count();
  if (longest > kC) return false;
  const double ctas = (double)(p.nseq * p.H * ((p.V + 31) / 32));
  const int64_t waves = (p.nseq * p.H * ((p.V + kV - 1) / kV) + sms - 1) / sms;
  return (5.5 + 0.24 * (double)longest) * (ctas > 124. ? ctas / 124. : 1.) < 4. + 13. * (double)waves;
}

}  // namespace

bool gdr_tc_supported(const GdrParams &p) {
  // bf16; whole 16-byte steps for the TMA; 32-bit TMA coordinates
  return p.io == 1 && p.rows > 0 && p.nseq > 0 && !few_tokens(p) && p.K <= 128 && p.K % 8 == 0 && p.V % 8 == 0 &&
         p.q_row % 8 == 0 && p.k_row % 8 == 0 && p.v_row % 8 == 0 && p.rows + kC < (1ll << 31) &&
         p.nseq * p.H * ((p.V + kV - 1) / kV) < (1ll << 31) && slots_of(p) * p.H < (1ll << 31);
}

size_t gdr_tc_workspace(const GdrParams &p) {
  const size_t nseg = (size_t)segments_of(p);
  const size_t states = nseg == 1 ? 0 : ((nseg - 1) * p.V + (nseg - 2) * p.K) * (size_t)(p.nseq * p.H * p.K);
  return kGdrStatusBytes + (size_t)(slots_of(p) * p.H) * sizeof(Rec) +
         (size_t)(slots_of(p) * p.Hk) * (p.K <= 64 ? 1 : 2) * kSlab + states * sizeof(float);
}

cudaError_t launch_gdr_tc(const GdrParams &p, void *workspace, cudaStream_t s) {
  GdrTcParams q;
  q.p = p;
  q.vtiles = (p.V + kV - 1) / kV;
  // (shared keys: once for all their value heads where there are chunks enough to
  // fill the SMs that way, twice over: 8 x 2048 tokens of 32 heads on 16 key heads
  // 117 us, head by head 123)
  q.share = p.H > p.Hk && slots_of(p) * p.Hk >= 12ll * device_sm_count() ? p.H / p.Hk : 1;
  q.units = slots_of(p) * p.H / q.share;
  q.chunks = p.cu ? 0 : (p.L + kC - 1) / kC;
  q.rec = static_cast<uint8_t *>(workspace) + kGdrStatusBytes;
  q.keys = q.rec + (size_t)(slots_of(p) * p.H) * sizeof(Rec);
  q.status = static_cast<int *>(workspace);
  q.nseg = segments_of(p);
  q.seg_state = reinterpret_cast<float *>(q.keys + (size_t)(slots_of(p) * p.Hk) * (p.K <= 64 ? 1 : 2) * kSlab);
  q.seg_map = q.seg_state + (size_t)(q.nseg - 1) * p.nseq * p.H * p.K * p.V;
  CUtensorMap mK, mQ, mV, mY;
  if (!encode(&mK, p.k, p.K, p.Hk, p.rows, p.k_row, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&mQ, p.q, p.K, p.Hk, p.rows, p.q_row, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&mV, p.v, p.V, p.H, p.rows, p.v_row, kV, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode(&mY, p.y, p.V, p.H, p.rows, p.H * p.V, 32, CU_TENSOR_MAP_SWIZZLE_NONE, kC / 2))
    return cudaErrorInvalidValue;
  return p.K <= 64 ? launch<64>(q, mK, mQ, mV, mY, s) : launch<128>(q, mK, mQ, mV, mY, s);
}

}  // namespace ssm
