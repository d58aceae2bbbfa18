// gdr_api.cu -- the exported C ABI of the gated delta rule's operators
// (include/ssm.h): argument validation on the host, then dispatch.  Nothing
// is launched when a check fails, and nothing here allocates memory.
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "ssm.h"

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <typename... Ps>
bool all_aligned(uintptr_t to, Ps... ps) {
  const void *arr[] = {static_cast<const void *>(ps)...};
  for (const void *p : arr)
    if (!aligned(p, to)) return false;
  return true;
}

bool overlap(const void *p, size_t np, const void *q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && np && nq && a < b + nq && b < a + np;
}

ssm_status_t from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return SSM_OK;
  if (e == cudaErrorNotSupported) return SSM_ERR_UNSUPPORTED;
  return SSM_ERR_CUDA;
}

// Sizes below kMaxSize, and tensors of at most kMaxValues values (far beyond
// a GPU's memory), keep every product the checks and kernels form in 64 bits.
constexpr int64_t kMaxSize = 1ll << 31;
constexpr double kMaxValues = 1e15;

// What the prompt scan and the step share: sizes, flags and dtype.
template <typename Args>
ssm_status_t check_heads(const Args *a) {
  if (a->io != SSM_F32 && a->io != SSM_BF16) return SSM_ERR_DTYPE;
  if (a->batch < 0 || a->heads <= 0 || a->key_heads <= 0 || a->heads % a->key_heads ||
      a->key_dim <= 0 || a->value_dim <= 0 || a->state_rows < 0)
    return SSM_ERR_SHAPE;
  if (a->flags & ~(SSM_DT_SOFTPLUS | GDR_BETA_SIGMOID | GDR_QK_L2NORM)) return SSM_ERR_UNSUPPORTED;
  if (!(fabsf(a->scale) <= 3.0e38f)) return SSM_ERR_SHAPE;
  if ((a->flags & GDR_QK_L2NORM) && !(a->l2_eps >= 0.f && a->l2_eps <= 3.0e38f)) return SSM_ERR_SHAPE;
  if (a->key_dim > ssm::kGdrMaxKeyDim || a->value_dim > 65536 || a->heads > 65535 ||
      a->batch >= kMaxSize || a->state_rows >= kMaxSize ||
      (double)a->state_rows * a->heads * a->key_dim * a->value_dim > kMaxValues)
    return SSM_ERR_UNSUPPORTED;
  // a row stride is 0 (dense) or at least the row itself
  const int64_t kr = a->key_heads * a->key_dim, vr = a->heads * a->value_dim;
  if ((a->q_row && a->q_row < kr) || (a->k_row && a->k_row < kr) || (a->v_row && a->v_row < vr) ||
      (a->dt_row && a->dt_row < a->heads) || (a->beta_row && a->beta_row < a->heads))
    return SSM_ERR_SHAPE;
  if (a->q_row >= kMaxSize || a->k_row >= kMaxSize || a->v_row >= kMaxSize ||
      a->dt_row >= kMaxSize || a->beta_row >= kMaxSize)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Bytes of `rows` rows of `width` values, `row` (0 = dense) apart.
size_t rows_bytes(int32_t io, int64_t rows, int64_t row, int64_t width) {
  const size_t es = io == SSM_BF16 ? 2 : 4;
  return rows > 0 ? (size_t)((rows - 1) * (row ? row : width) + width) * es : (size_t)0;
}

// Whether `out` overlaps an input of a scan or step of `rows` rows and
// `sequences` sequences, its states aside.
template <typename Args>
bool overlaps_inputs(const Args *a, int64_t rows, int64_t sequences, const void *out, size_t bytes) {
  const int64_t kr = a->key_heads * a->key_dim, vr = a->heads * a->value_dim;
  const size_t hb = a->dt ? (size_t)a->heads * sizeof(float) : 0;  // (not read without steps)
  return overlap(out, bytes, a->q, rows_bytes(a->io, rows, a->q_row, kr)) ||
         overlap(out, bytes, a->k, rows_bytes(a->io, rows, a->k_row, kr)) ||
         overlap(out, bytes, a->v, rows_bytes(a->io, rows, a->v_row, vr)) ||
         overlap(out, bytes, a->dt, rows_bytes(a->io, rows, a->dt_row, a->heads)) ||
         overlap(out, bytes, a->beta, rows_bytes(a->io, rows, a->beta_row, a->heads)) ||
         overlap(out, bytes, a->A, hb) || overlap(out, bytes, a->dt_bias, hb) ||
         overlap(out, bytes, a->slots, (size_t)sequences * sizeof(int32_t));
}

template <typename Args>
size_t state_bytes(const Args *a) {
  return (size_t)(a->state_rows * a->heads) * (size_t)(a->key_dim * a->value_dim) * sizeof(float);
}

// Whether `out`, an output of a prompt scan, overlaps an input, h0 among them.
bool overlaps_scan(const gdr_scan_args_t *a, const void *out, size_t bytes) {
  return overlaps_inputs(a, a->batch * a->seqlen, a->sequences, out, bytes) ||
         overlap(out, bytes, a->cu_seqlens, (size_t)(a->sequences + 1) * sizeof(int32_t)) ||
         (out != a->h0 && overlap(out, bytes, a->h0, state_bytes(a)));
}

template <typename Args>
void fill_heads(ssm::GdrParams &p, const Args *a) {
  p.H = a->heads;
  p.Hk = a->key_heads;
  p.K = a->key_dim;
  p.V = a->value_dim;
  p.state_rows = a->state_rows;
  p.q_row = a->q_row ? a->q_row : a->key_heads * a->key_dim;
  p.k_row = a->k_row ? a->k_row : a->key_heads * a->key_dim;
  p.v_row = a->v_row ? a->v_row : a->heads * a->value_dim;
  p.dt_row = a->dt_row ? a->dt_row : a->heads;
  p.beta_row = a->beta_row ? a->beta_row : a->heads;
  p.flags = a->flags;
  p.io = a->io;
  p.scale = a->scale;
  p.l2_eps = a->l2_eps;
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.dt = a->dt;
  p.beta = a->beta;
  p.A = a->A;
  p.dt_bias = a->dt_bias;
  p.slots = a->slots;
  p.y = a->y;
}

ssm::GdrParams scan_params(const gdr_scan_args_t *a) {
  ssm::GdrParams p;
  fill_heads(p, a);
  p.nseq = a->sequences;
  p.L = a->seqlen;
  p.rows = a->batch * a->seqlen;
  p.h0 = a->h0;
  p.h_last = a->h_last;
  p.cu = a->cu_seqlens;
  return p;
}

ssm_status_t check_gdr(const gdr_scan_args_t *a, bool shapes_only) {
  if (!a) return SSM_ERR_NULL;
  ssm_status_t st = check_heads(a);
  if (st != SSM_OK) return st;
  if (a->seqlen < 0 || a->sequences < 0) return SSM_ERR_SHAPE;
  if (a->seqlen >= kMaxSize || a->sequences >= kMaxSize ||
      (a->batch > 0 && a->seqlen > 0 && a->batch >= kMaxSize / a->seqlen) ||
      (double)a->batch * a->seqlen * a->heads * a->value_dim > kMaxValues)
    return SSM_ERR_UNSUPPORTED;
  if (shapes_only) return SSM_OK;
  if (a->cu_seqlens ? a->batch != 1 : a->sequences != a->batch) return SSM_ERR_SHAPE;
  if (!a->slots && (a->h0 || a->h_last) && a->state_rows < a->sequences) return SSM_ERR_SHAPE;
  const int64_t rows = a->batch * a->seqlen;
  if (a->sequences > 0 && rows > 0 && (!a->q || !a->k || !a->v || !a->beta || !a->y)) return SSM_ERR_NULL;
  // (read for every head, tokens or not)
  if (a->sequences > 0 && a->dt && !a->A) return SSM_ERR_NULL;
  if (!all_aligned(16, a->q, a->k, a->v, a->A, a->dt_bias, a->h0, a->y, a->h_last, a->workspace) ||
      !all_aligned(a->io == SSM_BF16 ? 2 : 4, a->dt, a->beta) ||
      !all_aligned(4, a->cu_seqlens, a->slots))
    return SSM_ERR_ALIGN;
  // (h_last may be h0; y may not)
  const size_t yb = rows_bytes(a->io, rows, 0, a->heads * a->value_dim), sb = state_bytes(a);
  if (overlaps_scan(a, a->y, yb) || overlap(a->y, yb, a->h0, sb) || overlap(a->y, yb, a->h_last, sb) ||
      overlaps_scan(a, a->h_last, sb))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

}  // namespace

extern "C" {

ssm_status_t gdr_chunk_scan_workspace(const gdr_scan_args_t *a, size_t *bytes) {
  if (!bytes) return SSM_ERR_NULL;
  ssm_status_t st = check_gdr(a, true);
  if (st != SSM_OK) return st;
  const ssm::GdrParams p = scan_params(a);
  *bytes = ssm::gdr_tc_supported(p) ? ssm::gdr_tc_workspace(p) : 0;
  return SSM_OK;
}

ssm_status_t gdr_chunk_scan_fwd(const gdr_scan_args_t *a, void *stream) {
  ssm_status_t st = check_gdr(a, false);
  if (st != SSM_OK) return st;
  if (a->sequences == 0) return SSM_OK;  // nothing to do, nothing launched
  const ssm::GdrParams p = scan_params(a);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!ssm::gdr_tc_supported(p)) return from_cuda(ssm::launch_gdr_recurrent(p, cs));
  const size_t wb = ssm::gdr_tc_workspace(p);
  if (!a->workspace || a->workspace_bytes < wb) return SSM_ERR_WORKSPACE;
  if (overlaps_scan(a, a->workspace, wb) || overlap(a->workspace, wb, a->h0, state_bytes(a)) ||
      overlap(a->workspace, wb, a->h_last, state_bytes(a)) ||
      overlap(a->workspace, wb, a->y, rows_bytes(a->io, p.rows, 0, a->heads * a->value_dim)))
    return SSM_ERR_SHAPE;
  return from_cuda(ssm::launch_gdr_tc(p, a->workspace, cs));
}

ssm_status_t gdr_scan_step(const gdr_step_args_t *a, void *stream) {
  if (!a) return SSM_ERR_NULL;
  ssm_status_t st = check_heads(a);
  if (st != SSM_OK) return st;
  if (a->batch > 0 && (!a->q || !a->k || !a->v || !a->beta || (a->dt && !a->A) || !a->state_io || !a->y))
    return SSM_ERR_NULL;
  if ((double)a->batch * a->heads * a->value_dim > kMaxValues) return SSM_ERR_UNSUPPORTED;
  if (!a->slots && a->state_rows < a->batch) return SSM_ERR_SHAPE;
  if (!all_aligned(16, a->q, a->k, a->v, a->A, a->dt_bias, a->state_io, a->y) ||
      !all_aligned(a->io == SSM_BF16 ? 2 : 4, a->dt, a->beta) || !all_aligned(4, a->slots))
    return SSM_ERR_ALIGN;
  const size_t yb = rows_bytes(a->io, a->batch, 0, a->heads * a->value_dim), sb = state_bytes(a);
  if (a->batch == 0) return SSM_OK;
  if (overlaps_inputs(a, a->batch, a->batch, a->y, yb) || overlaps_inputs(a, a->batch, a->batch, a->state_io, sb) ||
      overlap(a->y, yb, a->state_io, sb))
    return SSM_ERR_SHAPE;
  ssm::GdrParams p;
  fill_heads(p, a);
  p.nseq = a->batch;
  p.L = 1;
  p.rows = a->batch;
  p.h0 = p.h_last = a->state_io;
  p.cu = nullptr;
  return from_cuda(ssm::launch_gdr_step(p, static_cast<cudaStream_t>(stream)));
}

ssm_status_t gdr_gated_rmsnorm_fwd(const gdr_norm_args_t *a, void *stream) {
  if (!a) return SSM_ERR_NULL;
  if (a->io != SSM_F32 && a->io != SSM_BF16) return SSM_ERR_DTYPE;
  if (a->tokens < 0 || a->heads <= 0 || a->width <= 0 || !(a->eps >= 0.f) || a->eps > 3.0e38f)
    return SSM_ERR_SHAPE;
  if (a->flags || a->width > ssm::kHeadNormMaxWidth || a->tokens >= kMaxSize || a->heads > 65535 ||
      a->z_row >= kMaxSize)
    return SSM_ERR_UNSUPPORTED;
  if (a->z_row && a->z_row < a->heads * a->width) return SSM_ERR_SHAPE;
  if (a->tokens > 0 && (!a->x || !a->out)) return SSM_ERR_NULL;
  if (!all_aligned(16, a->x, a->z, a->weight, a->out)) return SSM_ERR_ALIGN;
  const size_t es = a->io == SSM_BF16 ? 2 : 4;
  const int64_t row = a->heads * a->width, zr = a->z_row ? a->z_row : row;
  const size_t bytes = (size_t)(a->tokens * row) * es;
  const size_t zb = a->tokens > 0 ? (size_t)((a->tokens - 1) * zr + row) * es : 0;
  if (a->out != a->x && overlap(a->out, bytes, a->x, bytes)) return SSM_ERR_SHAPE;
  if (overlap(a->out, bytes, a->z, zb) ||
      overlap(a->out, bytes, a->weight, (size_t)a->width * sizeof(float)))
    return SSM_ERR_SHAPE;
  if (a->tokens == 0) return SSM_OK;
  ssm::HeadNormParams p;
  p.tokens = a->tokens;
  p.heads = a->heads;
  p.width = a->width;
  p.z_row = zr;
  p.io = a->io;
  p.eps = a->eps;
  p.x = a->x;
  p.z = a->z;
  p.weight = a->weight;
  p.out = a->out;
  return from_cuda(ssm::launch_head_norm(p, static_cast<cudaStream_t>(stream)));
}

ssm_status_t ssm_conv1d_packed_fwd(const ssm_conv_packed_args_t *a, void *stream) {
  if (!a) return SSM_ERR_NULL;
  if (a->io != SSM_F32 && a->io != SSM_BF16) return SSM_ERR_DTYPE;
  if (a->tokens < 0 || a->channels <= 0 || a->width <= 0 || a->sequences < 0 || a->state_rows < 0)
    return SSM_ERR_SHAPE;
  if (a->width > ssm::kConvMaxWidth || (a->flags & ~SSM_CONV_SILU) || a->tokens >= kMaxSize ||
      a->channels >= (1ll << 24) || a->sequences >= kMaxSize || a->state_rows >= kMaxSize ||
      a->x_row >= kMaxSize)
    return SSM_ERR_UNSUPPORTED;
  if (a->x_row && a->x_row < a->channels) return SSM_ERR_SHAPE;
  if (!a->w) return SSM_ERR_NULL;
  const bool work = a->tokens > 0 && a->sequences > 0;
  if (work && (!a->x || !a->u || !a->cu_seqlens)) return SSM_ERR_NULL;
  if (a->state_io && !a->slots && a->state_rows < a->sequences) return SSM_ERR_SHAPE;
  if (!all_aligned(16, a->x, a->u, a->w, a->bias, a->state_io) ||
      !all_aligned(4, a->cu_seqlens, a->slots))
    return SSM_ERR_ALIGN;
  const size_t es = a->io == SSM_BF16 ? 2 : 4;
  const int64_t xr = a->x_row ? a->x_row : a->channels;
  const size_t xb = work ? (size_t)((a->tokens - 1) * xr + a->channels) * es : 0;
  const size_t ub = work ? (size_t)(a->tokens * a->channels) * es : 0;
  const size_t sb = (size_t)(a->state_rows * a->channels) * (size_t)(a->width - 1) * 4;
  if (!work) return SSM_OK;
  auto overlaps_inputs = [&](const void *out, size_t bytes) {
    return overlap(out, bytes, a->x, xb) ||
           overlap(out, bytes, a->w, (size_t)(a->channels * a->width) * sizeof(float)) ||
           overlap(out, bytes, a->bias, (size_t)a->channels * sizeof(float)) ||
           overlap(out, bytes, a->cu_seqlens, (size_t)(a->sequences + 1) * sizeof(int32_t)) ||
           overlap(out, bytes, a->slots, (size_t)a->sequences * sizeof(int32_t));
  };
  if (overlaps_inputs(a->u, ub) || overlaps_inputs(a->state_io, sb) || overlap(a->state_io, sb, a->u, ub))
    return SSM_ERR_SHAPE;
  ssm::ConvPackedParams p;
  p.tokens = a->tokens;
  p.Cc = a->channels;
  p.nseq = a->sequences;
  p.state_rows = a->state_rows;
  p.x_row = xr;
  p.W = (int)a->width;
  p.io = a->io;
  p.silu = (a->flags & SSM_CONV_SILU) != 0;
  p.x = a->x;
  p.w = a->w;
  p.bias = a->bias;
  p.state = a->width > 1 ? a->state_io : nullptr;
  p.cu = a->cu_seqlens;
  p.slots = a->slots;
  p.u = a->u;
  return from_cuda(ssm::launch_conv1d_packed(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
