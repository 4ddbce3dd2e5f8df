// kvapi.cu -- C entry points of the operators around the attention kernels:
// attn_qk_norm_rope (and its gradient), attn_kv_plan, attn_kv_write / _read and
// attn_kv_decode.  Host-side checks and dispatch; nothing is allocated.
#include <cmath>
#include <cstring>

#include "api.h"
#include "kv.h"

using attn::api_begin;
using attn::api_fail;
using attn::api_launched;
using attn::Region;
using attn::regions_overlap;

namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool is16(attn_dtype_t t) { return t == ATTN_BF16 || t == ATTN_FP16; }

attn_status_t check_status_word(const int32_t* status) {
  if ((uintptr_t)status % 4) return api_fail(ATTN_ERR_ALIGNMENT, "status is not 4-byte aligned");
  return ATTN_OK;
}

attn_status_t check_ints(const char* name, const void* ptr) {
  if (!ptr) return api_fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)ptr % 4) return api_fail(ATTN_ERR_ALIGNMENT, "%s is not 4-byte aligned", name);
  return ATTN_OK;
}

attn_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return api_fail(ATTN_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)ws % 256) return api_fail(ATTN_ERR_ALIGNMENT, "workspace is not 256-byte aligned");
  if (have < need)
    return api_fail(ATTN_ERR_WORKSPACE, "workspace too small (%zu < %zu)", have, need);
  return ATTN_OK;
}

// A [batch][token][head][d] tensor of `es`-byte elements: pointer and strides.
// An output's elements must not share memory, so its strides must be positive
// where the extent is above 1 and heads of one token must not overlap.
attn_status_t check_rows(const char* name, const void* ptr, const int64_t s[3], int64_t batch,
                         int64_t tokens, int64_t heads, int64_t d, int es, bool output) {
  if (!ptr) return api_fail(ATTN_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)ptr % 16) return api_fail(ATTN_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  const int64_t n[3] = {batch, tokens, heads};
  const int64_t al = 16 / es;
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0) return api_fail(ATTN_ERR_INVALID_ARG, "%s stride[%d] is negative", name, i);
    if (n[i] > 1 && s[i] % al)
      return api_fail(ATTN_ERR_ALIGNMENT, "%s stride[%d]=%lld is not a multiple of %lld elements",
                      name, i, (long long)s[i], (long long)al);
  }
  if (!output) return ATTN_OK;
  // sort the axes by stride: each must step over the extent of the smaller ones
  int ax[3] = {2, 1, 0};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j + 1 < 3; ++j)
      if ((n[ax[j]] > 1 ? s[ax[j]] : 0) > (n[ax[j + 1]] > 1 ? s[ax[j + 1]] : 0)) {
        const int t = ax[j];
        ax[j] = ax[j + 1];
        ax[j + 1] = t;
      }
  int64_t extent = d;
  for (int i = 0; i < 3; ++i) {
    if (n[ax[i]] <= 1) continue;
    if (s[ax[i]] < extent)
      return api_fail(ATTN_ERR_INVALID_ARG, "%s: rows share memory (stride[%d]=%lld)", name, ax[i],
                      (long long)s[ax[i]]);
    extent += (n[ax[i]] - 1) * s[ax[i]];
  }
  return ATTN_OK;
}

Region region_of(const void* ptr, const int64_t s[3], int64_t batch, int64_t tokens, int64_t heads,
                 int64_t d, int es) {
  Region r;
  r.lo = (uintptr_t)ptr;
  if (batch <= 0 || tokens <= 0 || heads <= 0) return r;
  // the axes that go anywhere, by stride
  const int64_t n[3] = {batch, tokens, heads};
  int ax[3], m = 0;
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1 || s[i] == 0) continue;
    int j = m++;
    for (; j > 0 && s[ax[j - 1]] > s[i]; --j) ax[j] = ax[j - 1];
    ax[j] = i;
  }
  int64_t width = d;  // of the axes inside the cut
  for (int k = 0; k < m; ++k) {
    const int64_t pitch = s[ax[k]];
    bool even = pitch >= width;
    for (int j = k + 1; j < m; ++j) even = even && s[ax[j]] % pitch == 0;
    if (even) r.rows[r.ways++] = {pitch * es, width * es};
    width += (n[ax[k]] - 1) * pitch;
  }
  r.bytes = width * es;
  return r;
}

Region flat(const void* ptr, int64_t bytes) {
  Region r;
  r.lo = (uintptr_t)ptr;
  r.bytes = bytes;
  return r;
}

// ------------------------------------------------------------------ norm and rotation

attn_status_t check_qk(const attn_qk_params_t* p) {
  if (!p) return api_fail(ATTN_ERR_INVALID_ARG, "params is NULL");
  if (!is16(p->dtype)) return api_fail(ATTN_ERR_UNSUPPORTED, "dtype must be BF16 or FP16");
  if (p->w_dtype != p->dtype && p->w_dtype != ATTN_FP32)
    return api_fail(ATTN_ERR_UNSUPPORTED, "w_dtype must equal dtype or be FP32");
  if (p->batch < 0 || p->seqlen < 0) return api_fail(ATTN_ERR_INVALID_ARG, "batch or seqlen < 0");
  if ((int64_t)p->batch * p->seqlen > INT32_MAX)
    return api_fail(ATTN_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens");
  if (p->heads_q <= 0 || p->heads_k < 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "heads_q must be positive and heads_k >= 0");
  if (p->heads_q > 65536 || p->heads_k > 65536)
    return api_fail(ATTN_ERR_UNSUPPORTED, "more than 65536 heads");
  const int d = p->head_dim;
  if (d != 64 && d != 128 && d != 192 && d != 256 && d != 512)
    return api_fail(ATTN_ERR_UNSUPPORTED, "head_dim %d: use 64, 128, 192, 256 or 512", d);
  if (p->rotary_dim < 0 || p->rotary_dim > d || p->rotary_dim % 16)
    return api_fail(ATTN_ERR_UNSUPPORTED, "rotary_dim %d: use a multiple of 16 up to head_dim",
                    p->rotary_dim);
  if (p->rotary_dim > 0 && p->max_pos < 0) return api_fail(ATTN_ERR_INVALID_ARG, "max_pos < 0");
  if (!std::isfinite(p->eps) || p->eps < 0.0f)
    return api_fail(ATTN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return ATTN_OK;
}

// The checks both directions share, and the kernel's parameters.
attn_status_t setup_qk(const attn_qk_params_t* p, const void* q, const void* k, const void* w_q,
                       const void* w_k, const float* cos, const float* sin,
                       const int32_t* positions, void* q_out, void* k_out, int32_t* status,
                       attn::QkParams& kp) {
  attn_status_t s;
  if (!p->norm && (w_q || w_k))
    return api_fail(ATTN_ERR_INVALID_ARG, "norm weights without norm");
  if (p->rotary_dim > 0 && p->max_pos > 0) {  // (tables of no rows are not read)
    if (!cos || !sin) return api_fail(ATTN_ERR_INVALID_ARG, "cos or sin is NULL");
    if ((uintptr_t)cos % 16 || (uintptr_t)sin % 16)
      return api_fail(ATTN_ERR_ALIGNMENT, "cos and sin must be 16-byte aligned");
  }
  if ((uintptr_t)w_q % 16 || (uintptr_t)w_k % 16)
    return api_fail(ATTN_ERR_ALIGNMENT, "norm weights must be 16-byte aligned");
  if (positions && (s = check_ints("positions", positions))) return s;
  if ((s = check_status_word(status))) return s;
  const void* x[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int64_t *xs[2] = {p->stride_q, p->stride_k}, *os[2] = {p->stride_qo, p->stride_ko};
  const int heads[2] = {p->heads_q, p->heads_k};
  static const char* const xn[2] = {"q", "k"};
  static const char* const on[2] = {"the output of q", "the output of k"};
  memset(&kp, 0, sizeof(kp));
  for (int i = 0; i < 2; ++i) {
    if (!heads[i]) continue;
    if ((s = check_rows(xn[i], x[i], xs[i], p->batch, p->seqlen, heads[i], p->head_dim, 2, false)) ||
        (s = check_rows(on[i], out[i], os[i], p->batch, p->seqlen, heads[i], p->head_dim, 2, true)))
      return s;
    attn::QkSide& sd = kp.side[i];
    sd.x = x[i];
    sd.out = out[i];
    sd.w = i ? w_k : w_q;
    sd.heads = heads[i];
    sd.x_b = xs[i][0], sd.x_t = xs[i][1], sd.x_h = xs[i][2];
    sd.o_b = os[i][0], sd.o_t = os[i][1], sd.o_h = os[i][2];
  }
  kp.cos = cos;
  kp.sin = sin;
  kp.positions = positions;
  kp.batch = p->batch;
  kp.seqlen = p->seqlen;
  kp.d = p->head_dim;
  kp.rot = p->rotary_dim;
  kp.inter = p->interleaved ? 1 : 0;
  kp.norm = p->norm ? 1 : 0;
  kp.w_f32 = p->w_dtype == ATTN_FP32;
  kp.max_pos = p->max_pos;
  kp.eps = p->eps;
  kp.status = status;
  return ATTN_OK;
}

Region qk_region(const attn_qk_params_t* p, const void* ptr, const int64_t s[3], int heads) {
  return region_of(ptr, s, p->batch, p->seqlen, heads, p->head_dim, 2);
}

bool same_view(const attn_qk_params_t* p, const void* a, const int64_t sa[3], const void* b,
               const int64_t sb[3], int heads) {
  return a == b && (p->batch == 1 || sa[0] == sb[0]) && (p->seqlen == 1 || sa[1] == sb[1]) &&
         (heads == 1 || sa[2] == sb[2]);
}

// Reads besides the rows themselves: weights, tables, positions.
attn_status_t check_qk_small(const attn_qk_params_t* p, const Region* outs, int n, const void* w_q,
                             const void* w_k, const float* cos, const float* sin,
                             const int32_t* positions, const int32_t* status) {
  const int64_t wb = (int64_t)p->head_dim * (p->w_dtype == ATTN_FP32 ? 4 : 2);
  const int64_t tb = (int64_t)p->max_pos * (p->rotary_dim / 2) * 4;
  const Region in[6] = {flat(w_q, w_q ? wb : 0), flat(w_k, w_k ? wb : 0),
                        flat(cos, p->rotary_dim ? tb : 0), flat(sin, p->rotary_dim ? tb : 0),
                        flat(positions, positions ? (int64_t)p->batch * p->seqlen * 4 : 0),
                        flat(status, status ? 4 : 0)};
  for (int i = 0; i < n; ++i)
    for (const Region& r : in)
      if (regions_overlap(outs[i], r))
        return api_fail(ATTN_ERR_INVALID_ARG, "an output overlaps weights, tables, positions or status");
  return ATTN_OK;
}

// 0: too many rows for a call
size_t qk_partial_bytes(const attn_qk_params_t* p, attn::QkParams& kp) {
  kp.batch = p->batch;
  kp.seqlen = p->seqlen;
  kp.side[0].heads = p->heads_q;
  kp.side[1].heads = p->heads_k;
  kp.d = p->head_dim;
  if (!attn::qk_bwd_blocks(kp, attn::num_sms())) return 0;
  return up256((size_t)(kp.blocks[0] + kp.blocks[1]) * p->head_dim * 4);
}

}  // namespace

extern "C" {

attn_status_t attn_qk_norm_rope(const attn_qk_params_t* p, const void* q, const void* k,
                                const void* w_q, const void* w_k, const float* cos,
                                const float* sin, const int32_t* positions, void* q_out,
                                void* k_out, int32_t* status, attn_stream_t stream) {
  api_begin();
  attn_status_t s = check_qk(p);
  if (s) return s;
  if (p->batch == 0 || p->seqlen == 0) return ATTN_OK;
  attn::QkParams kp;
  if ((s = setup_qk(p, q, k, w_q, w_k, cos, sin, positions, q_out, k_out, status, kp))) return s;
  const Region in[2] = {qk_region(p, q, p->stride_q, p->heads_q),
                        qk_region(p, k, p->stride_k, p->heads_k)};
  const Region out[2] = {qk_region(p, q_out, p->stride_qo, p->heads_q),
                         qk_region(p, k_out, p->stride_ko, p->heads_k)};
  const bool inplace[2] = {same_view(p, q, p->stride_q, q_out, p->stride_qo, p->heads_q),
                           same_view(p, k, p->stride_k, k_out, p->stride_ko, p->heads_k)};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (!(i == j && inplace[i]) && regions_overlap(out[i], in[j]))
        return api_fail(ATTN_ERR_INVALID_ARG, "an output overlaps an input");
  if (regions_overlap(out[0], out[1])) return api_fail(ATTN_ERR_INVALID_ARG, "outputs overlap");
  if ((s = check_qk_small(p, out, 2, w_q, w_k, cos, sin, positions, status))) return s;
  const cudaError_t e =
      attn::launch_qk_fwd(kp, p->dtype == ATTN_BF16, attn::num_sms(), (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return api_fail(ATTN_ERR_UNSUPPORTED, "too many rows for one call");
  return api_launched(e, 1, "norm and rotation kernel launch");
}

size_t attn_qk_norm_rope_bwd_workspace_size(const attn_qk_params_t* p) {
  if (!p || check_qk(p)) return 256;
  attn::QkParams kp;
  memset(&kp, 0, sizeof(kp));
  const size_t n = qk_partial_bytes(p, kp);
  return n < 256 ? 256 : n;
}

attn_status_t attn_qk_norm_rope_bwd(const attn_qk_params_t* p, const void* q, const void* k,
                                    const void* w_q, const void* w_k, const float* cos,
                                    const float* sin, const int32_t* positions,
                                    const void* dq_out, const void* dk_out, void* dq, void* dk,
                                    float* dw_q, float* dw_k, void* ws, size_t ws_bytes,
                                    int32_t* status, attn_stream_t stream) {
  api_begin();
  attn_status_t s = check_qk(p);
  if (s) return s;
  if ((dw_q && !w_q) || (dw_k && (!w_k || !p->heads_k)))
    return api_fail(ATTN_ERR_INVALID_ARG, "a gradient of weights that are not given");
  if ((uintptr_t)dw_q % 4 || (uintptr_t)dw_k % 4)
    return api_fail(ATTN_ERR_ALIGNMENT, "dw_q and dw_k must be 4-byte aligned");
  cudaStream_t st = (cudaStream_t)stream;
  if (p->batch == 0 || p->seqlen == 0) {  // no rows: the sums are zero
    float* const dw[2] = {dw_q, dw_k};
    for (float* w : dw)
      if (w && (s = api_launched(cudaMemsetAsync(w, 0, (size_t)p->head_dim * 4, st), 0, "dw reset")))
        return s;
    return ATTN_OK;
  }
  attn::QkParams kp;
  if ((s = setup_qk(p, q, k, w_q, w_k, cos, sin, positions, dq, dk, status, kp))) return s;
  const int heads[2] = {p->heads_q, p->heads_k};
  const void* dz[2] = {dq_out, dk_out};
  const int64_t* zs[2] = {p->stride_dqo, p->stride_dko};
  static const char* const zn[2] = {"dq_out", "dk_out"};
  for (int i = 0; i < 2; ++i) {
    if (!heads[i]) continue;
    if ((s = check_rows(zn[i], dz[i], zs[i], p->batch, p->seqlen, heads[i], p->head_dim, 2, false)))
      return s;
    kp.side[i].dz = dz[i];
    kp.side[i].dz_b = zs[i][0], kp.side[i].dz_t = zs[i][1], kp.side[i].dz_h = zs[i][2];
    kp.side[i].dw = i ? dw_k : dw_q;
  }
  const Region in[4] = {qk_region(p, q, p->stride_q, p->heads_q),
                        qk_region(p, k, p->stride_k, p->heads_k),
                        qk_region(p, dq_out, p->stride_dqo, p->heads_q),
                        qk_region(p, dk_out, p->stride_dko, p->heads_k)};
  const size_t need = qk_partial_bytes(p, kp);
  if (!need) return api_fail(ATTN_ERR_UNSUPPORTED, "too many rows for one call");
  if ((s = check_workspace(ws, ws_bytes, need))) return s;
  const int64_t wb = (int64_t)p->head_dim * 4;
  const Region out[5] = {qk_region(p, dq, p->stride_qo, p->heads_q),
                         qk_region(p, dk, p->stride_ko, p->heads_k), flat(dw_q, dw_q ? wb : 0),
                         flat(dw_k, dw_k ? wb : 0), flat(ws, (int64_t)need)};
  const bool inplace[2] = {same_view(p, dq_out, p->stride_dqo, dq, p->stride_qo, p->heads_q),
                           same_view(p, dk_out, p->stride_dko, dk, p->stride_ko, p->heads_k)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 4; ++j)
      if (!(i < 2 && j == i + 2 && inplace[i]) && regions_overlap(out[i], in[j]))
        return api_fail(ATTN_ERR_INVALID_ARG, "a gradient or the workspace overlaps an input");
    for (int j = i + 1; j < 5; ++j)
      if (regions_overlap(out[i], out[j])) return api_fail(ATTN_ERR_INVALID_ARG, "outputs overlap");
  }
  if ((s = check_qk_small(p, out, 5, w_q, w_k, cos, sin, positions, status))) return s;
  kp.partial = (float*)ws;
  const cudaError_t e = attn::launch_qk_bwd(kp, p->dtype == ATTN_BF16, st);
  return api_launched(e, dw_q || dw_k ? 2 : 1, "norm and rotation gradient launch");
}

// ------------------------------------------------------------------ page plan

attn_status_t attn_kv_plan(const attn_kv_plan_params_t* p, const int32_t* context,
                           const int32_t* fresh, int32_t* block_table,
                           const int32_t* free_pages, const int32_t* free_head,
                           int32_t* cu_seqlens, int32_t* seq_lens, int32_t* positions,
                           int32_t* slots, int32_t* free_head_out, int32_t* status,
                           attn_stream_t stream) {
  api_begin();
  attn_status_t s;
  if (!p) return api_fail(ATTN_ERR_INVALID_ARG, "params is NULL");
  if (p->batch < 0 || p->cols < 0 || p->rows < 0 || p->num_pages < 0 || p->n_free < 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "a size is negative");
  if (p->batch > attn::kPlanMaxBatch)
    return api_fail(ATTN_ERR_UNSUPPORTED, "batch %d > %d", p->batch, attn::kPlanMaxBatch);
  int shift = 0;
  while ((1 << shift) < p->page_size && shift < 8) ++shift;
  if (p->page_size < 16 || (1 << shift) != p->page_size)
    return api_fail(ATTN_ERR_UNSUPPORTED, "page_size %d: use 16, 32, 64, 128 or 256", p->page_size);
  if (((int64_t)p->cols << shift) > (1 << 30))
    return api_fail(ATTN_ERR_UNSUPPORTED, "cols * page_size > 2^30");
  if (((int64_t)p->num_pages << shift) > INT32_MAX)
    return api_fail(ATTN_ERR_UNSUPPORTED, "num_pages * page_size >= 2^31");
  if ((int64_t)p->batch * p->cols > INT32_MAX)
    return api_fail(ATTN_ERR_UNSUPPORTED, "batch * cols >= 2^31");
  if (p->batch > 1 && p->table_stride < p->cols)
    return api_fail(ATTN_ERR_INVALID_ARG, "table_stride < cols: rows of the table overlap");
  if ((s = check_status_word(status)) || (s = check_ints("cu_seqlens", cu_seqlens))) return s;
  if (p->batch && ((s = check_ints("context", context)) || (s = check_ints("fresh", fresh)) ||
                   (s = check_ints("seq_lens", seq_lens)) ||
                   (p->cols && (s = check_ints("block_table", block_table)))))
    return s;
  if (p->rows && ((s = check_ints("positions", positions)) || (s = check_ints("slots", slots))))
    return s;
  if (free_pages && ((s = check_ints("free_pages", free_pages)) ||
                     (s = check_ints("free_head", free_head)) ||
                     (s = check_ints("free_head_out", free_head_out))))
    return s;
  const int64_t tb = p->batch ? ((p->batch - 1) * p->table_stride + p->cols) * 4 : 0;
  const Region in[4] = {flat(context, p->batch * 4ll), flat(fresh, p->batch * 4ll),
                        flat(free_pages, free_pages ? p->n_free * 4ll : 0),
                        flat(free_head, free_pages ? 4 : 0)};
  const Region out[7] = {flat(cu_seqlens, (p->batch + 1) * 4ll), flat(seq_lens, p->batch * 4ll),
                         flat(positions, p->rows * 4ll), flat(slots, p->rows * 4ll),
                         flat(free_head_out, free_pages ? 4 : 0), flat(block_table, tb),
                         flat(status, status ? 4 : 0)};
  for (int i = 0; i < 7; ++i) {
    for (const Region& r : in)
      if (regions_overlap(out[i], r)) return api_fail(ATTN_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = i + 1; j < 7; ++j)
      if (regions_overlap(out[i], out[j])) return api_fail(ATTN_ERR_INVALID_ARG, "outputs overlap");
  }
  attn::PlanParams kp;
  memset(&kp, 0, sizeof(kp));
  kp.ctx = context;
  kp.fresh = fresh;
  kp.free_pages = free_pages;
  kp.free_head = free_pages ? free_head : nullptr;
  kp.table = block_table;
  kp.cu = cu_seqlens;
  kp.seq = seq_lens;
  kp.pos = positions;
  kp.slots = slots;
  kp.free_head_out = free_pages ? free_head_out : nullptr;
  kp.table_stride = p->table_stride;
  kp.batch = p->batch;
  kp.cols = p->cols;
  kp.page_shift = shift;
  kp.num_pages = p->num_pages;
  kp.rows = p->rows;
  kp.n_free = free_pages ? p->n_free : 0;
  kp.status = status;
  return api_launched(attn::launch_kv_plan(kp, attn::num_sms(), (cudaStream_t)stream), 1,
                      "page plan kernel launch");
}

}  // extern "C"

// ------------------------------------------------------------------ the 4-bit cache
namespace {

attn_status_t check_cache(const attn_kv4_cache_t* c, attn::Kv4& out) {
  if (!c) return api_fail(ATTN_ERR_INVALID_ARG, "cache is NULL");
  if (c->num_pages < 0 || c->heads_kv <= 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "num_pages < 0 or heads_kv < 1");
  if (c->heads_kv > 65536) return api_fail(ATTN_ERR_UNSUPPORTED, "more than 65536 heads");
  const bool dims = (c->d_qk == 64 && c->d_v == 64) || (c->d_qk == 128 && c->d_v == 128) ||
                    (c->d_qk == 192 && c->d_v == 128) || (c->d_qk == 256 && c->d_v == 256);
  if (!dims)
    return api_fail(ATTN_ERR_UNSUPPORTED,
                    "cache head dims (%d,%d): use (64,64) (128,128) (192,128) (256,256)", c->d_qk,
                    c->d_v);
  int shift = 0;
  while ((1 << shift) < c->page_size && shift < 8) ++shift;
  if (c->page_size < 16 || (1 << shift) != c->page_size)
    return api_fail(ATTN_ERR_UNSUPPORTED, "page_size %d: use 16, 32, 64, 128 or 256", c->page_size);
  if (((int64_t)c->num_pages << shift) > INT32_MAX)
    return api_fail(ATTN_ERR_UNSUPPORTED, "num_pages * page_size >= 2^31");
  const void* ptr[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
  for (const void* x : ptr) {
    if (c->num_pages && !x) return api_fail(ATTN_ERR_INVALID_ARG, "a cache array is NULL");
    if ((uintptr_t)x % 16) return api_fail(ATTN_ERR_ALIGNMENT, "a cache array is not 16-byte aligned");
  }
  out.k_codes = (uint8_t*)c->k_codes;
  out.v_codes = (uint8_t*)c->v_codes;
  out.k_scales = (uint16_t*)c->k_scales;
  out.v_scales = (uint16_t*)c->v_scales;
  out.num_pages = c->num_pages;
  out.page_size = c->page_size;
  out.page_shift = shift;
  out.heads = c->heads_kv;
  out.d_qk = c->d_qk;
  out.d_v = c->d_v;
  return ATTN_OK;
}

void cache_regions(const attn_kv4_cache_t* c, Region (&r)[4]) {
  const int64_t rows = (int64_t)c->num_pages * c->heads_kv * c->page_size;
  r[0] = flat(c->k_codes, rows * (c->d_qk / 2));
  r[1] = flat(c->k_scales, rows * (c->d_qk / 32) * 2);
  r[2] = flat(c->v_codes, rows * (c->d_v / 2));
  r[3] = flat(c->v_scales, rows * (c->d_v / 32) * 2);
}

attn_status_t rows_impl(const attn_kv4_cache_t* c, attn_dtype_t dtype, int tokens, const void* k,
                        const int64_t sk[2], const void* v, const int64_t sv[2],
                        const int32_t* slots, int32_t* status, attn_stream_t stream, bool write) {
  api_begin();
  attn::KvRowsParams kp;
  memset(&kp, 0, sizeof(kp));
  attn_status_t s = check_cache(c, kp.c);
  if (s) return s;
  if (!is16(dtype)) return api_fail(ATTN_ERR_UNSUPPORTED, "dtype must be BF16 or FP16");
  if (tokens < 0) return api_fail(ATTN_ERR_INVALID_ARG, "tokens < 0");
  if ((s = check_status_word(status))) return s;
  if (tokens == 0) return ATTN_OK;
  if (!sk || !sv) return api_fail(ATTN_ERR_INVALID_ARG, "strides must not be NULL");
  const int64_t vecs = (int64_t)c->heads_kv * (c->d_qk + c->d_v) / 8;
  if (vecs * tokens > INT32_MAX)
    return api_fail(ATTN_ERR_UNSUPPORTED, "more than 2^34 elements in one call");
  const int64_t k3[3] = {0, sk[0], sk[1]}, v3[3] = {0, sv[0], sv[1]};
  if ((s = check_rows("k", k, k3, 1, tokens, c->heads_kv, c->d_qk, 2, !write)) ||
      (s = check_rows("v", v, v3, 1, tokens, c->heads_kv, c->d_v, 2, !write)) ||
      (s = check_ints("slots", slots)))
    return s;
  Region held[4];
  cache_regions(c, held);
  const Region rows[2] = {region_of(k, k3, 1, tokens, c->heads_kv, c->d_qk, 2),
                          region_of(v, v3, 1, tokens, c->heads_kv, c->d_v, 2)};
  const Region ints[2] = {flat(slots, tokens * 4ll), flat(status, status ? 4 : 0)};
  for (const Region& h : held) {
    for (const Region& r : rows)
      if (regions_overlap(h, r)) return api_fail(ATTN_ERR_INVALID_ARG, "k or v overlaps the cache");
    for (const Region& r : ints)
      if (write && regions_overlap(h, r))
        return api_fail(ATTN_ERR_INVALID_ARG, "slots or status overlaps the cache");
  }
  if (write) {
    for (int i = 0; i < 4; ++i)
      for (int j = i + 1; j < 4; ++j)
        if (regions_overlap(held[i], held[j]))
          return api_fail(ATTN_ERR_INVALID_ARG, "arrays of the cache overlap");
  } else {
    if (regions_overlap(rows[0], rows[1])) return api_fail(ATTN_ERR_INVALID_ARG, "k overlaps v");
    for (const Region& r : rows)
      for (const Region& i : ints)
        if (regions_overlap(r, i)) return api_fail(ATTN_ERR_INVALID_ARG, "k or v overlaps slots or status");
  }
  kp.k = const_cast<void*>(k);
  kp.v = const_cast<void*>(v);
  kp.k_t = sk[0], kp.k_h = sk[1], kp.v_t = sv[0], kp.v_h = sv[1];
  kp.slots = slots;
  kp.tokens = tokens;
  kp.per_token = attn::FastDiv::of((uint32_t)vecs);
  kp.vec_k = attn::FastDiv::of((uint32_t)c->d_qk / 8);
  kp.vec_v = attn::FastDiv::of((uint32_t)c->d_v / 8);
  kp.status = status;
  const bool bf16 = dtype == ATTN_BF16;
  const cudaError_t e = write ? attn::launch_kv4_write(kp, bf16, attn::num_sms(), (cudaStream_t)stream)
                              : attn::launch_kv4_read(kp, bf16, attn::num_sms(), (cudaStream_t)stream);
  return api_launched(e, 1, write ? "cache write launch" : "cache read launch");
}

attn_status_t check_decode(const attn_kv4_decode_params_t* p, const attn_kv4_cache_t* c,
                           attn::DecodeParams& kp) {
  memset(&kp, 0, sizeof(kp));
  attn_status_t s = check_cache(c, kp.c);
  if (s) return s;
  if (!p) return api_fail(ATTN_ERR_INVALID_ARG, "params is NULL");
  if (!is16(p->dtype)) return api_fail(ATTN_ERR_UNSUPPORTED, "dtype must be BF16 or FP16");
  if (p->o_dtype != p->dtype && p->o_dtype != ATTN_FP32)
    return api_fail(ATTN_ERR_UNSUPPORTED, "o_dtype must equal dtype or be FP32");
  if (p->batch < 0 || p->seqlen_q < 0 || p->cols < 0 || p->heads_q <= 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "a size is negative, or heads_q < 1");
  if (p->seqlen_q > 256)
    return api_fail(ATTN_ERR_UNSUPPORTED,
                    "seqlen_q %d > 256: read the keys back (attn_kv_read) and use attn_fwd",
                    p->seqlen_q);
  if (p->heads_q % c->heads_kv)
    return api_fail(ATTN_ERR_INVALID_ARG, "heads_q (%d) is not divisible by heads_kv (%d)",
                    p->heads_q, c->heads_kv);
  if (p->heads_q / c->heads_kv > 128)
    return api_fail(ATTN_ERR_UNSUPPORTED, "more than 128 query heads for a kv head");
  if (((int64_t)p->cols << kp.c.page_shift) > (1 << 30))
    return api_fail(ATTN_ERR_UNSUPPORTED, "cols * page_size > 2^30");
  if (p->batch > 1 && p->table_stride < 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "table_stride < 0");
  if (p->window_left < -1 || p->sinks < 0)
    return api_fail(ATTN_ERR_INVALID_ARG, "window_left < -1 or sinks < 0");
  if (!(p->softmax_scale > 0.0f) || !std::isfinite(p->softmax_scale))
    return api_fail(ATTN_ERR_INVALID_ARG, "softmax_scale must be positive and finite");
  kp.batch = p->batch;
  kp.seqlen_q = p->seqlen_q;
  kp.heads_q = p->heads_q;
  kp.group = p->heads_q / c->heads_kv;
  kp.rows = p->seqlen_q * kp.group;
  const int per = 8 * attn::decode_col_tiles(kp.rows, c->d_v);
  kp.row_blocks = (kp.rows + per - 1) / per;
  kp.by_group = attn::FastDiv::of((uint32_t)kp.group);
  kp.by_blocks = attn::FastDiv::of((uint32_t)std::max(kp.row_blocks, 1));
  kp.cols = p->cols;
  kp.table_stride = p->table_stride;
  // a window as long as the longest sequence hides nothing
  const int64_t most = (int64_t)p->cols << kp.c.page_shift;
  kp.window_left = p->window_left >= 0 && p->window_left < most ? p->window_left : -1;
  kp.sinks = (int)(p->sinks < most ? p->sinks : most);
  kp.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  kp.o_f32 = p->o_dtype == ATTN_FP32;
  if ((int64_t)kp.batch * c->heads_kv * kp.row_blocks * per > INT32_MAX)
    return api_fail(ATTN_ERR_UNSUPPORTED, "batch * heads too large for the grid");
  return ATTN_OK;
}

// [two ints for each item][one for each run][two partial results a run]
struct DecodeLayout {
  size_t ends, partial, total;
  int blocks;
};
DecodeLayout decode_layout(const attn::DecodeParams& kp) {
  DecodeLayout l;
  const size_t items = (size_t)kp.batch * kp.c.heads * kp.row_blocks;
  l.blocks = attn::decode_blocks(kp, attn::num_sms());
  l.ends = up256(items * 8);
  l.partial = l.ends + up256(attn::decode_runs(l.blocks) * 4);
  const int rows = 8 * attn::decode_col_tiles(kp.rows, kp.c.d_v);
  l.total = l.partial + attn::decode_partial_floats(l.blocks, rows, kp.c.d_v) * 4;
  return l;
}

}  // namespace

extern "C" {

attn_status_t attn_kv_write(const attn_kv4_cache_t* cache, attn_dtype_t dtype, int tokens,
                             const void* k, const int64_t stride_k[2], const void* v,
                             const int64_t stride_v[2], const int32_t* slots, int32_t* status,
                             attn_stream_t stream) {
  return rows_impl(cache, dtype, tokens, k, stride_k, v, stride_v, slots, status, stream, true);
}

attn_status_t attn_kv_read(const attn_kv4_cache_t* cache, attn_dtype_t dtype, int tokens,
                            void* k, const int64_t stride_k[2], void* v,
                            const int64_t stride_v[2], const int32_t* slots, int32_t* status,
                            attn_stream_t stream) {
  return rows_impl(cache, dtype, tokens, k, stride_k, v, stride_v, slots, status, stream, false);
}

size_t attn_kv_decode_workspace_size(const attn_kv4_decode_params_t* p,
                                      const attn_kv4_cache_t* cache) {
  attn::DecodeParams kp;
  if (check_decode(p, cache, kp)) return 256;
  return decode_layout(kp).total;
}

attn_status_t attn_kv_decode(const attn_kv4_decode_params_t* p, const attn_kv4_cache_t* cache,
                              const void* q, const int32_t* block_table,
                              const int32_t* seq_lens, void* o, float* lse, void* ws,
                              size_t ws_bytes, int32_t* status, attn_stream_t stream) {
  api_begin();
  attn::DecodeParams kp;
  attn_status_t s = check_decode(p, cache, kp);
  if (s) return s;
  if ((s = check_status_word(status))) return s;
  const DecodeLayout l = decode_layout(kp);
  if ((s = check_workspace(ws, ws_bytes, l.total))) return s;
  if (p->batch == 0 || p->seqlen_q == 0) return ATTN_OK;
  const int oe = kp.o_f32 ? 4 : 2;
  if ((s = check_rows("q", q, p->stride_q, p->batch, p->seqlen_q, p->heads_q, cache->d_qk, 2, false)) ||
      (s = check_rows("o", o, p->stride_o, p->batch, p->seqlen_q, p->heads_q, cache->d_v, oe, true)) ||
      (s = check_ints("lse", lse)) || (s = check_ints("seq_lens", seq_lens)) ||
      (p->cols && (s = check_ints("block_table", block_table))))
    return s;
  Region in[7];
  Region held[4];
  cache_regions(cache, held);
  for (int i = 0; i < 4; ++i) in[i] = held[i];
  in[4] = region_of(q, p->stride_q, p->batch, p->seqlen_q, p->heads_q, cache->d_qk, 2);
  in[5] = flat(block_table, p->cols ? ((p->batch - 1) * p->table_stride + p->cols) * 4 : 0);
  in[6] = flat(seq_lens, p->batch * 4ll);
  const Region out[4] = {region_of(o, p->stride_o, p->batch, p->seqlen_q, p->heads_q, cache->d_v, oe),
                         flat(lse, (int64_t)p->batch * p->heads_q * p->seqlen_q * 4),
                         flat(ws, (int64_t)l.total), flat(status, status ? 4 : 0)};
  for (int i = 0; i < 4; ++i) {
    for (const Region& r : in)
      if (regions_overlap(out[i], r))
        return api_fail(ATTN_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    for (int j = i + 1; j < 4; ++j)
      if (regions_overlap(out[i], out[j])) return api_fail(ATTN_ERR_INVALID_ARG, "outputs overlap");
  }
  kp.q = q;
  kp.o = o;
  kp.lse = lse;
  kp.table = block_table;
  kp.seq_lens = seq_lens;
  kp.q_b = p->stride_q[0], kp.q_t = p->stride_q[1], kp.q_h = p->stride_q[2];
  kp.o_b = p->stride_o[0], kp.o_t = p->stride_o[1], kp.o_h = p->stride_o[2];
  kp.info = (int*)ws;
  kp.ends = (int*)((char*)ws + l.ends);
  kp.partial = (float*)((char*)ws + l.partial);
  kp.status = status;
  const cudaError_t e =
      attn::launch_kv4_decode(kp, p->dtype == ATTN_BF16, l.blocks, (cudaStream_t)stream);
  return api_launched(e, 2, "cache attention launch");
}

}  // extern "C"
