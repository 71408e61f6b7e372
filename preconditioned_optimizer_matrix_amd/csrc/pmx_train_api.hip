// C ABI of the training-step operators (include/pmx.h): argument checks and
// launches of the products grouped by expert, the token embedding and the
// distillation loss.  Nothing is enqueued unless every check has passed.
#include <math.h>

#include "pmx_checks.h"
#include "pmx_train.h"

namespace pmx {
namespace {

bool grouped_shape_ok(int64_t rows, int a, int b, int groups) {
  return rows >= 0 && rows <= kMaxRows && a >= 1 && a <= kMaxSide && b >= 1 && b <= kMaxSide &&
         groups >= 1 && groups <= PMX_MAX_GROUPS;
}
// tile counts and their splits are 32-bit on the device (32 x 128 tiles at least)
bool grouped_items_ok(int64_t rows, int n, int groups) {
  return (rows / 32 + groups) * (int64_t)((n + 127) / 128) * 64 <= kMaxRows;
}
size_t product_ws(int64_t rows, int k, int n, int groups, pmx_dtype t) {
  const int s = rows ? grouped_product_splits(rows, k, n, groups, t) : 1;
  return s > 1 ? (size_t)s * rows * n * sizeof(float) : 0;
}
size_t outer_ws(int64_t rows, int m, int n, int groups, pmx_dtype t) {
  const int s = grouped_outer_splits(rows, m, n, groups, t);
  return s > 1 ? (size_t)s * groups * m * n * sizeof(float) : 0;
}

DistillParams distill_params(const pmx_distill_problem* q, const pmx_context* h) {
  DistillParams p = {};
  p.z = q->z;
  p.ldz = q->ldz;
  p.ids = q->teacher_ids;
  p.ld_ids = q->ld_ids;
  p.teacher = q->teacher;
  p.ld_teacher = q->ld_teacher;
  p.labels = q->labels;
  p.weights = q->weights;
  p.rows = q->rows;
  p.vocab = q->vocab;
  p.top = q->top;
  p.dtype = q->dtype;
  p.teacher_dtype = q->teacher_dtype;
  p.ids64 = q->ids_type == PMX_I64;
  p.labels64 = q->labels_type == PMX_I64;
  p.tau = q->tau;
  p.mix = q->mix;
  p.num_cu = h->num_cu;
  return p;
}

bool distill_shape_ok(const pmx_distill_problem* q) {
  return q && q->struct_version == 1 && q->reserved == 0 && dtype_ok(q->dtype) && dtype_ok(q->teacher_dtype) &&
         q->rows >= 0 && q->rows <= kMaxRows && q->vocab >= 1 && q->vocab <= PMX_MAX_VOCAB && q->top >= 0 &&
         q->top <= PMX_MAX_TOP;
}

bool distill_ok(const pmx_distill_problem* q) {
  if (!distill_shape_ok(q)) return false;
  if (!itype_ok(q->ids_type) || !itype_ok(q->labels_type)) return false;
  // below, a difference of logits over tau leaves fp32's range
  if (!(q->tau >= 0x1p-100f) || !isfinite(q->tau) || !(q->mix >= 0.f) || !(q->mix <= 1.f)) return false;
  if (q->mix > 0.f && q->top < 1) return false;
  if (q->mix < 1.f && q->rows > 0 && !q->labels) return false;
  if (!layout_ok(q->z, q->rows, q->vocab, q->ldz, elem_size(q->dtype))) return false;
  if (q->top > 0 &&
      (!layout_ok(q->teacher_ids, q->rows, q->top, q->ld_ids, index_size(q->ids_type)) ||
       !layout_ok(q->teacher, q->rows, q->top, q->ld_teacher, elem_size(q->teacher_dtype))))
    return false;
  return (uintptr_t)q->labels % index_size(q->labels_type) == 0 && (uintptr_t)q->weights % 4 == 0;
}

// dz may be z itself (same address and row distance); any other overlap is refused.
bool dz_aliases(const pmx_distill_problem* q, const void* dz, int64_t lddz) {
  const size_t es = elem_size(q->dtype);
  const Extent out = extent(dz, q->rows, q->vocab, lddz, es);
  if (overlap(out, extent(q->z, q->rows, q->vocab, q->ldz, es)) && !(dz == q->z && lddz == q->ldz)) return true;
  const Extent in[] = {
      extent(q->teacher_ids, q->rows, q->top, q->ld_ids, index_size(q->ids_type)),
      extent(q->teacher, q->rows, q->top, q->ld_teacher, elem_size(q->teacher_dtype)),
      extent(q->labels, 1, q->rows, q->rows, index_size(q->labels_type)),
      extent(q->weights, 1, q->rows, q->rows, 4)};
  return any_overlap(out, in);
}

}  // namespace
}  // namespace pmx

using namespace pmx;

extern "C" {

// ------------------------------------------------------------ grouped products
pmx_status pmx_grouped_product_workspace_size(int64_t rows, int k, int n, int groups, pmx_dtype dtype,
                                              size_t* bytes) {
  if (!bytes || !dtype_ok(dtype) || !grouped_shape_ok(rows, k, n, groups)) return PMX_ERR_INVALID_VALUE;
  if (!grouped_items_ok(rows, n, groups)) return PMX_ERR_NOT_SUPPORTED;
  *bytes = product_ws(rows, k, n, groups, dtype);
  return PMX_OK;
}

pmx_status pmx_grouped_product(pmx_handle h, const void* A, pmx_dtype dtype, int64_t rows, int k, int64_t lda,
                               const void* B, int n, int64_t ldb, int64_t stride_b, int trans_b,
                               const void* offsets, pmx_itype itype, int groups, void* C,
                               pmx_dtype out_dtype, int64_t ldc, void* ws, size_t ws_bytes, void* stream) {
  if (!h || !dtype_ok(dtype) || !dtype_ok(out_dtype) || !itype_ok(itype) ||
      !grouped_shape_ok(rows, k, n, groups) || (trans_b != 0 && trans_b != 1))
    return PMX_ERR_INVALID_VALUE;
  if (dtype == PMX_F32 && out_dtype != PMX_F32) return PMX_ERR_NOT_SUPPORTED;
  const size_t es = elem_size(dtype), os = elem_size(out_dtype);
  const int br = trans_b ? n : k, bc = trans_b ? k : n;
  if (!layout_ok(A, rows, k, lda, es) || !layout_ok(B, br, bc, ldb, es) || !layout_ok(C, rows, n, ldc, os))
    return PMX_ERR_INVALID_VALUE;
  if (stride_b < 0 || stride_b > kMaxLd || (groups > 1 && stride_b > 0 && stride_b < (int64_t)(br - 1) * ldb + bc))
    return PMX_ERR_INVALID_VALUE;
  if (!offsets || (uintptr_t)offsets % index_size(itype) != 0) return PMX_ERR_INVALID_VALUE;
  if (!grouped_items_ok(rows, n, groups) || lda > kMaxGroupedLd || ldb > kMaxGroupedLd) return PMX_ERR_NOT_SUPPORTED;
  const Extent out = extent(C, rows, n, ldc, os);
  const size_t need = product_ws(rows, k, n, groups, dtype);
  const Extent in[] = {extent(A, rows, k, lda, es), extent_batch(B, groups, stride_b, br, bc, ldb, es),
                       extent(offsets, 1, groups + 1, groups + 1, index_size(itype)),
                       extent(ws, 1, (int64_t)need, (int64_t)need, 1)};
  if (any_overlap(out, in)) return PMX_ERR_ALIAS;
  if (workspace_bad(ws, ws_bytes, need)) return PMX_ERR_WORKSPACE;
  if (need && (overlap(in[3], in[0]) || overlap(in[3], in[1]) || overlap(in[3], in[2]))) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  GroupedParams p = {};
  p.a = A;
  p.lda = lda;
  p.b = B;
  p.ldb = ldb;
  p.stride_b = stride_b;
  p.c = C;
  p.ldc = ldc;
  p.offsets = offsets;
  p.off64 = itype == PMX_I64;
  p.groups = groups;
  p.rows = rows;
  p.n = n;
  p.k = k;
  p.trans_b = trans_b;
  p.dtype = dtype;
  p.out_dtype = out_dtype;
  p.part = (float*)ws;
  p.splits = grouped_product_splits(rows, k, n, groups, dtype);
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_grouped_product(p, s); });
}

pmx_status pmx_grouped_outer_workspace_size(int64_t rows, int m, int n, int groups, pmx_dtype dtype,
                                            size_t* bytes) {
  if (!bytes || !dtype_ok(dtype) || !grouped_shape_ok(rows, m, n, groups)) return PMX_ERR_INVALID_VALUE;
  if (!grouped_items_ok((int64_t)groups * m, n, groups)) return PMX_ERR_NOT_SUPPORTED;
  *bytes = outer_ws(rows, m, n, groups, dtype);
  return PMX_OK;
}

pmx_status pmx_grouped_outer(pmx_handle h, const void* A, pmx_dtype dtype, int64_t rows, int m, int64_t lda,
                             const void* B, int n, int64_t ldb, const void* offsets, pmx_itype itype,
                             int groups, void* C, pmx_dtype out_dtype, int64_t ldc, int64_t stride_c,
                             int accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (!h || !dtype_ok(dtype) || !dtype_ok(out_dtype) || !itype_ok(itype) ||
      !grouped_shape_ok(rows, m, n, groups) || (accumulate != 0 && accumulate != 1))
    return PMX_ERR_INVALID_VALUE;
  if (dtype == PMX_F32 && out_dtype != PMX_F32) return PMX_ERR_NOT_SUPPORTED;
  const size_t es = elem_size(dtype), os = elem_size(out_dtype);
  if (!layout_ok(A, rows, m, lda, es) || !layout_ok(B, rows, n, ldb, es) || !layout_ok(C, m, n, ldc, os))
    return PMX_ERR_INVALID_VALUE;
  if (stride_c < 0 || stride_c > kMaxLd || (groups > 1 && stride_c < (int64_t)(m - 1) * ldc + n))
    return PMX_ERR_INVALID_VALUE;
  if (!offsets || (uintptr_t)offsets % index_size(itype) != 0) return PMX_ERR_INVALID_VALUE;
  if (!grouped_items_ok((int64_t)groups * m, n, groups) || lda > kMaxGroupedLd || ldb > kMaxGroupedLd)
    return PMX_ERR_NOT_SUPPORTED;
  const Extent out = extent_batch(C, groups, stride_c, m, n, ldc, os);
  const size_t need = outer_ws(rows, m, n, groups, dtype);
  const Extent in[] = {extent(A, rows, m, lda, es), extent(B, rows, n, ldb, es),
                       extent(offsets, 1, groups + 1, groups + 1, index_size(itype)),
                       extent(ws, 1, (int64_t)need, (int64_t)need, 1)};
  if (any_overlap(out, in)) return PMX_ERR_ALIAS;
  if (workspace_bad(ws, ws_bytes, need)) return PMX_ERR_WORKSPACE;
  if (need && (overlap(in[3], in[0]) || overlap(in[3], in[1]) || overlap(in[3], in[2]))) return PMX_ERR_ALIAS;
  GroupedParams p = {};
  p.a = A;
  p.lda = lda;
  p.b = B;
  p.ldb = ldb;
  p.c = C;
  p.ldc = ldc;
  p.stride_c = stride_c;
  p.offsets = offsets;
  p.off64 = itype == PMX_I64;
  p.groups = groups;
  p.rows = rows;
  p.m = m;
  p.n = n;
  p.accumulate = accumulate;
  p.dtype = dtype;
  p.out_dtype = out_dtype;
  p.part = (float*)ws;
  p.splits = grouped_outer_splits(rows, m, n, groups, dtype);
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_grouped_outer(p, s); });
}

// ------------------------------------------------------------ embedding
pmx_status pmx_embedding(pmx_handle h, const void* table, pmx_dtype dtype, int vocab, int dim, int64_t ldt,
                         const void* ids, pmx_itype itype, int64_t tokens, float scale, void* Y, int64_t ldy,
                         void* stream) {
  if (!h || !dtype_ok(dtype) || !itype_ok(itype) || vocab < 1 || vocab > PMX_MAX_VOCAB || dim < 1 ||
      dim > kMaxSide || tokens < 0 || tokens > kMaxRows)
    return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype);
  if (!layout_ok(table, vocab, dim, ldt, es) || !layout_ok(Y, tokens, dim, ldy, es)) return PMX_ERR_INVALID_VALUE;
  if (tokens > 0 && (!ids || (uintptr_t)ids % index_size(itype) != 0)) return PMX_ERR_INVALID_VALUE;
  const Extent in[] = {extent(table, vocab, dim, ldt, es), extent(ids, 1, tokens, tokens, index_size(itype))};
  if (any_overlap(extent(Y, tokens, dim, ldy, es), in)) return PMX_ERR_ALIAS;
  if (tokens == 0) return PMX_OK;
  EmbedParams p = {};
  p.table = table;
  p.ld_table = ldt;
  p.ids = ids;
  p.ids64 = itype == PMX_I64;
  p.tokens = tokens;
  p.vocab = vocab;
  p.dim = dim;
  p.scale = scale;
  p.dtype = p.out_dtype = dtype;
  p.out = Y;
  p.ld_out = ldy;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_embed_lookup(p, s); });
}

pmx_status pmx_embedding_grad_workspace_size(int64_t tokens, int vocab, int dim, size_t* bytes) {
  if (!bytes || tokens < 0 || tokens > PMX_MAX_TOKENS || vocab < 1 || vocab > PMX_MAX_VOCAB || dim < 1 ||
      dim > kMaxSide)
    return PMX_ERR_INVALID_VALUE;
  *bytes = embed_grad_workspace(tokens, vocab, dim);
  return PMX_OK;
}

pmx_status pmx_embedding_grad(pmx_handle h, const void* dY, pmx_dtype dtype, int64_t tokens, int dim,
                              int64_t lddy, const void* ids, pmx_itype itype, int vocab, float scale,
                              int64_t padding_idx, void* dW, pmx_dtype out_dtype, int64_t lddw,
                              int accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (!h || !dtype_ok(dtype) || !dtype_ok(out_dtype) || !itype_ok(itype) || vocab < 1 ||
      vocab > PMX_MAX_VOCAB || dim < 1 || dim > kMaxSide || tokens < 0 || tokens > PMX_MAX_TOKENS ||
      (accumulate != 0 && accumulate != 1))
    return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype), os = elem_size(out_dtype);
  if (!layout_ok(dY, tokens, dim, lddy, es) || !layout_ok(dW, vocab, dim, lddw, os)) return PMX_ERR_INVALID_VALUE;
  if (tokens > 0 && (!ids || (uintptr_t)ids % index_size(itype) != 0)) return PMX_ERR_INVALID_VALUE;
  const size_t need = embed_grad_workspace(tokens, vocab, dim);
  const Extent out = extent(dW, vocab, dim, lddw, os);
  const Extent in[] = {extent(dY, tokens, dim, lddy, es), extent(ids, 1, tokens, tokens, index_size(itype)),
                       extent(ws, 1, (int64_t)need, (int64_t)need, 1)};
  if (any_overlap(out, in)) return PMX_ERR_ALIAS;
  if (workspace_bad(ws, ws_bytes, need)) return PMX_ERR_WORKSPACE;
  if (overlap(in[2], in[0]) || overlap(in[2], in[1])) return PMX_ERR_ALIAS;
  EmbedParams p = {};
  p.ids = ids;
  p.ids64 = itype == PMX_I64;
  p.tokens = tokens;
  p.vocab = vocab;
  p.dim = dim;
  p.scale = scale;
  p.dtype = dtype;
  p.out_dtype = out_dtype;
  p.out = dW;
  p.ld_out = lddw;
  p.dy = dY;
  p.ld_dy = lddy;
  p.padding_idx = padding_idx;
  p.accumulate = accumulate;
  p.ws = ws;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_embed_grad(p, s); });
}

// ------------------------------------------------------------ distillation
pmx_status pmx_distill_workspace_size(const pmx_distill_problem* q, size_t* bytes) {
  if (!bytes || !distill_shape_ok(q)) return PMX_ERR_INVALID_VALUE;
  *bytes = (size_t)distill_part_floats(q->rows, q->vocab, q->top, q->dtype) * sizeof(float);
  return PMX_OK;
}

pmx_status pmx_distill_loss(pmx_handle h, const pmx_distill_problem* q, float* rows_loss, float* total,
                            float* stats, void* dZ, int64_t lddz, void* ws, size_t ws_bytes, void* stream) {
  if (!h || !distill_ok(q) || !total || (uintptr_t)total % 4 || (uintptr_t)rows_loss % 4 || (uintptr_t)stats % 4)
    return PMX_ERR_INVALID_VALUE;
  if (q->rows > 0 && !rows_loss) return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(q->dtype);
  if (dZ && !layout_ok(dZ, q->rows, q->vocab, lddz, es)) return PMX_ERR_INVALID_VALUE;
  if (dZ && dz_aliases(q, dZ, lddz)) return PMX_ERR_ALIAS;
  const size_t need = (size_t)distill_part_floats(q->rows, q->vocab, q->top, q->dtype) * sizeof(float);
  const Extent outs[] = {extent(rows_loss, 1, q->rows, q->rows, 4), extent(total, 1, 1, 1, 4),
                         extent(stats, q->rows, 3, 3, 4), extent(ws, 1, (int64_t)need, (int64_t)need, 1)};
  const Extent in[] = {extent(q->z, q->rows, q->vocab, q->ldz, es),
                       extent(q->teacher_ids, q->rows, q->top, q->ld_ids, index_size(q->ids_type)),
                       extent(q->teacher, q->rows, q->top, q->ld_teacher, elem_size(q->teacher_dtype)),
                       extent(q->labels, 1, q->rows, q->rows, index_size(q->labels_type)),
                       extent(q->weights, 1, q->rows, q->rows, 4),
                       extent(dZ, q->rows, q->vocab, lddz, es)};
  for (int i = 0; i < 4; ++i) {
    if (any_overlap(outs[i], in)) return PMX_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return PMX_ERR_ALIAS;
  }
  if (workspace_bad(ws, ws_bytes, need)) return PMX_ERR_WORKSPACE;
  DistillParams p = distill_params(q, h);
  p.rows_loss = rows_loss;
  p.total = total;
  p.stats = stats;
  p.dz = dZ;
  p.lddz = lddz;
  p.part = (float*)ws;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_distill_loss(p, s); });
}

pmx_status pmx_distill_grad(pmx_handle h, const pmx_distill_problem* q, const float* stats,
                            const float* upstream, void* dZ, int64_t lddz, void* stream) {
  if (!h || !distill_ok(q) || (uintptr_t)stats % 4 || (uintptr_t)upstream % 4) return PMX_ERR_INVALID_VALUE;
  if (q->rows > 0 && (!stats || !dZ)) return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(q->dtype);
  if (!layout_ok(dZ, q->rows, q->vocab, lddz, es)) return PMX_ERR_INVALID_VALUE;
  if (dz_aliases(q, dZ, lddz)) return PMX_ERR_ALIAS;
  const Extent in[] = {extent(stats, q->rows, 3, 3, 4), extent(upstream, 1, 1, 1, 4)};
  if (any_overlap(extent(dZ, q->rows, q->vocab, lddz, es), in)) return PMX_ERR_ALIAS;
  if (q->rows == 0) return PMX_OK;
  DistillParams p = distill_params(q, h);
  p.stats = const_cast<float*>(stats);
  p.upstream = upstream;
  p.dz = dZ;
  p.lddz = lddz;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_distill_grad(p, s); });
}

}  // extern "C"
