// C ABI of the expert layer's operators (include/pmx.h): argument checks and
// launches of the layer norm, the router, the 8-bit checkpoints and products.
// Nothing is enqueued unless every check has passed.
#include <math.h>

#include "pmx_checks.h"
#include "pmx_layer.h"

namespace pmx {
namespace {

int64_t up128(int64_t n) { return (n + kBlock8 - 1) / kBlock8 * kBlock8; }

bool norm_shape_ok(int64_t rows, int cols) {
  return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= PMX_MAX_NORM_COLS;
}
bool vector_ok(const void* p, size_t elem) { return (uintptr_t)p % elem == 0; }

bool route_shape_ok(const pmx_route_problem* q) {
  return q && q->struct_version == 1 && q->reserved == 0 && dtype_ok(q->dtype) && q->rows >= 0 &&
         q->rows <= PMX_MAX_ROUTE_ROWS && q->experts >= 1 && q->experts <= PMX_MAX_GROUPS && q->top >= 1 &&
         q->top <= PMX_MAX_ROUTE_TOP && q->top <= q->experts && q->rows * q->top <= kMaxRows;
}
bool route_ok(const pmx_route_problem* q) {
  return route_shape_ok(q) && isfinite(q->balance) && isfinite(q->zloss) && (q->normalize == 0 || q->normalize == 1) &&
         layout_ok(q->z, q->rows, q->experts, q->ldz, elem_size(q->dtype));
}
RouteParams route_params(const pmx_route_problem* q, const pmx_context* h) {
  RouteParams p = {};
  p.z = q->z;
  p.ldz = q->ldz;
  p.dtype = q->dtype;
  p.rows = q->rows;
  p.experts = q->experts;
  p.top = q->top;
  p.live = q->live;
  p.normalize = q->normalize;
  p.balance = q->balance;
  p.zloss = q->zloss;
  p.num_cu = h->num_cu;
  return p;
}

// 8-bit values of `halves` padded halves of `cols`, and their scales
bool values_ok(const uint8_t* v, int64_t ldv, const uint8_t* s, int64_t lds, int64_t rows, int64_t cols, int halves) {
  const int64_t wide = halves * up128(cols);
  if (ldv < wide || ldv > kMaxLd || ldv % 16 != 0 || lds < wide / kBlock8 || lds > kMaxLd) return false;
  return rows == 0 || (v && s && (uintptr_t)v % 16 == 0);
}
Extent values_extent(const uint8_t* v, int64_t ldv, int64_t rows, int64_t cols, int halves) {
  return extent(v, rows, halves * up128(cols), ldv, 1);
}
Extent scales_extent(const uint8_t* s, int64_t lds, int64_t rows, int64_t cols, int halves) {
  return extent(s, rows, halves * up128(cols) / kBlock8, lds, 1);
}
bool shape8_ok(int64_t rows, int cols) { return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= kMaxSide; }

// Some two of the extents overlap, the first `outs` of which are outputs.
template <size_t N>
bool clash(const Extent (&e)[N], size_t outs) {
  for (size_t i = 0; i < outs; ++i)
    for (size_t j = i + 1; j < N; ++j)
      if (overlap(e[i], e[j])) return true;
  return false;
}

}  // namespace
}  // namespace pmx

using namespace pmx;

extern "C" {

// ------------------------------------------------------------ layer norm
pmx_status pmx_layer_norm(pmx_handle h, const void* X, pmx_dtype dtype, int64_t rows, int cols, int64_t ldx,
                          const void* weight, const void* bias, pmx_dtype param_dtype, float eps, void* Y,
                          int64_t ldy, float* stats, void* stream) {
  if (!h || !dtype_ok(dtype) || !dtype_ok(param_dtype) || !norm_shape_ok(rows, cols) || !(eps >= 0.f) || !isfinite(eps))
    return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
  if (!layout_ok(X, rows, cols, ldx, es) || !layout_ok(Y, rows, cols, ldy, es) || !vector_ok(weight, ps) ||
      !vector_ok(bias, ps) || !vector_ok(stats, 4))
    return PMX_ERR_INVALID_VALUE;
  const Extent all[] = {extent(Y, rows, cols, ldy, es), extent(stats, rows, 2, 2, 4), extent(X, rows, cols, ldx, es),
                        extent(weight, 1, cols, cols, ps), extent(bias, 1, cols, cols, ps)};
  if (clash(all, 2)) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  NormParams p = {};
  p.x = X;
  p.ldx = ldx;
  p.weight = weight;
  p.bias = bias;
  p.param_dtype = param_dtype;
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.eps = eps;
  p.y = Y;
  p.ldy = ldy;
  p.stats = stats;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_norm(p, s); });
}

pmx_status pmx_layer_norm_grad_workspace_size(int64_t rows, int cols, pmx_dtype dtype, size_t* bytes) {
  if (!bytes || !dtype_ok(dtype) || !norm_shape_ok(rows, cols)) return PMX_ERR_INVALID_VALUE;
  *bytes = norm_grad_floats(rows, cols, dtype) * sizeof(float);
  return PMX_OK;
}

pmx_status pmx_layer_norm_grad(pmx_handle h, const void* dY, pmx_dtype dtype, int64_t rows, int cols, int64_t lddy,
                               const void* X, int64_t ldx, const float* stats, const void* weight,
                               pmx_dtype param_dtype, void* dX, int64_t lddx, float* dweight, float* dbias,
                               int accumulate, void* ws, size_t ws_bytes, void* stream) {
  if (!h || !dtype_ok(dtype) || !dtype_ok(param_dtype) || !norm_shape_ok(rows, cols) ||
      (accumulate != 0 && accumulate != 1))
    return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
  if (!layout_ok(dY, rows, cols, lddy, es) || !layout_ok(X, rows, cols, ldx, es) || !vector_ok(weight, ps) ||
      !vector_ok(stats, 4) || !vector_ok(dweight, 4) || !vector_ok(dbias, 4) || (rows > 0 && !stats))
    return PMX_ERR_INVALID_VALUE;
  if (dX && !layout_ok(dX, rows, cols, lddx, es)) return PMX_ERR_INVALID_VALUE;
  const bool params = dweight || dbias;
  const size_t need = params ? norm_grad_floats(rows, cols, dtype) * sizeof(float) : 0;
  const bool same = dX && dX == dY && lddx == lddy;
  const Extent all[] = {extent(dX, rows, cols, lddx, es),
                        extent(dweight, 1, cols, cols, 4),
                        extent(dbias, 1, cols, cols, 4),
                        extent(ws, 1, (int64_t)need, (int64_t)need, 1),
                        same ? Extent() : extent(dY, rows, cols, lddy, es),
                        extent(X, rows, cols, ldx, es),
                        extent(stats, rows, 2, 2, 4),
                        extent(weight, 1, cols, cols, ps)};
  if (clash(all, 4)) return PMX_ERR_ALIAS;
  if (workspace_bad(ws, ws_bytes, need)) return PMX_ERR_WORKSPACE;
  if (!params && (!dX || rows == 0)) return PMX_OK;
  NormParams p = {};
  p.x = X;
  p.ldx = ldx;
  p.weight = weight;
  p.param_dtype = param_dtype;
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.stats = const_cast<float*>(stats);
  p.dy = dY;
  p.lddy = lddy;
  p.dx = dX;
  p.lddx = lddx;
  p.dw = dweight;
  p.db = dbias;
  p.accumulate = accumulate;
  p.part = (float*)ws;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_norm_grad(p, s); });
}

// ------------------------------------------------------------ router
pmx_status pmx_route_workspace_size(const pmx_route_problem* q, size_t* bytes) {
  if (!bytes || !route_shape_ok(q)) return PMX_ERR_INVALID_VALUE;
  *bytes = route_workspace(q->rows, q->experts);
  return PMX_OK;
}

pmx_status pmx_route(pmx_handle h, const pmx_route_problem* q, int32_t* ids, float* gates, int32_t* counts,
                     int32_t* offsets, int32_t* slots, int32_t* tokens, float* loss, void* ws, size_t ws_bytes,
                     void* stream) {
  if (!h || !route_ok(q) || !counts || !offsets || !loss || !vector_ok(ids, 4) || !vector_ok(gates, 4) ||
      !vector_ok(counts, 4) || !vector_ok(offsets, 4) || !vector_ok(slots, 4) || !vector_ok(tokens, 4) ||
      !vector_ok(loss, 4))
    return PMX_ERR_INVALID_VALUE;
  if (q->rows > 0 && (!ids || !gates || !slots != !tokens)) return PMX_ERR_INVALID_VALUE;
  const size_t need = route_workspace(q->rows, q->experts);
  const int64_t pairs = q->rows * q->top, e1 = q->experts + 1;
  const Extent all[] = {extent(ids, 1, pairs, pairs, 4),
                        extent(gates, 1, pairs, pairs, 4),
                        extent(counts, 1, e1, e1, 4),
                        extent(offsets, 1, e1, e1, 4),
                        extent(slots, 1, pairs, pairs, 4),
                        extent(tokens, 1, pairs, pairs, 4),
                        extent(loss, 1, 1, 1, 4),
                        extent(ws, 1, (int64_t)need, (int64_t)need, 1),
                        extent(q->z, q->rows, q->experts, q->ldz, elem_size(q->dtype)),
                        extent(q->live, 1, q->rows, q->rows, 1)};
  if (clash(all, 8)) return PMX_ERR_ALIAS;
  if (workspace_bad(ws, ws_bytes, need)) return PMX_ERR_WORKSPACE;
  RouteParams p = route_params(q, h);
  p.ids = ids;
  p.gates = gates;
  p.counts = counts;
  p.offsets = offsets;
  p.slots = slots;
  p.tokens = tokens;
  p.loss = loss;
  p.ws = ws;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_route(p, s); });
}

pmx_status pmx_route_grad(pmx_handle h, const pmx_route_problem* q, const int32_t* ids, const float* gates,
                          const int32_t* counts, const float* dgates, const float* upstream, void* dZ, int64_t lddz,
                          void* stream) {
  if (!h || !route_ok(q) || !counts || !vector_ok(ids, 4) || !vector_ok(gates, 4) || !vector_ok(counts, 4) ||
      !vector_ok(dgates, 4) || !vector_ok(upstream, 4))
    return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(q->dtype);
  if (!layout_ok(dZ, q->rows, q->experts, lddz, es) || (q->rows > 0 && dgates && (!ids || !gates)))
    return PMX_ERR_INVALID_VALUE;
  const int64_t pairs = q->rows * q->top, e1 = q->experts + 1;
  const bool same = dZ == q->z && lddz == q->ldz;
  const Extent all[] = {extent(dZ, q->rows, q->experts, lddz, es),
                        same ? Extent() : extent(q->z, q->rows, q->experts, q->ldz, es),
                        extent(q->live, 1, q->rows, q->rows, 1),
                        extent(ids, 1, pairs, pairs, 4),
                        extent(gates, 1, pairs, pairs, 4),
                        extent(counts, 1, e1, e1, 4),
                        extent(dgates, 1, pairs, pairs, 4),
                        extent(upstream, 1, 1, 1, 4)};
  if (clash(all, 1)) return PMX_ERR_ALIAS;
  if (q->rows == 0) return PMX_OK;
  RouteParams p = route_params(q, h);
  p.ids = const_cast<int32_t*>(ids);
  p.gates = const_cast<float*>(gates);
  p.counts = const_cast<int32_t*>(counts);
  p.dgates = dgates;
  p.upstream = upstream;
  p.dz = dZ;
  p.lddz = lddz;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_route_grad(p, s); });
}

// ------------------------------------------------------------ values in 8 bits
pmx_status pmx_fp8_store(pmx_handle h, const void* X, pmx_dtype dtype, int64_t rows, int cols, int64_t ldx,
                         uint8_t* values, int64_t ldv, uint8_t* scales, int64_t lds, void* stream) {
  if (!h || !dtype_ok(dtype) || !shape8_ok(rows, cols)) return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype);
  if (!layout_ok(X, rows, cols, ldx, es) || !values_ok(values, ldv, scales, lds, rows, cols, 1))
    return PMX_ERR_INVALID_VALUE;
  const Extent all[] = {values_extent(values, ldv, rows, cols, 1), scales_extent(scales, lds, rows, cols, 1),
                        extent(X, rows, cols, ldx, es)};
  if (clash(all, 2)) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  Store8Params p = {};
  p.x = X;
  p.ldx = ldx;
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.values = values;
  p.ldv = ldv;
  p.scales = scales;
  p.lds = lds;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_store8(p, s); });
}

pmx_status pmx_fp8_load(pmx_handle h, const uint8_t* values, int64_t ldv, const uint8_t* scales, int64_t lds,
                        int64_t rows, int cols, void* Y, pmx_dtype dtype, int64_t ldy, void* stream) {
  if (!h || !dtype_ok(dtype) || !shape8_ok(rows, cols)) return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype);
  if (!layout_ok(Y, rows, cols, ldy, es) || !values_ok(values, ldv, scales, lds, rows, cols, 1))
    return PMX_ERR_INVALID_VALUE;
  const Extent all[] = {extent(Y, rows, cols, ldy, es), values_extent(values, ldv, rows, cols, 1),
                        scales_extent(scales, lds, rows, cols, 1)};
  if (clash(all, 1)) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  Store8Params p = {};
  p.act = Y;
  p.lda = ldy;
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.values = const_cast<uint8_t*>(values);
  p.ldv = ldv;
  p.scales = const_cast<uint8_t*>(scales);
  p.lds = lds;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_load8(p, s); });
}

pmx_status pmx_fp8_store_weight(pmx_handle h, const void* W, pmx_dtype dtype, int groups, int n, int k, int64_t ldw,
                                int64_t stride_w, int transposed, uint8_t* values, int64_t ldv, int64_t stride_v,
                                uint8_t* scales, int64_t lds, int64_t stride_s, void* stream) {
  if (!h || !dtype_ok(dtype) || groups < 1 || groups > PMX_MAX_GROUPS || n < 1 || n > kMaxSide || k < 1 ||
      k > kMaxSide || (transposed != 0 && transposed != 1))
    return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype);
  const int vr = transposed ? k : n, vc = transposed ? n : k, sr = (vr + 127) / 128;
  if (!layout_ok(W, n, k, ldw, es) || !values_ok(values, ldv, scales, lds, vr, vc, 1)) return PMX_ERR_INVALID_VALUE;
  if (stride_w < 0 || stride_w > kMaxLd || stride_v < 0 || stride_v > kMaxLd || stride_v % 16 != 0 || stride_s < 0 ||
      stride_s > kMaxLd)
    return PMX_ERR_INVALID_VALUE;
  if (groups > 1 && (stride_v < (int64_t)(vr - 1) * ldv + up128(vc) || stride_s < (int64_t)(sr - 1) * lds + up128(vc) / kBlock8 ||
                     (stride_w > 0 && stride_w < (int64_t)(n - 1) * ldw + k)))
    return PMX_ERR_INVALID_VALUE;
  const int64_t tiles = (int64_t)((n + 127) / 128) * ((k + 127) / 128) * groups;
  if (tiles > ((int64_t)1 << 23)) return PMX_ERR_NOT_SUPPORTED;  // blocks of one launch
  const Extent all[] = {extent_batch(values, groups, stride_v, vr, up128(vc), ldv, 1),
                        extent_batch(scales, groups, stride_s, sr, up128(vc) / kBlock8, lds, 1),
                        extent_batch(W, groups, stride_w, n, k, ldw, es)};
  if (clash(all, 2)) return PMX_ERR_ALIAS;
  Store8Params p = {};
  p.x = W;
  p.ldx = ldw;
  p.dtype = dtype;
  p.rows = n;
  p.cols = k;
  p.values = values;
  p.ldv = ldv;
  p.scales = scales;
  p.lds = lds;
  p.batch = groups;
  p.stride_x = stride_w;
  p.stride_v = stride_v;
  p.stride_s = stride_s;
  p.transposed = transposed;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_store8_weight(p, s); });
}

pmx_status pmx_silu_checkpoint(pmx_handle h, const void* H, pmx_dtype dtype, int64_t rows, int cols, int64_t ldh,
                               int gated, void* A, int64_t lda, uint8_t* values, int64_t ldv, uint8_t* scales,
                               int64_t lds, void* stream) {
  if (!h || !dtype_ok(dtype) || !shape8_ok(rows, cols) || (gated != 0 && gated != 1)) return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype);
  const int halves = 1 + gated;
  if (!layout_ok(H, rows, (int64_t)halves * cols, ldh, es) || !layout_ok(A, rows, cols, lda, es) ||
      !values_ok(values, ldv, scales, lds, rows, cols, halves))
    return PMX_ERR_INVALID_VALUE;
  const Extent all[] = {extent(A, rows, cols, lda, es), values_extent(values, ldv, rows, cols, halves),
                        scales_extent(scales, lds, rows, cols, halves), extent(H, rows, (int64_t)halves * cols, ldh, es)};
  if (clash(all, 3)) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  Store8Params p = {};
  p.x = H;
  p.ldx = ldh;
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.gated = gated;
  p.act = A;
  p.lda = lda;
  p.values = values;
  p.ldv = ldv;
  p.scales = scales;
  p.lds = lds;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_silu8(p, s); });
}

pmx_status pmx_silu_checkpoint_grad(pmx_handle h, const void* dA, pmx_dtype dtype, int64_t rows, int cols, int64_t ldda,
                                    const uint8_t* values, int64_t ldv, const uint8_t* scales, int64_t lds, int gated,
                                    void* dH, int64_t lddh, void* A, int64_t lda, void* stream) {
  if (!h || !dtype_ok(dtype) || !shape8_ok(rows, cols) || (gated != 0 && gated != 1)) return PMX_ERR_INVALID_VALUE;
  const size_t es = elem_size(dtype);
  const int halves = 1 + gated;
  if (!layout_ok(dA, rows, cols, ldda, es) || !layout_ok(dH, rows, (int64_t)halves * cols, lddh, es) ||
      (A && !layout_ok(A, rows, cols, lda, es)) || !values_ok(values, ldv, scales, lds, rows, cols, halves))
    return PMX_ERR_INVALID_VALUE;
  const Extent all[] = {extent(dH, rows, (int64_t)halves * cols, lddh, es), extent(A, rows, cols, lda, es),
                        extent(dA, rows, cols, ldda, es), values_extent(values, ldv, rows, cols, halves),
                        scales_extent(scales, lds, rows, cols, halves)};
  if (clash(all, 2)) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  Store8Params p = {};
  p.dtype = dtype;
  p.rows = rows;
  p.cols = cols;
  p.gated = gated;
  p.dact = dA;
  p.ldda = ldda;
  p.dx = dH;
  p.lddx = lddh;
  p.act = A;
  p.lda = lda;
  p.values = const_cast<uint8_t*>(values);
  p.ldv = ldv;
  p.scales = const_cast<uint8_t*>(scales);
  p.lds = lds;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_silu8_grad(p, s); });
}

// ------------------------------------------------------------ products in 8 bits
namespace {
bool fp8_shape_ok(int64_t rows, int k, int n, int groups) {
  return rows >= 0 && rows <= kMaxRows && k >= 1 && k <= kMaxSide && n >= 1 && n <= kMaxSide && groups >= 1 &&
         groups <= PMX_MAX_GROUPS;
}
// tile counts are 32-bit on the device
bool fp8_items_ok(int64_t rows, int n, int groups) {
  return (rows / 16 + groups) * (int64_t)((n + 63) / 64) * 64 <= kMaxRows;
}
}  // namespace

pmx_status pmx_fp8_product(pmx_handle h, const uint8_t* A, int64_t rows, int k, int64_t lda, const uint8_t* A_scales,
                           int64_t ldas, const uint8_t* B, int n, int64_t ldb, int64_t stride_b,
                           const uint8_t* B_scales, int64_t ldbs, int64_t stride_bs, const void* offsets,
                           pmx_itype itype, int groups, void* C, pmx_dtype out_dtype, int64_t ldc, void* stream) {
  if (!h || !dtype_ok(out_dtype) || !itype_ok(itype) || !fp8_shape_ok(rows, k, n, groups)) return PMX_ERR_INVALID_VALUE;
  const size_t os = elem_size(out_dtype);
  const int64_t kp = up128(k);
  const int sn = (n + 127) / 128;
  if (!values_ok(A, lda, A_scales, ldas, rows, k, 1) || !values_ok(B, ldb, B_scales, ldbs, n, k, 1) ||
      !layout_ok(C, rows, n, ldc, os))
    return PMX_ERR_INVALID_VALUE;
  if (stride_b < 0 || stride_b > kMaxLd || stride_b % 16 != 0 || stride_bs < 0 || stride_bs > kMaxLd)
    return PMX_ERR_INVALID_VALUE;
  if (groups > 1 && ((stride_b > 0 && stride_b < (int64_t)(n - 1) * ldb + kp) ||
                     (stride_bs > 0 && stride_bs < (int64_t)(sn - 1) * ldbs + kp / kBlock8)))
    return PMX_ERR_INVALID_VALUE;
  if ((!offsets && groups > 1) || !vector_ok(offsets, index_size(itype))) return PMX_ERR_INVALID_VALUE;
  if (!fp8_items_ok(rows, n, groups) || lda > kMaxGroupedLd || ldb > kMaxGroupedLd || ldas > kMaxGroupedLd ||
      ldbs > kMaxGroupedLd)
    return PMX_ERR_NOT_SUPPORTED;
  const Extent all[] = {extent(C, rows, n, ldc, os),
                        values_extent(A, lda, rows, k, 1),
                        scales_extent(A_scales, ldas, rows, k, 1),
                        extent_batch(B, groups, stride_b, n, kp, ldb, 1),
                        extent_batch(B_scales, groups, stride_bs, sn, kp / kBlock8, ldbs, 1),
                        extent(offsets, 1, groups + 1, groups + 1, index_size(itype))};
  if (clash(all, 1)) return PMX_ERR_ALIAS;
  if (rows == 0) return PMX_OK;
  Fp8Params p = {};
  p.a = A;
  p.lda = lda;
  p.sa = A_scales;
  p.ldsa = ldas;
  p.b = B;
  p.ldb = ldb;
  p.stride_b = stride_b;
  p.sb = B_scales;
  p.ldsb = ldbs;
  p.stride_sb = stride_bs;
  p.offsets = offsets;
  p.off64 = itype == PMX_I64;
  p.groups = groups;
  p.rows = rows;
  p.n = n;
  p.k = (int)kp;
  p.c = C;
  p.ldc = ldc;
  p.out_dtype = out_dtype;
  p.num_cu = h->num_cu;
  return enqueue(h, stream, [&](hipStream_t s) { return launch_fp8(p, s); });
}

}  // extern "C"
