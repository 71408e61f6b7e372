// Argument checks shared by the C entries of the training step's operators.
#pragma once

#include "pmx_host.h"

namespace pmx {
namespace {

bool dtype_ok(pmx_dtype t) { return t == PMX_F32 || t == PMX_BF16; }
bool itype_ok(pmx_itype t) { return t == PMX_I32 || t == PMX_I64; }
size_t elem_size(pmx_dtype t) { return t == PMX_F32 ? 4 : 2; }
size_t index_size(pmx_itype t) { return t == PMX_I32 ? 4 : 8; }

constexpr int64_t kMaxRows = 0x7fffffff;
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int kMaxSide = 1 << 20;  // k, m, n of the grouped products, columns
constexpr int64_t kMaxGroupedLd = (int64_t)1 << 22;  // offsets inside a tile are 32-bit

// rows x cols with row distance ld >= cols; 0 rows: nothing.
bool layout_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  if (ld < cols || ld > kMaxLd) return false;
  if (rows == 0) return true;
  return p && (uintptr_t)p % elem == 0;
}
Extent extent(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
  Extent e;
  if (!p || rows <= 0 || cols <= 0) return e;
  e.lo = (uintptr_t)p;
  e.hi = e.lo + (uintptr_t)((rows - 1) * ld + cols) * elem;
  e.valid = true;
  return e;
}
Extent extent_batch(const void* p, int64_t batch, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                    size_t elem) {
  Extent e = extent(p, rows, cols, ld, elem);
  if (e.valid) e.hi += (uintptr_t)((batch - 1) * stride) * elem;
  return e;
}

template <size_t N>
bool any_overlap(const Extent& out, const Extent (&in)[N]) {
  for (const Extent& e : in)
    if (overlap(out, e)) return true;
  return false;
}

// Runs `f` on the handle's device and stream; no exception leaves the C ABI.
template <typename F>
pmx_status enqueue(pmx_handle h, void* stream, F&& f) {
  try {
    DeviceGuard dg(h->device);
    if (!dg.ok) return PMX_ERR_HIP;
    Enq q{h, (hipStream_t)stream};
    return from_hip(q.run(PMX_KC_OTHER, [&] { return f(q.s); }));
  } catch (...) {
    return PMX_ERR_HIP;
  }
}

bool workspace_bad(const void* ws, size_t have, size_t need) {
  return need > 0 && (!ws || have < need || (uintptr_t)ws % 256 != 0);
}

}  // namespace
}  // namespace pmx
