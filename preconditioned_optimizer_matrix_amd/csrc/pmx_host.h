// Host-side helpers shared by the translation units that carry the C ABI:
// the handle, the device guard, extents and overlap, traced enqueueing.
#pragma once

#include <stddef.h>

#include <vector>

#include "pmx_internal.h"

struct pmx_context {
  int device;
  int num_cu;
  int gemm_blocks_per_cu;  // persistent GEMM grid: blocks per CU (0: one block per tile)
  int gemm_cfg;            // forced tile configuration (-1: by shape)
  int gemm_map;            // tile order mode
  int bf16_cfg;            // bf16 GEMM tile (-1: by shape, 0 128^2, 1 256^2 x 8 waves, 2 x 4)
  int bf16_map;            // bf16 GEMM: 1 deals whole matrices to XCDs, 0 plain order
  int skinny_variant;      // skinny products: 0 In through LDS, 1 In read directly
  int bf16_dma;            // bf16 GEMM: 1 uses direct global-to-LDS loads for whole tiles (measured slower; off)
  int bf16_mn;             // bf16 polar: 1 reads X for I - X^T X via LDS transpose reads (no X^T copy)
  int bf16_persist;        // bf16 GEMM: 1 runs whole-tile launches on persistent blocks, each
                           // loading its next tile's first k tile ahead of the epilogue
  int bf16_early;          // bf16 persistent GEMM: 1 issues each k tile's loads before the previous tile's barrier
  int small_fused;         // 1: one fused launch for orders <= kSmallMaxN
  int split_k;             // 1: split-k tail for the fp32 products of the iterations
  int bf16_sym;            // 1: bf16 X^T X and R^2 run upper-triangle tiles, mirrored
  int bf16_sym_small;      // 1: ... with 128 x 128 tiles
  int f64_tile;            // fp64 GEMM block tile (0: by the launch's size, else 64 or 128)
  // host-polled convergence (pmx_set_host_poll): updates per published point,
  // two pinned host flags (device-mapped) and the events behind them
  int poll_chunk = 0;
  int32_t* poll_host = nullptr;
  int32_t* poll_dev = nullptr;
  hipEvent_t poll_ev[2] = {nullptr, nullptr};
  // launch trace (benchmarking): event pairs recorded around every launch
  bool trace = false;
  struct Rec {
    int cls;
    hipEvent_t a, b;
  };
  std::vector<Rec> recs;
  std::vector<hipEvent_t> pool;
  size_t used = 0;
  hipEvent_t next_event() {
    if (used == pool.size()) {
      hipEvent_t e = nullptr;
      if (hipEventCreate(&e) != hipSuccess) return nullptr;
      pool.push_back(e);
    }
    return pool[used++];
  }
};

namespace pmx {

// Current-device guard: make the handle's device current for the call and
// restore the caller's device afterwards.
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) {
      ok = false;
      return;
    }
    if (prev != dev && hipSetDevice(dev) != hipSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

// Byte extent of a (strided batch of) row-major matrices.
struct Extent {
  uintptr_t lo = 0, hi = 0;
  bool valid = false;
};

inline Extent extent_of(const void* p, int rows, int cols, int64_t ld, int64_t stride, int batch,
                 size_t elem) {
  Extent e;
  if (!p || rows <= 0 || cols <= 0) return e;
  const int64_t last = (int64_t)(batch - 1) * stride + (int64_t)(rows - 1) * ld + cols;
  e.lo = (uintptr_t)p;
  e.hi = e.lo + (uintptr_t)last * elem;
  e.valid = true;
  return e;
}

inline bool overlap(const Extent& a, const Extent& b) {
  return a.valid && b.valid && a.lo < b.hi && b.lo < a.hi;
}

// Distinct matrices of one batch must not overlap when written.
inline bool batch_layout_ok(int rows, int cols, int64_t ld, int64_t stride, int batch) {
  if (ld < cols) return false;
  if (batch > 1 && stride < (int64_t)(rows - 1) * ld + cols) return false;
  return stride >= 0;
}

inline pmx_status from_hip(hipError_t e) { return e == hipSuccess ? PMX_OK : PMX_ERR_HIP; }

// Enqueue helper: runs a launcher on the call's stream, bracketed by trace
// events when the handle's trace is enabled.
struct Enq {
  pmx_context* h;
  hipStream_t s;
  template <typename F>
  hipError_t run(int cls, F&& f) {
    hipEvent_t a = nullptr, b = nullptr;
    if (h && h->trace) {
      a = h->next_event();
      b = h->next_event();
      if (a && b) (void)hipEventRecord(a, s);
    }
    const hipError_t e = f();
    if (a && b) {
      (void)hipEventRecord(b, s);
      h->recs.push_back({cls, a, b});
    }
    return e;
  }
};

}  // namespace pmx

#define PMX_TRY(expr)                          \
  do {                                         \
    hipError_t _e = (expr);                    \
    if (_e != hipSuccess) return PMX_ERR_HIP;  \
  } while (0)
