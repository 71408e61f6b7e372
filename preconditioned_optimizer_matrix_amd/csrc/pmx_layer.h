// Parameter blocks and launchers of the expert layer's operators: layer norm
// (pmx_norm.hip), the router with its balance loss (pmx_route.hip), values kept
// in 8 bits (pmx_checkpoint.hip) and products of them (pmx_fp8.hip); reductions
// and row pieces they share.
#pragma once

#include "pmx_train.h"

namespace pmx {

// ---------------------------------------------------------------------------
// Reductions over 16 lanes (a DPP row) and over a wave; every lane gets the result.  All lanes
// are active (one that is not would count as 0), so an exchange is one instruction with its sum.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;  // quad_perm, row_half_mirror, row_mirror

__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  return v + dpp<kMirror>(v);
}
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kXor1>(v));
  v = fmaxf(v, dpp<kXor2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  return fmaxf(v, dpp<kMirror>(v));
}
template <int CTRL>
__device__ __forceinline__ int dpp(int i) {
  return __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  // rows 0 and 1, 2 and 3, then the halves change places
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
__device__ __forceinline__ float wave_max(float v) {
  v = row_max(v);
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147180559945309f;
// exp(x) for x <= 0, 0 for -inf and NaN: the product's rounding error goes back in as a
// factor.
__device__ __forceinline__ float exp_acc(float x) {
  x = fmaxf(x, -200.f);
  const float y = x * kLog2e;
  const float r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -y));
  const float e = __builtin_amdgcn_exp2f(y);
  return fmaf(e, r * kLn2, e);
}

// ---------------------------------------------------------------------------
// Pieces of 16 bytes of a row of n elements, at any element alignment.
typedef u32x4_t piece_a2 __attribute__((aligned(2)));
typedef u32x4_t piece_a4 __attribute__((aligned(4)));
template <size_t A>
struct Parts;
template <>
struct Parts<2> {
  typedef u32x2_t half __attribute__((aligned(2)));
  typedef uint32_t word __attribute__((aligned(2)));
};
template <>
struct Parts<4> {
  typedef u32x2_t half __attribute__((aligned(4)));
  typedef uint32_t word;
};
template <typename E>
constexpr int kPiece = 16 / (int)sizeof(E);

// Elements c .. of a row of n, zeros past its end (a row's last piece: 8, 4 and 2 bytes of it).
template <typename E>
__device__ __forceinline__ u32x4_t load_piece(const E* row, int c, int n) {
  constexpr int V = kPiece<E>;
  typedef typename Parts<sizeof(E)>::half half_t;
  typedef typename Parts<sizeof(E)>::word word_t;
  u32x4_t v = {0u, 0u, 0u, 0u};
  const int left = n - c;
  if (left >= V) {
    if constexpr (sizeof(E) == 2) v = *reinterpret_cast<const piece_a2*>(row + c);
    else v = *reinterpret_cast<const piece_a4*>(row + c);
  }
  if (n % V != 0 && left > 0 && left < V) {  // the first for all lanes alike
    const E* p = row + c;
    if (left & (V / 2)) {
      const u32x2_t h = *reinterpret_cast<const half_t*>(p);
      v[0] = h[0];
      v[1] = h[1];
      p += V / 2;
    }
    const bool second = left & (V / 2);
    if (left & (V / 4)) {
      const uint32_t w = *reinterpret_cast<const word_t*>(p);
      v[0] = second ? v[0] : w;
      v[2] = second ? w : 0u;
      p += V / 4;
    }
    if constexpr (sizeof(E) == 2)
      if (left & 1) {
        const uint32_t w = *p;
        const int at = left >> 1;  // the word it lies in
        v[0] = at == 0 ? w : v[0];
        v[1] = at == 1 ? w : v[1];
        v[2] = at == 2 ? w : v[2];
        v[3] = at == 3 ? w : v[3];
      }
  }
  return v;
}
template <typename E>
__device__ __forceinline__ float element(const u32x4_t& v, int j) {
  if constexpr (sizeof(E) == 2) return j & 1 ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
  else return __uint_as_float(v[j]);
}
// Rounds kPiece<E> values to elements c .. of a row of n.
template <typename E>
__device__ __forceinline__ void store_piece(E* row, int c, int n, const float (&f)[kPiece<E>]) {
  constexpr int V = kPiece<E>;
  u32x4_t v;
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(f[j]);
  }
  typedef typename Parts<sizeof(E)>::half half_t;
  typedef typename Parts<sizeof(E)>::word word_t;
  const int left = n - c;
  if (left >= V) {
    if constexpr (sizeof(E) == 2) *reinterpret_cast<piece_a2*>(row + c) = v;
    else *reinterpret_cast<piece_a4*>(row + c) = v;
  }
  if (n % V != 0 && left > 0 && left < V) {
    E* p = row + c;
    const bool second = left & (V / 2);
    if (second) {
      *reinterpret_cast<half_t*>(p) = u32x2_t{v[0], v[1]};
      p += V / 2;
    }
    if (left & (V / 4)) {
      *reinterpret_cast<word_t*>(p) = second ? v[2] : v[0];
      p += V / 4;
    }
    if constexpr (sizeof(E) == 2)
      if (left & 1) *p = (E)(left >> 1 == 0 ? v[0] : left >> 1 == 1 ? v[1] : left >> 1 == 2 ? v[2] : v[3]);
  }
}

// ---------------------------------------------------------------------------
// Layer norm.
struct NormParams {
  const void* x;
  int64_t ldx;
  const void* weight;  // null: ones
  const void* bias;    // null: zeros
  int param_dtype;
  int dtype;
  int64_t rows;
  int cols;
  float eps;
  void* y;             // forward
  int64_t ldy;
  float* stats;        // [rows][2]: mean, 1 / sqrt(variance + eps)
  const void* dy;      // gradient
  int64_t lddy;
  void* dx;
  int64_t lddx;
  float* dw;
  float* db;
  int accumulate;
  float* part;         // [blocks][2][cols]
  int blocks;
  int num_cu;
};
size_t norm_grad_floats(int64_t rows, int cols, int dtype);
hipError_t launch_norm(const NormParams& p, hipStream_t s);
hipError_t launch_norm_grad(NormParams p, hipStream_t s);

// ---------------------------------------------------------------------------
// Router.
struct RouteParams {
  const void* z;
  int64_t ldz;
  int dtype;
  int64_t rows;
  int experts, top;
  const uint8_t* live;  // null: every token
  int normalize;
  float balance, zloss;
  int32_t* ids;         // [rows][top]
  float* gates;
  int32_t* counts;      // [experts + 1]; the last: live tokens
  int32_t* offsets;     // [experts + 1]
  int32_t* slots;       // [rows][top]
  int32_t* tokens;      // [rows * top]
  float* loss;
  void* ws;
  // gradient
  const float* dgates;
  const float* upstream;
  void* dz;
  int64_t lddz;
  int num_cu;
};
size_t route_workspace(int64_t rows, int experts);
hipError_t launch_route(const RouteParams& p, hipStream_t s);
hipError_t launch_route_grad(const RouteParams& p, hipStream_t s);

// ---------------------------------------------------------------------------
// Values in 8 bits: e4m3, a power of two 2^(code - 127) for each 128 of a row.
constexpr int kBlock8 = 128;
struct Store8Params {
  const void* x;       // rows x cols; gated: rows x 2 cols
  int64_t ldx;
  int dtype;
  int64_t rows;
  int cols;
  uint8_t* values;     // rows x up128(cols); gated: twice that
  int64_t ldv;
  uint8_t* scales;
  int64_t lds;
  int gated;
  void* act;           // silu of x (times the second half) in x's type
  int64_t lda;
  const void* dact;    // gradient of act
  int64_t ldda;
  void* dx;            // gradient of x
  int64_t lddx;
  // weights: `batch` matrices of rows x cols, one code for each 128 x 128
  int batch;
  int64_t stride_x, stride_v, stride_s;
  int transposed;
  int num_cu;
};
hipError_t launch_store8(const Store8Params& p, hipStream_t s);
hipError_t launch_load8(const Store8Params& p, hipStream_t s);  // writes act
hipError_t launch_store8_weight(const Store8Params& p, hipStream_t s);
hipError_t launch_silu8(const Store8Params& p, hipStream_t s);
hipError_t launch_silu8_grad(const Store8Params& p, hipStream_t s);

// ---------------------------------------------------------------------------
// Products of 8-bit values, grouped by expert: C[t][j] = sum_k A[t][k] B_e[j][k].
struct Fp8Params {
  const uint8_t* a;    // rows x k
  int64_t lda;
  const uint8_t* sa;   // rows x k / 128
  int64_t ldsa;
  const uint8_t* b;    // per group n x k
  int64_t ldb, stride_b;
  const uint8_t* sb;   // per group ceil(n / 128) x k / 128
  int64_t ldsb, stride_sb;
  const void* offsets; // null: one group of all rows
  int off64;
  int groups;
  int64_t rows;
  int n, k;            // k a multiple of 128
  void* c;
  int64_t ldc;
  int out_dtype;
  int num_cu;
};
hipError_t launch_fp8(const Fp8Params& p, hipStream_t s);

}  // namespace pmx
