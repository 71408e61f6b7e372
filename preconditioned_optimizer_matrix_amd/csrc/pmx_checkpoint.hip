// Values in 8 bits, and activations kept in them for the backward pass.
//
// A row is cut into blocks of 128 values.  A block has one power of two, 2^k,
// the least with max |x| <= 448 2^k (448 is e4m3's largest value; k >= -126; 0
// for a block of zeros), kept as k + 127, and each value the e4m3 number nearest
// to x 2^-k, ties to even.  Scaling by 2^-k is exact, so there is one rounding:
// half a step of three bits, or 2^-10 of the largest scaled value below 2^-6.
// The power of two is what the matrix instructions take as a scale (pmx_fp8.hip)
// and makes every decoded value a bf16 number: reading back rounds nothing.
// Infinities and NaN are stored as NaN and left out of the maximum.
//
// silu with its checkpoint: a = x s(x), s(x) = 1 / (1 + exp(-x)), gated a = x s(x) u
// for x the first and u the second half of the row, each half in whole blocks.
// Backward from the stored values: da/dx = s (1 + x (1 - s)), and a once more.
//
// Bound: HBM; each value is read and written once.  16 lanes share a block, 8
// values a lane: 16 bytes of bf16 in, 8 bytes out, the maximum over a DPP row.
//
// Measured: gated silu, 32768 x 4096 bf16, 1.07 GB 199 to 209 us (5.2 TB/s), backward with
// the activation 1.34 GB 241 us (5.6 TB/s); stored and read back, 8192 x 4096 bf16, 101 MB
// 17 to 18 and 16.5 us; weights, 32 of 4096 x 1024 bf16, 403 MB 90 us, transposed 93.
#include <algorithm>

#include "pmx_layer.h"

namespace pmx {
namespace {

// s(x), and 1 - s(x) without what the difference would cancel: with t = exp(-|x|) one is
// 1 / (1 + t), the other t / (1 + t), each a few ulps off wherever x lies.  For bf16 results
// t may be off by |x| 2^-24, the rounding of the exponent's argument: at most 2^-17, where t
// is not 0, and theirs is 2^-8 (32768 x 4096 bf16 forward 124 us, 127.5 with exp_acc).
template <typename E>
__device__ __forceinline__ float sigmoid(float x, float& one_minus) {
  const float t = sizeof(E) == 4 ? exp_acc(-fabsf(x)) : __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
  const float d = 1.f + t, q = __builtin_amdgcn_rcpf(d);
  const float r = fmaf(q, fmaf(-d, q, 1.f), q), tr = t * r;  // one Newton step: v_rcp is off by up to an ulp
  one_minus = x >= 0.f ? tr : r;
  return x >= 0.f ? r : tr;
}

// |x| as bits where finite, else 0: whole-number order is that of the magnitudes.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? a : 0.f;  // NaN compares false
}

// The block's code for the largest finite magnitude of it.
__device__ __forceinline__ int scale_code(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // exponent (biased) and mantissa: 448 = 1.75 * 2^8; the least k with amax <= 448 2^k
  int code = (int)(u >> 23) - 8 + ((u & 0x7FFFFF) > 0x600000);
  code = max(code, 1);  // also the subnormal ones
  return amax > 0.f ? code : 127;
}
__device__ __forceinline__ float code_power(int code) {  // 2^(code - 127); 255: NaN
  return code == 255 ? __builtin_nanf("") : code == 0 ? 0x1p-127f : __uint_as_float((uint32_t)code << 23);
}
__device__ __forceinline__ float inverse_power(int code) {  // 2^(127 - code), 1 <= code <= 253
  return __uint_as_float((uint32_t)(254 - code) << 23);
}
__device__ __forceinline__ float storable(float x, float inv) {
  return fabsf(x) < __builtin_inff() ? x * inv : __builtin_nanf("");
}

__device__ __forceinline__ u32x2_t encode8(const float (&f)[8], float inv) {
  u32x2_t q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(storable(f[4 * h], inv), storable(f[4 * h + 1], inv), w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(storable(f[4 * h + 2], inv), storable(f[4 * h + 3], inv), w, true);
    q[h] = (uint32_t)w;
  }
  return q;
}
__device__ __forceinline__ void decode8(float (&f)[8], u32x2_t q, float power) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
    f[4 * h] = lo[0] * power;
    f[4 * h + 1] = lo[1] * power;
    f[4 * h + 2] = hi[0] * power;
    f[4 * h + 3] = hi[1] * power;
  }
}

// Elements c .. c + 7 of a row of n, zeros past its end; and back.
template <typename E>
__device__ __forceinline__ void load8(float (&f)[8], const E* row, int c, int n) {
  constexpr int V = kPiece<E>;
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) {
    const u32x4_t v = load_piece(row, c + i * V, n);
#pragma unroll
    for (int j = 0; j < V; ++j) f[i * V + j] = element<E>(v, j);
  }
}
template <typename E>
__device__ __forceinline__ void store8(E* row, int c, int n, const float (&f)[8]) {
  constexpr int V = kPiece<E>;
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) {
    float g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = f[i * V + j];
    store_piece(row, c + i * V, n, g);
  }
}

// One block of a row: values, code.
__device__ __forceinline__ void put_block(const float (&f)[8], uint8_t* values, uint8_t* scales, int block, int lane16) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(f[j]));
  const int code = scale_code(row_max(m));
  *reinterpret_cast<u32x2_t*>(values + (int64_t)block * kBlock8 + 8 * lane16) = encode8(f, inverse_power(code));
  if (lane16 == 0) scales[block] = (uint8_t)code;
}
__device__ __forceinline__ void get_block(float (&f)[8], const uint8_t* values, const uint8_t* scales, int block,
                                          int lane16) {
  decode8(f, *reinterpret_cast<const u32x2_t*>(values + (int64_t)block * kBlock8 + 8 * lane16), code_power(scales[block]));
}

// Blocks of rows dealt out to groups of 16 lanes: a power of two of them, `across`, side by side in a row.
struct Deal {
  int across_log, blocks;  // blocks of a row (of one half)
};
Deal deal_of(int cols) {
  Deal d = {0, (cols + kBlock8 - 1) / kBlock8};
  while (d.across_log < 4 && (1 << d.across_log) < d.blocks) ++d.across_log;
  return d;
}
template <typename F>
__device__ __forceinline__ void each_block(const Deal& d, int64_t rows, F&& f) {
  const int group = threadIdx.x >> 4, lane16 = threadIdx.x & 15;
  const int at = group & ((1 << d.across_log) - 1), down = 16 >> d.across_log;
  for (int64_t row = (int64_t)blockIdx.x * down + (group >> d.across_log); row < rows; row += (int64_t)gridDim.x * down)
    for (int b = at; b < d.blocks; b += 1 << d.across_log) f(row, b, lane16);
}

template <typename E>
__global__ __launch_bounds__(256) void store8_kernel(Store8Params p, Deal d) {
  each_block(d, p.rows, [&](int64_t row, int b, int lane16) {
    float f[8];
    load8(f, reinterpret_cast<const E*>(p.x) + row * p.ldx, b * kBlock8 + 8 * lane16, p.cols);
    put_block(f, p.values + row * p.ldv, p.scales + row * p.lds, b, lane16);
  });
}

template <typename E>
__global__ __launch_bounds__(256) void load8_kernel(Store8Params p, Deal d) {
  each_block(d, p.rows, [&](int64_t row, int b, int lane16) {
    float f[8];
    get_block(f, p.values + row * p.ldv, p.scales + row * p.lds, b, lane16);
    store8(reinterpret_cast<E*>(p.act) + row * p.lda, b * kBlock8 + 8 * lane16, p.cols, f);
  });
}

template <typename E, bool GATED>
__global__ __launch_bounds__(256) void silu8_kernel(Store8Params p, Deal d) {
  each_block(d, p.rows, [&](int64_t row, int b, int lane16) {
    const E* x = reinterpret_cast<const E*>(p.x) + row * p.ldx;
    uint8_t *v = p.values + row * p.ldv, *s = p.scales + row * p.lds;
    const int c = b * kBlock8 + 8 * lane16;
    float f[8], u[8], a[8];
    load8(f, x, c, p.cols);
    if (GATED) load8(u, x + p.cols, c, p.cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float rest;
      a[j] = f[j] * sigmoid<E>(f[j], rest);
      if (GATED) a[j] *= u[j];
    }
    put_block(f, v, s, b, lane16);
    if (GATED) put_block(u, v, s, d.blocks + b, lane16);
    store8(reinterpret_cast<E*>(p.act) + row * p.lda, c, p.cols, a);
  });
}

template <typename E, bool GATED>
__global__ __launch_bounds__(256) void silu8_grad_kernel(Store8Params p, Deal d) {
  each_block(d, p.rows, [&](int64_t row, int b, int lane16) {
    const uint8_t *v = p.values + row * p.ldv, *s = p.scales + row * p.lds;
    const int c = b * kBlock8 + 8 * lane16;
    float x[8], u[8], g[8], du[8], a[8];
    load8(g, reinterpret_cast<const E*>(p.dact) + row * p.ldda, c, p.cols);
    get_block(x, v, s, b, lane16);
    if (GATED) get_block(u, v, s, d.blocks + b, lane16);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float rest;
      const float sg = sigmoid<E>(x[j], rest), y = x[j] * sg;
      a[j] = GATED ? y * u[j] : y;
      if (GATED) {
        du[j] = g[j] * y;
        g[j] *= u[j];
      }
      g[j] *= sg * (1.f + x[j] * rest);
    }
    E* dx = reinterpret_cast<E*>(p.dx) + row * p.lddx;
    store8(dx, c, p.cols, g);
    if (GATED) store8(dx + p.cols, c, p.cols, du);
    if (p.act) store8(reinterpret_cast<E*>(p.act) + row * p.lda, c, p.cols, a);
  });
}

// Weights: one code for each 128 x 128 tile.  A block takes a tile, 8 rows of 16
// groups at a time; transposed, the bytes turn in LDS (pitch 132: the column
// reads of 32 lanes fall on distinct banks).
template <typename E>
__global__ __launch_bounds__(256) void store8_weight_kernel(Store8Params p, int tiles_c, int tiles_r) {
  __shared__ float red[4];
  __shared__ __attribute__((aligned(16))) uint8_t turn[128 * 132];
  const int64_t t = blockIdx.x;
  const int tc = (int)(t % tiles_c), tr = (int)(t / tiles_c % tiles_r);
  const int64_t e = t / tiles_c / tiles_r;
  const int group = threadIdx.x >> 4, lane16 = threadIdx.x & 15, c = tc * kBlock8 + 8 * lane16;
  const E* x = reinterpret_cast<const E*>(p.x) + e * p.stride_x;
  float f[8][8], m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = tr * kBlock8 + 16 * i + group;
    if (r < p.rows) {
      load8(f[i], x + r * p.ldx, c, p.cols);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(f[i][j]));
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  const int code = scale_code(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  const float inv = inverse_power(code);
  uint8_t *v = p.values + e * p.stride_v, *s = p.scales + e * p.stride_s;
  if (!p.transposed) {
    if (threadIdx.x == 0) s[tr * p.lds + tc] = (uint8_t)code;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = tr * kBlock8 + 16 * i + group;
      if (r < p.rows) *reinterpret_cast<u32x2_t*>(v + r * p.ldv + c) = encode8(f[i], inv);
    }
    return;
  }
  if (threadIdx.x == 0) s[tc * p.lds + tr] = (uint8_t)code;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const u32x2_t q = encode8(f[i], inv);
    uint32_t* w = reinterpret_cast<uint32_t*>(turn + (16 * i + group) * 132 + 8 * lane16);
    w[0] = q[0];
    w[1] = q[1];
  }
  __syncthreads();
  // row k of the transposed tile: 16 lanes of 8 bytes
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = 16 * i + group;
    if (tc * kBlock8 + k >= p.cols) continue;
    u32x2_t q = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j >> 2] |= (uint32_t)turn[(8 * lane16 + j) * 132 + k] << (8 * (j & 3));
    *reinterpret_cast<u32x2_t*>(v + (int64_t)(tc * kBlock8 + k) * p.ldv + tr * kBlock8 + 8 * lane16) = q;
  }
}

unsigned grid_of(const Store8Params& p, const Deal& d) {
  const int64_t down = 16 >> d.across_log;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((p.rows + down - 1) / down, (int64_t)p.num_cu * 32));
}

}  // namespace

hipError_t launch_store8(const Store8Params& p, hipStream_t s) {
  const Deal d = deal_of(p.cols);
  if (p.dtype == PMX_BF16) store8_kernel<uint16_t><<<grid_of(p, d), 256, 0, s>>>(p, d);
  else store8_kernel<float><<<grid_of(p, d), 256, 0, s>>>(p, d);
  return hipGetLastError();
}

hipError_t launch_load8(const Store8Params& p, hipStream_t s) {
  const Deal d = deal_of(p.cols);
  if (p.dtype == PMX_BF16) load8_kernel<uint16_t><<<grid_of(p, d), 256, 0, s>>>(p, d);
  else load8_kernel<float><<<grid_of(p, d), 256, 0, s>>>(p, d);
  return hipGetLastError();
}

hipError_t launch_silu8(const Store8Params& p, hipStream_t s) {
  const Deal d = deal_of(p.cols);
  const unsigned g = grid_of(p, d);
  if (p.dtype == PMX_BF16) {
    if (p.gated) silu8_kernel<uint16_t, true><<<g, 256, 0, s>>>(p, d);
    else silu8_kernel<uint16_t, false><<<g, 256, 0, s>>>(p, d);
  } else {
    if (p.gated) silu8_kernel<float, true><<<g, 256, 0, s>>>(p, d);
    else silu8_kernel<float, false><<<g, 256, 0, s>>>(p, d);
  }
  return hipGetLastError();
}

hipError_t launch_silu8_grad(const Store8Params& p, hipStream_t s) {
  const Deal d = deal_of(p.cols);
  const unsigned g = grid_of(p, d);
  if (p.dtype == PMX_BF16) {
    if (p.gated) silu8_grad_kernel<uint16_t, true><<<g, 256, 0, s>>>(p, d);
    else silu8_grad_kernel<uint16_t, false><<<g, 256, 0, s>>>(p, d);
  } else {
    if (p.gated) silu8_grad_kernel<float, true><<<g, 256, 0, s>>>(p, d);
    else silu8_grad_kernel<float, false><<<g, 256, 0, s>>>(p, d);
  }
  return hipGetLastError();
}

hipError_t launch_store8_weight(const Store8Params& p, hipStream_t s) {
  const int tiles_c = (p.cols + 127) / 128, tiles_r = (int)((p.rows + 127) / 128);
  const dim3 grid((unsigned)((int64_t)tiles_c * tiles_r * p.batch));
  if (p.dtype == PMX_BF16) store8_weight_kernel<uint16_t><<<grid, 256, 0, s>>>(p, tiles_c, tiles_r);
  else store8_weight_kernel<float><<<grid, 256, 0, s>>>(p, tiles_c, tiles_r);
  return hipGetLastError();
}

}  // namespace pmx
