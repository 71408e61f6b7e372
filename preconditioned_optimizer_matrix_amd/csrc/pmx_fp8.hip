// Products of 8-bit values grouped by expert: C[t][j] = sum_k A[t][k] B_e[j][k]
// over e4m3 values with a power of two for each 128 of k, a row's own for A, a
// 128 x 128 tile's for B.
#include <algorithm>

#include "pmx_groups.h"
#include "pmx_layer.h"

namespace pmx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// 64 x 64 tiles, four waves of 32 x 32, k tiles of 128 through LDS.
constexpr int kPitch = 144;

template <typename O>
__global__ __launch_bounds__(256) void fp8_kernel(Fp8Params p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * 64 * kPitch];
  __shared__ Table T;
  const int tiles_n = (p.n + 63) / 64, kb = p.k / 128;
  build_table(T, p, 64, tiles_n, 0);
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63, wm = (wid >> 1) * 32, wn = (wid & 1) * 32;
  uint8_t *sa = smem, *sb = smem + 64 * kPitch;
  for (int q = blockIdx.x; q < T.tile[p.groups]; q += gridDim.x) {
    const int e = group_of(T, p.groups, q), r0 = T.begin[e], M = T.begin[e + 1] - r0;
    int tm, tn;
    tile_of(q - T.tile[e], (M + 63) / 64, tiles_n, tm, tn);
    const int m0 = tm * 64, n0 = tn * 64;
    const uint8_t *A = p.a + (int64_t)r0 * p.lda, *B = p.b + e * p.stride_b;
    const uint8_t *SA = p.sa + (int64_t)r0 * p.ldsa, *SB = p.sb + e * p.stride_sb;
    f32x16 acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.f;
    const int ra = min(m0 + wm + (lane & 31), M - 1), rb = min(n0 + wn + (lane & 31), p.n - 1);
    for (int kt = 0; kt < kb; ++kt) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int idx = threadIdx.x + 256 * i, r = idx >> 3, c = (idx & 7) * 16;
        *reinterpret_cast<u32x4_t*>(sa + r * kPitch + c) =
            *reinterpret_cast<const u32x4_t*>(A + (int64_t)min(m0 + r, M - 1) * p.lda + kt * 128 + c);
        *reinterpret_cast<u32x4_t*>(sb + r * kPitch + c) =
            *reinterpret_cast<const u32x4_t*>(B + (int64_t)min(n0 + r, p.n - 1) * p.ldb + kt * 128 + c);
      }
      const int ca = SA[(int64_t)ra * p.ldsa + kt], cb = SB[(int64_t)(rb >> 7) * p.ldsb + kt];
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int o = (lane & 31) * kPitch + 64 * s + 32 * (lane >> 5);
        const i32x4 a0 = *reinterpret_cast<const i32x4*>(sa + wm * kPitch + o), a1 = *reinterpret_cast<const i32x4*>(sa + wm * kPitch + o + 16);
        const i32x4 b0 = *reinterpret_cast<const i32x4*>(sb + wn * kPitch + o), b1 = *reinterpret_cast<const i32x4*>(sb + wn * kPitch + o + 16);
        const i32x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7), b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, 0, 0, 0, cb, 0, ca);
      }
    }
    const int row = m0 + wm + (lane & 31);
    if (row < M)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int col = n0 + wn + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
        if (col < p.n) {
          O* c = reinterpret_cast<O*>(p.c) + (int64_t)(r0 + row) * p.ldc + col;
          if constexpr (sizeof(O) == 4) *c = acc[v];
          else *c = (O)pack_bf16(acc[v], 0.f);
        }
      }
  }
  // rows in no group
  const int lo = T.begin[0], hi = T.begin[p.groups];
  const int64_t outside = lo + (p.rows - hi);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < outside * p.n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / p.n;
    reinterpret_cast<O*>(p.c)[(r < lo ? r : hi + r - lo) * p.ldc + (i - r * p.n)] = 0;
  }
}

}  // namespace

int fp8_splits(int64_t rows, int k, int n, int groups) { return 1; }

hipError_t launch_fp8(const Fp8Params& p, hipStream_t s) {
  const int64_t tiles = (p.rows / 64 + std::min<int64_t>(p.groups, p.rows)) * ((p.n + 63) / 64);
  const dim3 grid((unsigned)std::min<int64_t>(tiles, p.num_cu * 8));
  if (p.out_dtype == PMX_BF16) fp8_kernel<uint16_t><<<grid, 256, 0, s>>>(p);
  else fp8_kernel<float><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace pmx
