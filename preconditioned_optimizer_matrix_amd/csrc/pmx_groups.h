// What the products grouped by expert share: the table of the groups' rows and
// tiles that each block builds from the device's offsets, the order of tiles,
// and the way rows of results leave.
#pragma once

#include "pmx_train.h"

namespace pmx {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

// ------------------------------------------------------------ group table
struct Table {
  int begin[PMX_MAX_GROUPS + 1];  // clamped, monotone row offsets
  int tile[PMX_MAX_GROUPS + 1];   // first tile of each group
};

// One wave fills the table: inclusive maximum scan of the clamped offsets, then
// the exclusive sum of ceil(rows / bm) * tiles_n (product) or `fixed` tiles a
// group (outer).  Without offsets all rows are one group.
template <typename P>
__device__ __forceinline__ void build_table(Table& T, const P& p, int bm, int tiles_n, int fixed) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int b = 0; b <= p.groups; b += 64) {
      const int i = b + lane;
      int v = 0;
      if (i <= p.groups) {
        int64_t o = p.offsets ? load_index(p.offsets, i, p.off64) : i * p.rows;
        o = o < 0 ? 0 : o > p.rows ? p.rows : o;
        v = (int)o;
      }
      for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(v, d);
        if (lane >= d && x > v) v = x;
      }
      if (v < carry) v = carry;
      if (i <= p.groups) T.begin[i] = v;
      carry = __shfl(v, 63);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave reads what its other lanes wrote
    __builtin_amdgcn_wave_barrier();
    carry = 0;
    for (int b = 0; b <= p.groups; b += 64) {
      const int i = b + lane;
      int n = 0;
      if (i < p.groups) {
        const int rows = T.begin[i + 1] - T.begin[i];
        n = fixed ? fixed : (rows + bm - 1) / bm * tiles_n;
      }
      int v = n;
      for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(v, d);
        if (lane >= d) v += x;
      }
      if (i <= p.groups) T.tile[i] = carry + v - n;
      carry += __shfl(v, 63);
    }
  }
  __syncthreads();
}

// the group of tile `t`: the last e with tile[e] <= t
__device__ __forceinline__ int group_of(const Table& T, int groups, int t) {
  int lo = 0, hi = groups;  // tile[lo] <= t < tile[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (T.tile[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Tiles of a matrix in groups of 8 tile rows per column sweep.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 8;
  const int per = GM * tiles_n, g = t / per, first = g * GM;
  const int size = tiles_m - first < GM ? tiles_m - first : GM;
  const int in = t - g * per;
  tm = first + in % size;
  tn = in / size;
}

// Rows of C leave through LDS: a wave writes 32 rows of its tile, then stores
// them as 16-byte pieces, whole 128-byte lines, instead of 8- and 16-byte ones
// of 32 rows at a time.  `stage`: the wave's own 32 x (WN + 8 or 4) elements.
template <int WN, typename O>
__device__ __forceinline__ void store_rows(const f32x16* acc, O* stage, O* c, int64_t ldc, int row0,
                                           int rows, int col0, int cols) {
  constexpr int PIT = WN + 16 / (int)sizeof(O), V = 16 / (int)sizeof(O), LPR = WN / V;  // lanes a row
  const int lane = threadIdx.x & 63;
  O* w = stage + (lane & 31) * PIT + 4 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < WN / 32; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4_t v = {acc[j][4 * g], acc[j][4 * g + 1], acc[j][4 * g + 2], acc[j][4 * g + 3]};
      if constexpr (sizeof(O) == 4) *reinterpret_cast<f32x4_t*>(w + 32 * j + 8 * g) = v;
      else *reinterpret_cast<u32x2_t*>(w + 32 * j + 8 * g) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
  // the wave's lanes exchange through LDS: nothing moves across this point
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const int cl = lane % LPR * V, left = cols - (col0 + cl);
#pragma unroll
  for (int r = 0; r < 32; r += 64 / LPR) {
    const int rr = r + lane / LPR;
    if (row0 + rr >= rows || left <= 0) continue;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stage + rr * PIT + cl);
    O* d = c + (int64_t)(row0 + rr) * ldc + col0 + cl;
    if (left >= V) {
      if constexpr (sizeof(O) == 2) *reinterpret_cast<u32x4_a2*>(d) = v;
      else *reinterpret_cast<u32x4_a4*>(d) = v;
    } else {
#pragma unroll
      for (int j = 0; j < V - 1; ++j)
        if (j < left) {
          if constexpr (sizeof(O) == 2) d[j] = (O)(v[j >> 1] >> (16 * (j & 1)));
          else d[j] = __uint_as_float(v[j]);
        }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace
}  // namespace pmx
