// Layer norm over the last dimension, forward and backward.
//   m = mean x, r = 1 / sqrt(mean (x - m)^2 + eps), h = (x - m) r
//   y = h w + b
//   dx = r (g - mean g - h mean(g h)), g = dy w
//   dw = sum_t dy h, db = sum_t dy
//
// Bound: HBM.  A row stays in registers, packed as it was read, from its load
// to its result, so the variance is the two-pass one of the mean's deviations
// and costs no second read.  An fp32 row's first sum rounds, and with it the mean, by some
// 2^-24 of the largest |x|, which is much where the mean is large beside the spread; so
// the second pass adds up the deviations d too, whose mean D corrects the mean and the
// variance, mean d^2 - D^2, and is taken off every d (16384 x 1024 23.4 us with it and
// without, 55924 x 300 26.6 and 25.3, 3355 x 5000 32 and 29).  Of bf16 values, 8 bits each, a
// sum of 16384 is exact unless they differ by a factor of four, and then the spread is as
// large.  16 lanes hold short rows, a wave those of up to 1024
// elements, four to sixteen waves longer ones.  Blocks are persistent: the next
// row's loads are under way while this one is reduced, weights stay in registers
// (the longest rows': in LDS), and in the backward pass a thread's columns stay the
// same, so it sums dy and dy h of its rows in registers.  The block's teams add those
// sums pairwise in LDS, a second launch adds the blocks' in their order: no atomics,
// the same bits on every call.  Statistics and sums are fp32.
//
// Measured (bytes of the rows alone): 32768 x 1024 bf16 forward 22 us, 6.1 TB/s, backward
// 38, 5.3 TB/s, of which 4 to 5 the join; 16384 x 1024 fp32 21 and 35; 524288 x 64 bf16 37
// and 51; 8192 x 4096 bf16 24 and 42; 2048 x 16384 bf16 31 and 47.  8 rows: 3.3 us.
#include <algorithm>

#include "pmx_layer.h"

namespace pmx {
namespace {

// LANES a row, NV pieces of 16 bytes a lane, TEAMS rows at a time a block.
template <typename E_, int LANES_, int NV_, int TEAMS_>
struct NCfg {
  typedef E_ E;
  static constexpr int LANES = LANES_, NV = NV_, TEAMS = TEAMS_, V = kPiece<E_>;
  static constexpr int W = LANES < 64 ? 1 : LANES / 64, THREADS = LANES * TEAMS, COLS = LANES * NV * V;
  // 1024 threads have 128 registers each: weights in LDS, and with 16 elements a lane no row ahead
  static constexpr bool LDS_W = LANES == 1024, AHEAD = !(LDS_W && NV * V == 16);
};

// Sums over the team's lanes of N values; red: [2][waves][N], alternating.
template <class C, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*red)[C::THREADS / 64][N], int& flip) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = C::LANES == 16 ? row_sum(v[i]) : wave_sum(v[i]);
  if constexpr (C::W > 1) {
    const int wid = threadIdx.x >> 6, team = wid / C::W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[flip][wid][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = red[flip][team * C::W][i];
#pragma unroll
      for (int w = 1; w < C::W; ++w) s += red[flip][team * C::W + w][i];
      v[i] = s;
    }
    flip ^= 1;  // the next sum writes the other half: one barrier a sum
  }
}

// A thread's elements of a parameter vector, `other` where there is none.
template <class C>
__device__ __forceinline__ void load_param(float (&w)[C::NV][C::V], const void* p, int dtype, int cols, int lane,
                                           float other) {
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    const int c = (i * C::LANES + lane) * C::V;
    if (!p) {
#pragma unroll
      for (int j = 0; j < C::V; ++j) w[i][j] = other;
    } else if (dtype == PMX_F32) {
#pragma unroll
      for (int k = 0; k < C::V; k += 4) {
        const u32x4_t v = load_piece(reinterpret_cast<const float*>(p), c + k, cols);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][k + j] = element<float>(v, j);
      }
    } else {
      const u32x4_t v = load_piece(reinterpret_cast<const uint16_t*>(p), c, cols);
#pragma unroll
      for (int j = 0; j < C::V; ++j) w[i][j] = element<uint16_t>(v, j);
    }
  }
}

template <class C>
__device__ __forceinline__ void load_row(u32x4_t (&v)[C::NV], const void* p, int64_t ld, int64_t row, int cols,
                                         int lane) {
  const typename C::E* r = reinterpret_cast<const typename C::E*>(p) + row * ld;
#pragma unroll
  for (int i = 0; i < C::NV; ++i) v[i] = load_piece(r, (i * C::LANES + lane) * C::V, cols);
}

// The rows' registers are wanted here, and nothing computed from them is kept past it.  In
// the backward pass of the longest rows, which have no registers left (it costs time
// elsewhere: 32768 x 1024 bf16 44 -> 48 us); and between two rows of the fp32 forward pass,
// where the wait for the next row would else come behind the loads of the one after it
// (3355 x 5000 36.8 -> 34.4 us).
template <int N>
__device__ __forceinline__ void again(u32x4_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void norm_kernel(NormParams p) {
  typedef typename C::E E;
  constexpr int N2 = sizeof(E) == 4 ? 2 : 1;  // sums of the second pass
  __shared__ float red1[2][C::THREADS / 64][1], red2[2][C::THREADS / 64][N2];
  const int team = threadIdx.x / C::LANES, lane = threadIdx.x % C::LANES;
  const int64_t step = (int64_t)gridDim.x * C::TEAMS;
  const float cols = (float)p.cols, inv = 1.f / cols;
  int flip = 0;
  int64_t base = (int64_t)blockIdx.x * C::TEAMS;
  // the block's teams go round together (barriers); a team past the end repeats the last row
  auto row_of = [&](int64_t b) { return min(b + team, p.rows - 1); };
  u32x4_t x[C::NV];
  load_row<C>(x, p.x, p.ldx, row_of(base), p.cols, lane);
  float w[C::NV][C::V], b[C::NV][C::V];
  load_param<C>(w, p.weight, p.param_dtype, p.cols, lane, 1.f);
  load_param<C>(b, p.bias, p.param_dtype, p.cols, lane, 0.f);
  if constexpr (N2 == 2) again(x);
  for (; base < p.rows; base += step) {
    u32x4_t next[C::NV];
    const bool more = base + step < p.rows;
    if (more) load_row<C>(next, p.x, p.ldx, row_of(base + step), p.cols, lane);
    float t[1] = {0.f};
#pragma unroll
    for (int i = 0; i < C::NV; ++i)
#pragma unroll
      for (int j = 0; j < C::V; ++j) t[0] += element<E>(x[i], j);
    team_sum<C, 1>(t, red1, flip);
    const float mean = t[0] / cols;
    float s[N2] = {}, off = 0.f;
#pragma unroll
    for (int i = 0; i < C::NV; ++i)
#pragma unroll
      for (int j = 0; j < C::V; ++j) {
        float d = element<E>(x[i], j) - mean;
        d = (i * C::LANES + lane) * C::V + j < p.cols ? d : 0.f;
        s[0] = fmaf(d, d, s[0]);
        if constexpr (N2 == 2) {
          s[1] += d;
          x[i][j] = __float_as_uint(d);
        }
      }
    team_sum<C, N2>(s, red2, flip);
    if constexpr (N2 == 2) {
      // a row of equal values: d is the same few units of the last place everywhere, both sums
      // are exact, and what is left of d and of the variance is 0
      // s[1] / cols, rounded once: the quotient's error goes back in (the compiler's division takes
      // three times the instructions)
      off = s[1] * inv;
      off = fmaf(fmaf(-off, cols, s[1]), inv, off);
    }
    float var = s[0] / cols;
    if constexpr (N2 == 2) {
      var = fmaf(-off, off, var);
      var = var < 0.f ? 0.f : var;
    }
    const float r = 1.f / sqrtf(var + p.eps);
    const int64_t row = base + team;
    if (row < p.rows) {
      E* y = reinterpret_cast<E*>(p.y) + row * p.ldy;
#pragma unroll
      for (int i = 0; i < C::NV; ++i) {
        float f[C::V];
#pragma unroll
        for (int j = 0; j < C::V; ++j) f[j] = (element<E>(x[i], j) - (N2 == 2 ? off : mean)) * r * w[i][j] + b[i][j];
        store_piece(y, (i * C::LANES + lane) * C::V, p.cols, f);
      }
      if (lane == 0 && p.stats) {
        p.stats[2 * row] = mean + off;
        p.stats[2 * row + 1] = r;
      }
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < C::NV; ++i) x[i] = next[i];
      if constexpr (N2 == 2) again(x);
    }
  }
}

// V floats to elements c .. of a row of n.
template <int V>
__device__ __forceinline__ void store_piece4(float* row, int c, int n, const float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 4) {
    const float q[4] = {f[k], f[k + 1], f[k + 2], f[k + 3]};
    store_piece(row, c + k, n, q);
  }
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void norm_grad_kernel(NormParams p) {
  typedef typename C::E E;
  constexpr int HALF = C::TEAMS / 2;
  __shared__ float red[2][C::THREADS / 64][2];
  // weights [NV * V][LANES]; the teams' sums, half of them at a time
  __shared__ float lw[C::LDS_W ? C::COLS : 1];
  __shared__ float sums[HALF ? HALF : 1][2][HALF ? C::COLS : 1];
  const int team = threadIdx.x / C::LANES, lane = threadIdx.x % C::LANES;
  const int64_t step = (int64_t)gridDim.x * C::TEAMS;
  const float inv = 1.f / (float)p.cols;
  int flip = 0;
  int64_t base = (int64_t)blockIdx.x * C::TEAMS;
  auto row_of = [&](int64_t b) { return min(b + team, p.rows - 1); };
  u32x4_t x[C::NV], g[C::NV];
  float mean, r;
  auto fetch = [&](u32x4_t(&a)[C::NV], u32x4_t(&b)[C::NV], float& m, float& q, int64_t at) {
    const int64_t row = row_of(at);
    load_row<C>(a, p.x, p.ldx, row, p.cols, lane);
    load_row<C>(b, p.dy, p.lddy, row, p.cols, lane);
    m = p.stats[2 * row];
    q = p.stats[2 * row + 1];
  };
  fetch(x, g, mean, r, base);
  float wr[C::NV][C::V], dw[C::NV][C::V], db[C::NV][C::V];
  load_param<C>(wr, p.weight, p.param_dtype, p.cols, lane, 1.f);
  if constexpr (C::LDS_W) {  // each lane its own: no barrier
#pragma unroll
    for (int i = 0; i < C::NV; ++i)
#pragma unroll
      for (int j = 0; j < C::V; ++j) lw[(i * C::V + j) * C::LANES + lane] = wr[i][j];
  }
  auto w = [&](int i, int j) { return C::LDS_W ? lw[(i * C::V + j) * C::LANES + lane] : wr[i][j]; };
#pragma unroll
  for (int i = 0; i < C::NV; ++i)
#pragma unroll
    for (int j = 0; j < C::V; ++j) dw[i][j] = db[i][j] = 0.f;
  for (; base < p.rows; base += step) {
    u32x4_t nx[C::NV], ng[C::NV];
    float nmean = 0.f, nr = 0.f;
    const bool more = base + step < p.rows;
    if (C::AHEAD && more) fetch(nx, ng, nmean, nr, base + step);
    const int64_t row = base + team;
    const bool own = row < p.rows;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < C::NV; ++i)
#pragma unroll
      for (int j = 0; j < C::V; ++j) {
        const float dy = element<E>(g[i], j), h = (element<E>(x[i], j) - mean) * r, gw = dy * w(i, j);
        s[0] += gw;
        s[1] += gw * h;
        if (own) {
          dw[i][j] += dy * h;
          db[i][j] += dy;
        }
      }
    team_sum<C, 2>(s, red, flip);
    if constexpr (C::LDS_W) {
      again(x);
      again(g);
    }
    if (own && p.dx) {
      const float m0 = s[0] * inv, m1 = s[1] * inv;
      E* dx = reinterpret_cast<E*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < C::NV; ++i) {
        float f[C::V];
#pragma unroll
        for (int j = 0; j < C::V; ++j) {
          const float h = (element<E>(x[i], j) - mean) * r;
          f[j] = r * (element<E>(g[i], j) * w(i, j) - m0 - h * m1);
        }
        store_piece(dx, (i * C::LANES + lane) * C::V, p.cols, f);
      }
    }
    if (!more) break;
    if constexpr (C::AHEAD) {
#pragma unroll
      for (int i = 0; i < C::NV; ++i) {
        x[i] = nx[i];
        g[i] = ng[i];
      }
      mean = nmean;
      r = nr;
    } else {
      fetch(x, g, mean, r, base + step);
    }
  }
  if (!p.part) return;
  // the teams' sums, pairwise: the upper half of those left hands its sums to the lower
#pragma unroll
  for (int half = HALF; half > 0; half /= 2) {
    if (team >= half && team < 2 * half)
#pragma unroll
      for (int i = 0; i < C::NV; ++i)
#pragma unroll
        for (int j = 0; j < C::V; ++j) {
          sums[team - half][0][(i * C::V + j) * C::LANES + lane] = dw[i][j];
          sums[team - half][1][(i * C::V + j) * C::LANES + lane] = db[i][j];
        }
    __syncthreads();
    if (team < half)
#pragma unroll
      for (int i = 0; i < C::NV; ++i)
#pragma unroll
        for (int j = 0; j < C::V; ++j) {
          dw[i][j] += sums[team][0][(i * C::V + j) * C::LANES + lane];
          db[i][j] += sums[team][1][(i * C::V + j) * C::LANES + lane];
        }
    __syncthreads();
  }
  if (team) return;
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    store_piece4<C::V>(out, (i * C::LANES + lane) * C::V, p.cols, dw[i]);
    store_piece4<C::V>(out + p.cols, (i * C::LANES + lane) * C::V, p.cols, db[i]);
  }
}

// dw and db: the blocks' sums in their order, 32 segments of them at a time.
__global__ __launch_bounds__(1024) void norm_join_kernel(NormParams p) {
  __shared__ float seg[32][33];
  const int in = threadIdx.x & 31, s = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + in;  // of 2 cols
  const int64_t wide = 2 * (int64_t)p.cols;
  const int per = (p.blocks + 31) / 32, b0 = min(s * per, p.blocks), b1 = min(b0 + per, p.blocks);
  float v = 0.f;
  if (c < wide) {
    int b = b0;
    for (; b + 8 <= b1; b += 8) {  // eight loads on their way
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p.part[(b + i) * wide + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += x[i];
    }
    for (; b < b1; ++b) v += p.part[b * wide + c];
  }
  seg[s][in] = v;
  __syncthreads();
  if (s == 0 && c < wide) {
    float t = seg[0][in];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += seg[i][in];
    float* out = c < p.cols ? p.dw : p.db;
    if (out) {
      out += c < p.cols ? c : c - p.cols;
      *out = p.accumulate ? *out + t : t;
    }
  }
}

// The configuration of a row length: f(NCfg).
template <typename E, typename F>
hipError_t with_cfg(int cols, F&& f) {
  constexpr int V = kPiece<E>;
  if (cols <= 16 * V) return f(NCfg<E, 16, 1, 32>());
  if (cols <= 32 * V) return f(NCfg<E, 16, 2, 32>());
  if (cols <= 64 * V) return f(NCfg<E, 64, 1, 8>());
  if (cols <= 128 * V) return f(NCfg<E, 64, 2, 8>());
  if constexpr (sizeof(E) == 4) {
    if (cols <= 256 * V) return f(NCfg<E, 64, 4, 8>());
  } else {
    if (cols <= 256 * V) return f(NCfg<E, 256, 1, 2>());
  }
  if (cols <= 512 * V) return f(NCfg<E, 256, 2, 2>());
  if (cols <= 1024 * V) return f(NCfg<E, 512, 2, 1>());
  if (cols <= 2048 * V) return f(NCfg<E, 1024, 2, 1>());
  if constexpr (sizeof(E) == 4) return f(NCfg<E, 1024, 4, 1>());
  return hipErrorInvalidValue;
}
template <typename F>
hipError_t with_cfg(int dtype, int cols, F&& f) {
  return dtype == PMX_BF16 ? with_cfg<uint16_t>(cols, f) : with_cfg<float>(cols, f);
}

// Blocks of the backward pass: two a unit where a lane has one piece of a row on its
// way, else one, which halves what the second launch reads: 65536 x 512 bf16 (one piece)
// 38 and 45 us, 32768 x 1024 (two) 41 and 39, 2048 x 4096 23 and 18.
int grad_blocks(int64_t rows, int teams, int pieces) {
  const int64_t most = pieces == 1 && rows >= 4096 ? 512 : 256;
  return (int)std::min<int64_t>((rows + teams - 1) / teams, most);
}

}  // namespace

size_t norm_grad_floats(int64_t rows, int cols, int dtype) {
  if (rows == 0) return 0;
  size_t n = 0;
  (void)with_cfg(dtype, cols, [&](auto c) {
    n = (size_t)grad_blocks(rows, decltype(c)::TEAMS, decltype(c)::NV) * 2 * cols;
    return hipSuccess;
  });
  return n;
}

hipError_t launch_norm(const NormParams& p, hipStream_t s) {
  return with_cfg(p.dtype, p.cols, [&](auto c) {
    typedef decltype(c) C;
    const int64_t blocks = std::min<int64_t>((p.rows + C::TEAMS - 1) / C::TEAMS, p.num_cu * 4);
    norm_kernel<C><<<dim3((unsigned)blocks), dim3(C::THREADS), 0, s>>>(p);
    return hipGetLastError();
  });
}

hipError_t launch_norm_grad(NormParams p, hipStream_t s) {
  p.blocks = 0;
  const bool params = p.dw || p.db;
  if (!params) p.part = nullptr;
  if (p.rows > 0) {
    const hipError_t e = with_cfg(p.dtype, p.cols, [&](auto c) {
      typedef decltype(c) C;
      p.blocks = grad_blocks(p.rows, C::TEAMS, C::NV);
      norm_grad_kernel<C><<<dim3(p.blocks), dim3(C::THREADS), 0, s>>>(p);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!params) return hipSuccess;
  norm_join_kernel<<<dim3((2 * p.cols + 31) / 32), dim3(1024), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace pmx
