// Products of 8-bit values grouped by expert: C[t][j] = sum_k A[t][k] B_e[j][k]
// over e4m3 values with a power of two for each 128 of k, a row's own for A, a
// 128 x 128 tile's for B.
//
// Design (CDNA4):
//  * bf16 results, through tiles: the scaled 8-bit matrix instructions, which take
//    the powers of two as the bytes they are stored as, so scaling costs nothing.
//    A lane's four scale bytes of four k tiles are one register, and each
//    instruction names the byte it takes.  These instructions cut each of eight
//    neighbouring products off (towards zero) 2^-13 below the power of two of the
//    largest of the eight (an operand below e4m3's normal numbers, 2^-6, counting as
//    2^-6, a zero not), before the sums of eight are added in fp32.  That is a
//    choice of fewer bits: the operands themselves were rounded by 2^-4, normally
//    distributed ones lose 1.5e-5 of the result's norm at k = 1024, and exact sums
//    take twice the instructions' time and more.  At worst, eight by eight one large
//    product beside seven small ones and all large ones cancelling, 7 2^-13 of the
//    sum of magnitudes; more only among products that small operands make small.
//  * fp32 results, and few rows a group, where memory is what is waited for (16 rows,
//    32 experts of 4096 x 1024 14.6 us and 14.4 by the 8-bit instructions, 60 rows
//    24.9 and 26.8, 16 rows, one of 8192 x 8192 20.9 and 21.2): the values are
//    widened to bf16, exactly, and multiplied at half the rate; the sum over each 128
//    of k is scaled (ldexp, exact) and added in fp32.
//  * Tiles by rule (choose): for few rows a group, weights go from memory to the
//    matrix cores without LDS; 64 x 64 and 128 x 128 through LDS, two k tiles;
//    256 x 256 (bf16) loaded straight into LDS, two groups of waves taking turns at
//    the matrix cores.
//  * The matrix instruction's operands are swapped (B first), so a lane ends with
//    four neighbouring columns of one row of C.
//  * Rows past a group's end read the group's last row (256 x 256: zeros); their
//    results are not stored.
//
// Measured, bf16: 32768 rows, 32 experts of 4096 x 1024 134 to 153 us (1.8 to 2.05
// PFLOP/s), 141 to 160 with a router's uneven groups; it also writes 268 MB, 53 us at a copy's rate.  8192 x
// 8192 x 8192 390 to 440 us, 2.5 to 2.8 PFLOP/s, by what clock the card holds: the
// instructions alone reach 4.5 at full clock, and are busy 65 to 69% of the cycles (the
// uneven groups: 55%).  16
// rows through 16 experts 14.4 to 15.2 us for 67 MB of weights.  fp32: 375 to 380 us, 0.73 PFLOP/s.
#include <algorithm>

#include "pmx_groups.h"
#include "pmx_layer.h"

namespace pmx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8 join8(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// Eight e4m3 values as bf16, exactly.
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false),
               b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true),
               c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false),
               d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Rows of C in no group, [0, lo) and [hi, rows): zeros.
template <typename O>
__device__ __forceinline__ void zero_outside(const Fp8Params& p, int lo, int hi) {
  const int64_t outside = lo + (p.rows - hi);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < outside * p.n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / p.n;
    reinterpret_cast<O*>(p.c)[(r < lo ? r : hi + r - lo) * p.ldc + (i - r * p.n)] = 0;
  }
}

// ------------------------------------------------------------ few rows a group
// Weights go from memory to the matrix cores without LDS: a wave has 16 columns of a
// group and 16 of its rows at a time, a lane loads 32 bytes of a row of B, 16 rows of
// whole 128-byte lines an instruction pair, four k tiles on their way.  S = 1: every
// wave its own columns; S = 4: a block's waves share the contraction and add their
// results in LDS.
template <typename O, int S>
__global__ __launch_bounds__(256, S == 1 ? 4 : 3) void fp8_stream_kernel(Fp8Params p, int blocks) {
  __shared__ float sum[S == 1 ? 1 : 4][16][17];
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int slot = blockIdx.x / blocks, kb = p.k / 128;
  const int n0 = ((blockIdx.x - slot * blocks) * (S == 1 ? 4 : 1) + (S == 1 ? wid : 0)) * 16;
  // the slot-th group that has rows: offsets clamped, and none below an earlier one
  int e = slot, first = 0, last = (int)p.rows, lo = 0, hi = (int)p.rows;
  if (p.offsets) {
    e = -1;
    hi = 0;
    int seen = 0;
    for (int base = 0; base < p.groups; base += 64) {
      const int i = base + lane;
      auto offset = [&](int j) {
        const int64_t o = load_index(p.offsets, min(j, p.groups), p.off64);
        return (int)(o < 0 ? 0 : o > p.rows ? p.rows : o);
      };
      int begin = offset(i);
      const int after = offset(i + 1);
      if (base == 0) lo = __builtin_amdgcn_readfirstlane(begin);
      for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(begin, d);
        if (lane >= d) begin = max(begin, x);
      }
      begin = max(begin, hi);
      const int end = max(begin, after);
      const uint64_t live = __ballot(i < p.groups && end > begin);
      const uint64_t mine = __ballot((live >> lane & 1) && seen + __popcll(live & ((1ull << lane) - 1)) == slot);
      if (mine) {
        const int l = __builtin_ctzll(mine);
        e = base + l;
        first = __builtin_amdgcn_readlane(begin, l);
        last = __builtin_amdgcn_readlane(end, l);
      }
      seen += __popcll(live);
      hi = wave_max(end);
    }
  }
  zero_outside<O>(p, lo, hi);
  if (e < 0 || (S == 1 && n0 >= p.n)) return;
  const int k0 = S == 1 ? 0 : kb * wid / 4, k1 = S == 1 ? kb : kb * (wid + 1) / 4;
  const uint8_t* B = p.b + e * p.stride_b + (int64_t)min(n0 + l16, p.n - 1) * p.ldb + 32 * g;
  const uint8_t* SB = p.sb + e * p.stride_sb + (int64_t)(n0 >> 7) * p.ldsb;
  // four scale bytes from k tile kt on
  auto scales = [&](const uint8_t* q, int kt) {
    typedef uint32_t u32_a1 __attribute__((aligned(1)));
    if (kb >= 4) {
      const int o = min(kt, kb - 4);
      return (int)(*reinterpret_cast<const u32_a1*>(q + o) >> (8 * (kt - o)));
    }
    int v = 0;
    for (int j = 0; kt + j < kb; ++j) v |= (int)q[kt + j] << (8 * j);
    return v;
  };
  for (int r0 = first; r0 < last; r0 += 16) {
    const int64_t row = min(r0 + l16, last - 1);
    const uint8_t *A = p.a + row * p.lda + 32 * g, *SA = p.sa + row * p.ldsa;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    bool bad = false;
    i32x4 b[4][2], a[4][2];
    auto load = [&](int d, int kt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b[d][h] = *reinterpret_cast<const i32x4*>(B + kt * 128 + 16 * h);
        a[d][h] = *reinterpret_cast<const i32x4*>(A + kt * 128 + 16 * h);
      }
    };
    int sa = 0, sb = 0;
    if (k0 < k1) {
      sa = scales(SA, k0);
      sb = scales(SB, k0);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (k0 + d < k1) load(d, k0 + d);
    auto step = [&](int kt, auto which) {
      constexpr int D = decltype(which)::value;
      if (kt >= k1) return;
      const i32x8 xa = join8(a[D][0], a[D][1]), xb = join8(b[D][0], b[D][1]);
      f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t)
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(xb[2 * t], xb[2 * t + 1]), widen(xa[2 * t], xa[2 * t + 1]), part, 0, 0, 0);
      const int ea = sa >> (8 * D) & 255, eb = sb >> (8 * D) & 255;
      bad |= ea == 255 || eb == 255;
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] += __builtin_ldexpf(part[v], ea + eb - 254);
      if (kt + 4 < k1) load(D, kt + 4);
    };
    for (int kt = k0; kt < k1; kt += 4) {
      int na = 0, nb = 0;
      if (kt + 4 < k1) {
        na = scales(SA, kt + 4);
        nb = scales(SB, kt + 4);
      }
      step(kt, std::integral_constant<int, 0>());
      step(kt + 1, std::integral_constant<int, 1>());
      step(kt + 2, std::integral_constant<int, 2>());
      step(kt + 3, std::integral_constant<int, 3>());
      sa = na;
      sb = nb;
    }
    if (bad)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] = __builtin_nanf("");
    if constexpr (S == 1) {
      const int col = n0 + 4 * g;
      O* c = reinterpret_cast<O*>(p.c) + row * p.ldc + col;
      if (r0 + l16 < last) {
        if (col + 4 <= p.n) {
          typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
          typedef f32x4_t f32x4_a4 __attribute__((aligned(4)));
          if constexpr (sizeof(O) == 2) *reinterpret_cast<u32x2_a2*>(c) = u32x2_t{pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3])};
          else *reinterpret_cast<f32x4_a4*>(c) = acc;
        } else {
#pragma unroll
          for (int v = 0; v < 3; ++v)
            if (col + v < p.n) {
              if constexpr (sizeof(O) == 2) c[v] = (O)pack_bf16(acc[v], 0.f);
              else c[v] = acc[v];
            }
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v) sum[wid][l16][4 * g + v] = acc[v];
      __syncthreads();
      const int r = threadIdx.x >> 4, col = threadIdx.x & 15;
      if (r0 + r < last && n0 + col < p.n) {
        const float t = (sum[0][r][col] + sum[1][r][col]) + (sum[2][r][col] + sum[3][r][col]);
        O* c = reinterpret_cast<O*>(p.c) + (int64_t)(r0 + r) * p.ldc + n0 + col;
        if constexpr (sizeof(O) == 2) *c = (O)pack_bf16(t, 0.f);
        else *c = t;
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------ tiles through registers and LDS
// S x S tiles, four waves of S/2 x S/2, k tiles of 128 bytes a row at a pitch of
// 144 (16 rows' pieces fall on distinct banks), two of them; the next one's loads (64 x
// 64: the next two's) are under way while one is multiplied.
constexpr int kPitch = 144;

template <typename O, int S>
__global__ __launch_bounds__(256, S == 64 ? 3 : 2) void fp8_tile_kernel(Fp8Params p) {
  constexpr int W = S / 2, F = W / 32, N = S * 8 / 256, STAGE = 2 * S * kPitch, D = S == 64 ? 2 : 1;
  constexpr int OUT = 32 * (W + 16 / (int)sizeof(O)) * (int)sizeof(O);  // a wave's rows of C on their way out
  static_assert(4 * OUT <= 2 * STAGE, "the waves' rows fit the k tiles' place");
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE];
  __shared__ Table T;
  const int tiles_n = (p.n + S - 1) / S, kb = p.k / 128;
  build_table(T, p, S, tiles_n, 0);
  zero_outside<O>(p, T.begin[0], T.begin[p.groups]);
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63, wm = (wid >> 1) * W, wn = (wid & 1) * W;
  const int items = T.tile[p.groups];
  // neighbouring tiles to one XCD: blocks are dealt to the 8 of them in turn
  const int per = gridDim.x >> 3;
  for (int q = gridDim.x & 7 ? (int)blockIdx.x : ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3); q < items; q += gridDim.x) {
    const int e = group_of(T, p.groups, q), r0 = T.begin[e], M = T.begin[e + 1] - r0;
    int tm, tn;
    tile_of(q - T.tile[e], (M + S - 1) / S, tiles_n, tm, tn);
    const int m0 = tm * S, n0 = tn * S;
    const uint8_t *pa[N], *pb[N], *SA[F], *SB[F];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + 256 * i, r = idx >> 3, c = (idx & 7) * 16;
      pa[i] = p.a + (int64_t)(r0 + min(m0 + r, M - 1)) * p.lda + c;
      pb[i] = p.b + e * p.stride_b + (int64_t)min(n0 + r, p.n - 1) * p.ldb + c;
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
      SA[i] = p.sa + (int64_t)(r0 + min(m0 + wm + 32 * i + (lane & 31), M - 1)) * p.ldsa;
      SB[i] = p.sb + e * p.stride_sb + (int64_t)(min(n0 + wn + 32 * i, p.n - 1) >> 7) * p.ldsb;
    }
    u32x4_t va[D][N], vb[D][N];
    int ca[D][F], cb[D][F], sa[F], sb[F];
    auto load = [&](int d, int kt) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        va[d][i] = *reinterpret_cast<const u32x4_t*>(pa[i] + kt * 128);
        vb[d][i] = *reinterpret_cast<const u32x4_t*>(pb[i] + kt * 128);
      }
#pragma unroll
      for (int i = 0; i < F; ++i) {
        ca[d][i] = SA[i][kt];
        cb[d][i] = SB[i][kt];
      }
    };
    auto store = [&](int d, uint8_t* st) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int idx = threadIdx.x + 256 * i, o = (idx >> 3) * kPitch + (idx & 7) * 16;
        *reinterpret_cast<u32x4_t*>(st + o) = va[d][i];
        *reinterpret_cast<u32x4_t*>(st + S * kPitch + o) = vb[d][i];
      }
#pragma unroll
      for (int i = 0; i < F; ++i) {
        sa[i] = ca[d][i];
        sb[i] = cb[d][i];
      }
    };
    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    bool bad[F][F] = {};
    load(0, 0);
    if (D == 2 && kb > 1) load(D - 1, 1);
    store(0, smem);
    if (D == 2 && kb > 2) load(0, 2);
    __syncthreads();
    // k tile kt is in LDS, kt + 1 (and, two deep, kt + 2) under way
    auto step = [&](int kt, auto parity) {
      constexpr int P = decltype(parity)::value, NEXT = D == 2 ? 1 - P : 0;
      int ta[F], tb[F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        ta[i] = sa[i];
        tb[i] = sb[i];
      }
      if (D == 1 && kt + 1 < kb) load(0, kt + 1);
      const uint8_t* st = smem + (kt & 1) * STAGE;
      const uint8_t* la = st + (wm + (lane & 31)) * kPitch + 32 * (lane >> 5);
      const uint8_t* lb = st + (S + wn + (lane & 31)) * kPitch + 32 * (lane >> 5);
      auto frag = [&](const uint8_t* q, int i, int s) {
        const i32x4* f = reinterpret_cast<const i32x4*>(q + i * 32 * kPitch + 64 * s);
        return join8(f[0], f[1]);
      };
      if constexpr (sizeof(O) == 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          i32x8 fa[F], fb[F];
#pragma unroll
          for (int i = 0; i < F; ++i) {
            fa[i] = frag(la, i, s);
            fb[i] = frag(lb, i, s);
          }
#pragma unroll
          for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 0, 0, 0, tb[j], 0, ta[i]);
        }
      } else {
        // lane l widens the 8 values from 32 (l / 32) + 8 t on: the same places of k in both operands
        f32x16 part[F][F];
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) part[i][j][v] = 0.f;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          i32x8 fa[F], fb[F];
#pragma unroll
          for (int i = 0; i < F; ++i) {
            fa[i] = frag(la, i, s);
            fb[i] = frag(lb, i, s);
          }
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            bf16x8 xa[F], xb[F];
#pragma unroll
            for (int i = 0; i < F; ++i) {
              xa[i] = widen(fa[i][2 * t], fa[i][2 * t + 1]);
              xb[i] = widen(fb[i][2 * t], fb[i][2 * t + 1]);
            }
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
              for (int j = 0; j < F; ++j)
                part[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xb[j], xa[i], part[i][j], 0, 0, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j) {
            const int ex = ta[i] + tb[j] - 254;
            bad[i][j] |= ta[i] == 255 || tb[j] == 255;
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] += __builtin_ldexpf(part[i][j][v], ex);
          }
      }
      if (kt + 1 < kb) store(NEXT, smem + (~kt & 1) * STAGE);
      if (D == 2 && kt + 3 < kb) load(NEXT, kt + 3);
      __syncthreads();
    };
    if constexpr (D == 2) {
      for (int kt = 0; kt < kb; kt += 2) {
        step(kt, std::integral_constant<int, 0>());
        if (kt + 1 < kb) step(kt + 1, std::integral_constant<int, 1>());
      }
    } else {
      for (int kt = 0; kt < kb; ++kt) step(kt, std::integral_constant<int, 0>());
    }
    if constexpr (sizeof(O) == 4)
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
          if (bad[i][j])
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = __builtin_nanf("");
    O* c = reinterpret_cast<O*>(p.c) + (int64_t)r0 * p.ldc;
    O* stage = reinterpret_cast<O*>(smem + wid * OUT);
#pragma unroll
    for (int i = 0; i < F; ++i)
      store_rows<W, O>(acc[i], stage, c, p.ldc, m0 + wm + 32 * i, M, n0 + wn, p.n);
    __syncthreads();  // the k tiles' place is free
  }
}

// ------------------------------------------------------------ 256 x 256 tiles
// Eight waves of 128 x 64, one persistent block a unit.  Operands go from memory
// straight to LDS, two k tiles of 128 (64 KB each); a load instruction writes its
// wave's 64 x 16 bytes in lane order, eight rows of 128 bytes, and the 16-byte piece
// c of row r lies at c ^ swizzle(r), so 16 rows' pieces fall on distinct banks (r & 7
// instead: half of LDS's time goes into bank conflicts).
//
// Waves 0-3 and 4-7 take turns: in one the first group reads its operands of k tile
// kt from LDS while the second multiplies kt - 1 from registers, in the next they
// change.  A group's results leave in a turn of their own, in which the other
// multiplies or reads; the k tiles of a block's items follow each other without a
// gap.  Loads are issued between the matrix instructions, where they cost no time:
//   second group, multiplying kt: all of B's kt + 2, whose place both have read
//   first group, multiplying kt:  the second's half of A's kt + 1, then its own of kt + 2
// and have at least a turn to land.  Loads and stores of a wave are counted together,
// in order: N stores under way between them let a wait leave N more.
// (Loads before the matrix instructions: 8192 x 8192 x 8192 440 us, between them 389.
// 32768 rows, 32 experts of 4096 x 1024, 268 MB of results: 182 us with all waiting
// for the stores, 155 with stores that pass the caches by.)
constexpr int kSide = 256, kHalf = 32 * 1024, kStage = 2 * kHalf;  // bytes of an operand's part, of a k tile
constexpr int kLargeK = 4;                                         // k tiles it takes at least
typedef __attribute__((address_space(3))) void* lds_ptr;
__device__ __forceinline__ int swizzle(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}

// LDS accesses are written out, reads with their wait in the same block: the compiler
// takes any it sees to depend on the loads to LDS under way and would wait for them.
__device__ __forceinline__ int lds_int(const int* p) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(lds_address(p)) : "memory");
  return v;
}

// Two row tiles of 32 (4096 bytes apart), both halves of the k tile: at[s][q] is the
// lane's address of piece q of half s.
template <int OFF>
__device__ __forceinline__ void read_two(i32x8 (&f)[2][2], const uint32_t (&at)[2][2]) {
  i32x4 x[8];
  asm volatile(
      "ds_read_b128 %0, %8 offset:%c12\n\t"
      "ds_read_b128 %1, %9 offset:%c12\n\t"
      "ds_read_b128 %2, %8 offset:%c13\n\t"
      "ds_read_b128 %3, %9 offset:%c13\n\t"
      "ds_read_b128 %4, %10 offset:%c12\n\t"
      "ds_read_b128 %5, %11 offset:%c12\n\t"
      "ds_read_b128 %6, %10 offset:%c13\n\t"
      "ds_read_b128 %7, %11 offset:%c13\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
      : "v"(at[0][0]), "v"(at[0][1]), "v"(at[1][0]), "v"(at[1][1]), "n"(OFF), "n"(OFF + 4096)
      : "memory");
  f[0][0] = join8(x[0], x[1]);
  f[0][1] = join8(x[2], x[3]);
  f[1][0] = join8(x[4], x[5]);
  f[1][1] = join8(x[6], x[7]);
}

// What hangs on it is computed where it is used, not kept in registers over the loop
// (which has none left).
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The kernel's arguments, read again where they are used between items: kept in
// scalar registers over the loop they would push its own out.
typedef const __attribute__((address_space(4))) Fp8Params* Args;
__device__ __forceinline__ Args args() {
  Args a = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(a));
  return a;
}

// A tile of C, and its operands as buffers: rows past the end read as zeros.
struct LItem {
  int e, row0, rows, n0;  // rows: of the group from row0 on
  const uint8_t *a, *b;
  int na, nb;  // bytes
};

struct Large {
  const Table& T;
  uint8_t* smem;
  int kb, wid, wm, wn, lda, ldb, q;
  uint32_t oa[2], ob[2];  // this lane's offsets in even and odd groups of eight rows
  uint32_t at[2][2];      // of its pieces of row lane % 32 of a part, in LDS

  __device__ __forceinline__ Large(const Fp8Params& p, const Table& T_, uint8_t* s) : T(T_), smem(s) {
    const int lane = threadIdx.x & 63, r = lane & 31;
    kb = p.k / 128;
    lda = (int)p.lda;
    ldb = (int)p.ldb;
    q = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);  // the grid is a multiple of 8
    wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = (wid >> 2) * 128;
    wn = (wid & 3) * 64;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int piece = ((lane & 7) ^ swizzle(8 * j + (lane >> 3))) * 16;
      oa[j] = (uint32_t)((lane >> 3) * lda + piece);
      ob[j] = (uint32_t)((lane >> 3) * ldb + piece);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        at[s][j] = lds_address(smem) + r * 128 + ((4 * s + 2 * (lane >> 5) + j) ^ swizzle(r)) * 16;
  }
  // The block's next item; false: there is none, and `it` stays.
  __device__ __forceinline__ bool next(LItem& it) {
    const Args p = args();
    const int groups = p->groups, tiles_n = (p->n + kSide - 1) / kSide;
    if (q >= __builtin_amdgcn_readfirstlane(lds_int(&T.tile[groups]))) return false;
    // the last group whose first tile is not behind q: of every `step`-th one, then of those after it
    const int lane = threadIdx.x & 63, step = (groups + 63) >> 6;
    int e = 0;
    for (int s = step, base = 0;; s = 1) {
      const int i = base + lane * s;
      const int first = lds_int(&T.tile[min(i, groups)]);
      const uint64_t le = __ballot(i < groups && first <= q);
      e = base + (63 - __builtin_clzll(le)) * s;
      if (s == 1) break;
      base = e;
    }
    it.e = __builtin_amdgcn_readfirstlane(e);
    const int r0 = __builtin_amdgcn_readfirstlane(lds_int(&T.begin[it.e]));
    const int M = __builtin_amdgcn_readfirstlane(lds_int(&T.begin[it.e + 1])) - r0;
    int tm, tn;
    tile_of(q - __builtin_amdgcn_readfirstlane(lds_int(&T.tile[it.e])), (M + kSide - 1) / kSide, tiles_n, tm, tn);
    it.row0 = __builtin_amdgcn_readfirstlane(r0 + tm * kSide);
    it.rows = min(kSide, r0 + M - it.row0);
    it.n0 = __builtin_amdgcn_readfirstlane(tn * kSide);
    it.a = p->a + (int64_t)it.row0 * p->lda;
    it.b = p->b + it.e * p->stride_b + (int64_t)it.n0 * p->ldb;
    it.na = (it.rows - 1) * (int)p->lda + p->k;
    it.nb = (min(kSide, p->n - it.n0) - 1) * (int)p->ldb + p->k;
    q += gridDim.x;
    return true;
  }
  // eight rows of k tile kt of `it`, or past its last one of `nx`, to place `g`
  __device__ __forceinline__ void load_a(const LItem& it, const LItem& nx, int kt, int g, int j) const {
    const bool over = kt >= kb;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(over ? nx.a : it.a), 0, over ? nx.na : it.na, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(smem + (g & 1) * kStage + j * 1024), 16, oa[j & 1],
                                             (over ? kt - kb : kt) * 128 + 8 * j * lda, 0, 0);
  }
  __device__ __forceinline__ void load_b(const LItem& it, const LItem& nx, int kt, int g, int j) const {
    const bool over = kt >= kb;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(over ? nx.b : it.b), 0, over ? nx.nb : it.nb, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(smem + (g & 1) * kStage + kHalf + j * 1024), 16, ob[j & 1],
                                             (over ? kt - kb : kt) * 128 + 8 * j * ldb, 0, 0);
  }
};

// Scale bytes of four k tiles, of this lane's rows and its columns' tile.
struct Scales {
  int a[4], b;
  // from k tile kt on (at a row's end its last four: skip(kt) bits too early)
  __device__ __forceinline__ void load(const Large& L, const LItem& it, int kt) {
    typedef int int_a1 __attribute__((aligned(1)));
    const Args p = args();
    const int o = min(kt, L.kb - 4), r = here(threadIdx.x & 31), ldsa = (int)p->ldsa;
    const uint8_t* s = p->sa + (int64_t)it.row0 * ldsa + o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = *reinterpret_cast<const int_a1*>(s + (uint32_t)(min(L.wm + 32 * i + r, it.rows - 1) * ldsa));
    b = *reinterpret_cast<const int_a1*>(p->sb + it.e * p->stride_sb + (int64_t)(min(it.n0 + L.wn, p->n - 1) >> 7) * p->ldsb + o);
  }
  static __device__ __forceinline__ int skip(const Large& L, int kt) { return 8 * (kt - min(kt, L.kb - 4)); }
  __device__ __forceinline__ void shift(int bits) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = (int)((uint32_t)a[i] >> bits);
    b = (int)((uint32_t)b >> bits);
  }
  __device__ __forceinline__ void wait() {  // here, not behind what is issued next
    asm volatile("" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]), "+v"(b));
  }
};

// The two turns of k tile kt, the block's g-th.  FIRST: the item's first, before which
// up to 16 stores were issued after its loads.  cur: its lowest bytes are k tile
// kt - 1's; next: of the following four, or of the next item.
template <int GROUP, bool FIRST>
__device__ __forceinline__ void large_turns(f32x16 (&acc)[4][2], const Large& L, const LItem& it, const LItem& nx, int kt,
                                            int g, Scales& cur, Scales& next) {
  const int w = L.wid & 3;
  if (FIRST || (kt & 3) == 0) {
    cur = next;
    cur.shift(Scales::skip(L, kt));
  } else {
    cur.shift(8);
  }
  uint32_t a[2][2], b[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      a[s][j] = L.at[s][j] + ((g & 1) * kStage + L.wm * 128);
      b[s][j] = L.at[s][j] + ((g & 1) * kStage + kHalf + L.wn * 128);
    }
  i32x8 fb[2][2], f0[2][2], f1[2][2];
  read_two<0>(fb, b);
  read_two<0>(f0, a);
  read_two<8192>(f1, a);
  // B's kt + 1 has landed; the second group's half of A's kt (the first's of kt + 1 may be under way)
  if constexpr (GROUP == 1 && FIRST) asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
  else if constexpr (GROUP == 1) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  else if constexpr (FIRST) asm volatile("s_waitcnt vmcnt(20)" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if (kt + 1 == L.kb) next.load(L, nx, 0);
  else if ((kt & 3) == 3) next.load(L, it, kt + 1);
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[s][j], i < 2 ? f0[s][i] : f1[s][i - 2], acc[i][j],
                                                                   0, 0, 0, cur.b, 0, cur.a[i]);
      const int t = 4 * s + i;
      if constexpr (GROUP == 1) L.load_b(it, nx, kt + 2, g, 8 * w + t);
      else if (t < 4) L.load_a(it, nx, kt + 1, g + 1, 16 + 4 * w + t);
      else L.load_a(it, nx, kt + 2, g, 4 * w + t - 4);
      __builtin_amdgcn_sched_barrier(0);
    }
  __builtin_amdgcn_s_setprio(0);
  __builtin_amdgcn_sched_barrier(0);
  // the first group's half of A's kt + 1, which the loads of this turn follow
  if constexpr (GROUP == 0 && FIRST) asm volatile("s_waitcnt vmcnt(24)" ::: "memory");
  else if constexpr (GROUP == 0) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// A wave's 128 x 64 results, 32 rows at a time through its 4 KB of LDS (16-byte pieces
// swizzled as the operands'): 16 stores of whole 128-byte lines where C is aligned and
// the tile's columns are whole.  They pass the caches by: a launch has more than 16 MB of
// them (256 tiles, of the last column of tiles one column at least), and 32 MB is the
// size of all L2s.  (From registers, 32 bytes of a row at a time: 151 -> 186 us, past
// the caches 238.)
__device__ __forceinline__ void large_store(f32x16 (&acc)[4][2], const Large& L, const LItem& it, const uint8_t* stage) {
  const Args p = args();
  const int lane = here(threadIdx.x & 63), r = lane & 31, ldc = (int)p->ldc;
  uint16_t* c = reinterpret_cast<uint16_t*>(p->c) + (int64_t)it.row0 * p->ldc + it.n0;
  const bool whole = it.n0 + kSide <= p->n && p->ldc % 8 == 0 && p->ldc <= (1 << 21) && ((uintptr_t)p->c & 15) == 0;
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(c, 0, whole ? ((it.rows - 1) * ldc + kSide) * 2 : 0, 0x00020000);
  const uint32_t w = lds_address(stage) + r * 128 + swizzle(r) * 16 + 8 * (lane >> 5);
  const uint32_t rd0 = lds_address(stage) + (lane >> 3) * 128 + ((lane & 7) ^ (lane >> 4)) * 16, rd1 = rd0 ^ 64;
  const int row0 = L.wm + (lane >> 3), col = L.wn + (lane & 7) * 8, left = p->n - it.n0 - col;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const u32x2_t x = {pack_bf16(acc[i][j][4 * v], acc[i][j][4 * v + 1]), pack_bf16(acc[i][j][4 * v + 2], acc[i][j][4 * v + 3])};
        asm volatile("ds_write_b64 %0, %1" ::"v"(w ^ (64 * j + 16 * v)), "v"(x) : "memory");
      }
    u32x4_t x[4];  // a wave's accesses to LDS keep their order
    asm volatile(
        "ds_read_b128 %0, %4\n\t"
        "ds_read_b128 %1, %5 offset:1024\n\t"
        "ds_read_b128 %2, %4 offset:2048\n\t"
        "ds_read_b128 %3, %5 offset:3*1024\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3])
        : "v"(rd0), "v"(rd1)
        : "memory");
    if (whole) {  // rows past the group's end are past the buffer's
#pragma unroll
      for (int k = 0; k < 4; ++k)
        __builtin_amdgcn_raw_buffer_store_b128(x[k], rsrc, (row0 * ldc + col) * 2, (32 * i + 8 * k) * ldc * 2, 2);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = row0 + 32 * i + 8 * k;
        uint16_t* d = c + (int64_t)row * p->ldc + col;
        if (row < it.rows && left >= 8) *reinterpret_cast<u32x4_a2*>(d) = x[k];
        if (row < it.rows && left < 8)
#pragma unroll 1
          for (int t = 0; t < left; ++t) {
            uint32_t u;
            asm volatile("ds_read_u16 %0, %1\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(u)
                         : "v"((k & 1 ? rd1 : rd0) + 1024 * k + 2 * t)
                         : "memory");
            d[t] = (uint16_t)u;
          }
      }
    }
  }
  if (!whole) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // of another number
}

template <int GROUP>
__device__ __forceinline__ void large_group(Large& L, LItem it) {
  LItem nx = it;
  bool more = L.next(nx);
  int g = 0;
  Scales cur, next;
  next.load(L, it, 0);
  next.wait();
  if constexpr (GROUP == 1) __builtin_amdgcn_s_barrier();  // one turn behind
  for (;;) {
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    large_turns<GROUP, true>(acc, L, it, nx, 0, g, cur, next);
#pragma unroll 1
    for (int kt = 1; kt < L.kb; ++kt) large_turns<GROUP, false>(acc, L, it, nx, kt, g + kt, cur, next);
    g += L.kb;
    next.wait();
    // through the second group's half of A's last k tile, which both have read, and whose
    // place the first group loads again only when it next multiplies
    large_store(acc, L, it, L.smem + (g - 1 & 1) * kStage + kHalf / 2 + (L.wid & 3) * 4096);
    __builtin_amdgcn_s_barrier();
    if (!more) break;
    it = nx;
    more = L.next(nx);
  }
  if constexpr (GROUP == 0) __builtin_amdgcn_s_barrier();
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads past the last item
}

__global__ __launch_bounds__(512, 2) void fp8_large_kernel(Fp8Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  __shared__ Table T;
  build_table(T, p, kSide, (p.n + kSide - 1) / kSide, 0);
  zero_outside<uint16_t>(p, T.begin[0], T.begin[p.groups]);
  Large L(p, T, smem);
  LItem it = {};
  if (!L.next(it)) return;
  // the first k tile, and of the second what the turns before it do not load
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    L.load_a(it, it, 0, 0, 4 * L.wid + j);
    L.load_b(it, it, 0, 0, 4 * L.wid + j);
    L.load_b(it, it, 1, 1, 4 * L.wid + j);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) L.load_a(it, it, 1, 1, 2 * L.wid + j);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  if (L.wid >> 2) large_group<1>(L, it);
  else large_group<0>(L, it);
}

// ------------------------------------------------------------ launchers
// The host knows the mean of the groups' rows only, so the rules go by it.
// Without LDS up to 2 rows a group, and 128 x 128 tiles: bf16, 32 experts of 4096 x
// 1024, 16 rows 14.4 and 15.3 us, 60 rows 25.2 and 25.9, but 250 rows 29.2 and 26.1.
// Up to 16 rows where there is not one such tile a unit, since its waves share the
// contraction: 8 experts of 1024 x 4096, 64 rows 10.9 and 17.5 us, 128 rows 12.3 and
// 17.8; or in fp32, whose tiles widen rows that are not there: 200 rows 28.3 and 35.0.
// 256 x 256 from 256 rows (bf16, four k tiles, one tile a unit), and 128 x 128: 32 of
// 4096 x 1024, 32768 rows 134 and 243 us, 10000 rows 63 and 72; one of 4096 x 4096, 4096
// rows 60 and 79.  A last column of tiles that is nearly empty counts like the others: one of
// 1024, 32768 rows, 257 columns 25 and 28 us, 300 columns 30 and 27.5, 384 22 and 27.
// 128 x 128 where there is one a unit, and 64 x 64: 6000 rows 48 and 57 us; one of 2003
// x 1152, 1023 rows, 144 tiles, 14.1 and 10.4 us.  In fp32, whose widening and matrix
// instructions cost more than the weights' reading, not below 64 rows a group: 1000
// rows 48.7 and 37.0 us (bf16 27.3 and 27.9).
enum { STREAM = 0, SMALL = 1, MIDDLE = 2, LARGE = 3 };

int choose(int64_t rows, int k, int n, int groups, int out_dtype, int num_cu) {
  const int64_t avg = rows / groups;
  const bool wide = (rows / 128 + groups) * ((n + 127) / 128) >= num_cu;
  if (avg <= 2 || (avg <= 16 && (!wide || out_dtype == PMX_F32))) return STREAM;
  if (out_dtype == PMX_BF16 && avg >= 256 && n >= 256 && k >= 128 * kLargeK && (rows / 256) * ((n + 255) / 256) >= num_cu)
    return LARGE;
  return wide && !(out_dtype == PMX_F32 && avg <= 64) ? MIDDLE : SMALL;
}

template <typename O>
hipError_t launch(const Fp8Params& p, hipStream_t s) {
  const int cfg = choose(p.rows, p.k, p.n, p.groups, p.out_dtype, p.num_cu);
  if (cfg == STREAM) {
    // waves of 16 columns, or where there are not eight a unit four to as many
    const int slots = (int)std::min<int64_t>(p.groups, p.rows);  // groups that can have rows
    const int64_t waves = (int64_t)slots * ((p.n + 15) / 16);
    if (waves >= 8 * (int64_t)p.num_cu) {
      const int blocks = (p.n + 63) / 64;
      fp8_stream_kernel<O, 1><<<dim3((unsigned)(blocks * slots)), 256, 0, s>>>(p, blocks);
    } else {
      const int blocks = (p.n + 15) / 16;
      fp8_stream_kernel<O, 4><<<dim3((unsigned)(blocks * slots)), 256, 0, s>>>(p, blocks);
    }
  } else if (cfg == LARGE) {
    if constexpr (sizeof(O) == 2) fp8_large_kernel<<<dim3((unsigned)(p.num_cu / 8 * 8)), 512, 0, s>>>(p);
  } else {
    const int side = cfg == SMALL ? 64 : 128;
    const int64_t tiles = (p.rows / side + std::min<int64_t>(p.groups, p.rows)) * ((p.n + side - 1) / side);
    const dim3 grid((unsigned)std::min<int64_t>(tiles, p.num_cu * (cfg == SMALL ? 3 : 2)));
    if (cfg == SMALL) fp8_tile_kernel<O, 64><<<grid, 256, 0, s>>>(p);
    else fp8_tile_kernel<O, 128><<<grid, 256, 0, s>>>(p);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8(const Fp8Params& p, hipStream_t s) {
  return p.out_dtype == PMX_BF16 ? launch<uint16_t>(p, s) : launch<float>(p, s);
}

}  // namespace pmx
