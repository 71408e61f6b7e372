// Matrix products grouped by expert.  The rows of A (and of the outer form's
// B) are sorted by group; offsets[e] .. offsets[e + 1] are group e's rows and
// stay on the device.
//   product, trans_b: C[t][j] = sum_k A[t][k] B_e[j][k]     (NT)
//   product:          C[t][j] = sum_k A[t][k] B_e[k][j]     (NN)
//   outer:            C_e[i][j] = sum_t A[t][i] B[t][j]     (TN)
// NT is the forward pass of out x in weights, NN its input gradient, TN its
// weight gradient.
//
// Design (CDNA4):
//  * Every block builds the groups' row ranges and tile counts from the
//    offsets (one wave, scans), so a launch needs neither the host's knowledge
//    of the sizes nor a table kernel.  Offsets are clamped to [0, rows] and
//    made monotone, so no offset leads outside the matrices.
//  * bf16: v_mfma_f32_32x32x16_bf16, k tiles of 64, operands through LDS, double
//    buffered; the registers hold the loads of the tile after the next.  An
//    operand stored k-contiguous is staged as rows; one stored along its rows
//    or columns (NN's B, TN's A and B) is staged as it lies and read with LDS
//    transpose reads.  fp32: v_mfma_f32_32x32x2_f32, k tiles of 16 or
//    32.
//  * The MFMA operands are swapped (B first), so a lane ends with four
//    consecutive columns of one row of C: 8- and 16-byte pieces.
//  * Rows past a group's end are read from the group's last row (their results
//    are not stored); places past the contraction's end are zeros in both
//    operands, so whatever lies there (infinities, NaN) does not enter.
//  * Loads are 16 bytes at any element alignment; a piece over a row's end is
//    read as the row's last 16 bytes and shifted.
//  * Accumulation in fp32, one rounding at the end.  With too few tiles to fill
//    the card the contraction is cut into splits whose fp32 partial results are
//    joined in order by a second launch.
//
// Measured, 32768 bf16 rows, 32 experts of 4096 x 1024 (275 GFLOP): forward 293 us,
// 0.94 PFLOP/s; input gradient 295; weight gradient, which also writes 537 MB of
// fp32, 352 to 362 (393 to 409 one call at a time under a profiler), added to what is there 487, into bf16 322.  In the large
// tile's blocks the matrix cores are busy 58 to 66% of the time, 36 in the weight
// gradient.  Short groups, weight gradient: 16 rows an expert 136 us, 60 168, 200
// 182 (537 MB of results at a copy's rate: 106).  16 rows through 13 of the experts:
// 22 us for 107 MB of weights, 4.9 TB/s.  2011 fp32 rows, 7 experts of 1001 x 500
// (2 GFLOP): 33 to 38 us each way, matrix cores busy 62 to 64%.
#include <algorithm>

#include "pmx_groups.h"

namespace pmx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

enum Form : int { NT = 0, NN = 1, TN = 2 };
constexpr bool a_kc(int f) { return f != TN; }  // A stored with k contiguous
constexpr bool b_kc(int f) { return f == NT; }

constexpr int kCU = 256;

// Groups by their rows, for the outer form's persistent blocks: a tile's time
// goes with its group's rows, and tiles of equal time side by side, every other
// round of them dealt out backwards, leave a block 3% over the mean where the
// groups' own order leaves 16 (32 groups of uneven lengths, 8 tiles a block):
// 32768 rows, 32 experts of 4096 x 1024, 374 and 392 us instead of 385 and 425
// for two routings.  More than 64 groups keep their order.
__device__ __forceinline__ void order_groups(int (&order)[64], const Table& T, int groups) {
  if (threadIdx.x < 64) {
    const int e = threadIdx.x, n = e < groups ? T.begin[e + 1] - T.begin[e] : 0;
    int rank = 0;
    if (groups <= 64)
      for (int j = 0; j < groups; ++j) {
        const int m = __shfl(n, j);
        rank += m > n || (m == n && j < e);
      }
    if (e < groups && groups <= 64) order[rank] = e;
  }
  __syncthreads();
}

// ------------------------------------------------------------ loads
template <typename E>
__device__ __forceinline__ u32x4_t load16(const E* p) {
  if constexpr (sizeof(E) == 2) return *reinterpret_cast<const u32x4_a2*>(p);
  else return *reinterpret_cast<const u32x4_a4*>(p);
}

// Elements c .. c + 15 / sizeof(E) of a row of n elements, zeros past its end.
template <typename E>
__device__ __forceinline__ u32x4_t load_win(const E* row, int c, int n) {
  constexpr int VEC = 16 / (int)sizeof(E);
  u32x4_t v = {0u, 0u, 0u, 0u};
  if (c + VEC <= n) return load16(row + c);
  if (c >= n) return v;
  if (n >= VEC) {  // the row's last 16 bytes, moved down
    v = load16(row + n - VEC);
    const int sh = (c + VEC - n) * 8 * (int)sizeof(E);  // 16 .. 112 bits
    uint64_t lo = v[0] | ((uint64_t)v[1] << 32), hi = v[2] | ((uint64_t)v[3] << 32);
    if (sh >= 64) {
      lo = hi >> (sh - 64);
      hi = 0;
    } else {
      lo = (lo >> sh) | (hi << (64 - sh));
      hi >>= sh;
    }
    return {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < n) v[j >> 1] |= (uint32_t)row[c + j] << (16 * (j & 1));
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < n) v[j] = __float_as_uint(row[c + j]);
  }
  return v;
}

// ------------------------------------------------------------ tiles
// Block tile BM x BN x BK, wave tile WM x WN; LDS layout of an operand of
// `R` rows: k-contiguous [R][BK + 16 bytes], or [BK][pitch] as it lies.  The
// pitch of the transpose-read form is 8, 16 or 48 dwords modulo 64, which puts
// the four k rows of a read on distinct banks; fp32 reads rows of consecutive
// words (any pitch).
template <typename E_, int BM_, int BN_, int BK_, int WM_, int WN_, int MINB_>
struct Cfg {
  typedef E_ E;
  static constexpr int BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, MINB = MINB_;
  static constexpr int VEC = 16 / (int)sizeof(E);
  static constexpr int WAVES = (BM / WM) * (BN / WN), THREADS = 64 * WAVES;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int LDK = BK + VEC;
  static constexpr int pitch(int r) {
    return sizeof(E) == 2 ? (r == 32 ? 32 : r == 128 ? 144 : r + 32) : r + 4;
  }
  static constexpr int size(bool kc, int r) { return kc ? r * LDK : BK * pitch(r); }
};

template <class C, bool KC, int R>
struct Operand {
  typedef typename C::E E;
  static constexpr int N = R * C::BK / C::VEC / C::THREADS;  // 16-byte pieces a thread
  static_assert(N * C::THREADS * C::VEC == R * C::BK, "pieces a thread");
  static constexpr int PER = KC ? C::BK / C::VEC : R / C::VEC;  // pieces a stored row
  const E* ptr[N];   // the piece at k tile 0
  const E* base;     // the operand's origin (element k = 0, row or column 0)
  int64_t ld;
  int r0, limit;     // first row (column) of the tile, rows (columns) there are

  // KC: rows r0 .. r0 + R - 1 of `limit` rows, read past the end from the last
  // one.  Otherwise columns r0 .. of `limit`.
  __device__ __forceinline__ void init(const E* b, int64_t ld_, int r0_, int limit_) {
    base = b;
    ld = ld_;
    r0 = r0_;
    limit = limit_;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + C::THREADS * i, s = idx / PER, c = idx % PER * C::VEC;
      if (KC) {
        const int row = r0 + s < limit ? r0 + s : limit - 1;
        ptr[i] = base + (int64_t)row * ld + c;
      } else {
        ptr[i] = base + (int64_t)s * ld + r0 + c;
      }
    }
  }
  // whole k tile starting at k0; columns (not KC) all inside
  __device__ __forceinline__ void load(u32x4_t (&v)[N], int k0) const {
    const int64_t o = KC ? k0 : (int64_t)k0 * ld;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load16(ptr[i] + o);
  }
  // any k tile: zeros at k >= kend and past the last column
  __device__ __forceinline__ void load_edge(u32x4_t (&v)[N], int k0, int kend) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + C::THREADS * i, s = idx / PER, c = idx % PER * C::VEC;
      if (KC) {
        v[i] = load_win(ptr[i] - c, k0 + c, kend);
      } else {
        v[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (k0 + s < kend) v[i] = load_win(base + (int64_t)(k0 + s) * ld, r0 + c, limit);
      }
    }
  }
  __device__ __forceinline__ void store(E* lds, const u32x4_t (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + C::THREADS * i, s = idx / PER, c = idx % PER * C::VEC;
      *reinterpret_cast<u32x4_t*>(lds + s * (KC ? C::LDK : C::pitch(R)) + c) = v[i];
    }
  }
};

// bf16 fragment of 32 rows, 16 k: lane l has row l % 32, k = 8 (l / 32) .. + 7.
// Not KC: two transpose reads; in each group of 16 lanes, lane j receives
// element j % 4 of the 8 bytes addressed by lanes 4 t + j / 4 (t = 0 .. 3), so
// the lane addresses k row 8 (g / 2) + j / 4 (+ 4) and column 16 (g % 2) + 4 (j % 4).
template <class C, bool KC, int R>
__device__ __forceinline__ bf16x8 frag(const uint16_t* lds, int row, int s) {
  const int lane = threadIdx.x & 63;
  if constexpr (KC) {
    return *reinterpret_cast<const bf16x8*>(lds + (row + (lane & 31)) * C::LDK + (lane >> 5) * 8 + 16 * s);
  } else {
    constexpr int P = C::pitch(R);
    const int g = lane >> 4, j = lane & 15;
    const uint16_t* q = lds + (16 * s + 8 * (g >> 1) + (j >> 2)) * P + row + 16 * (g & 1) + 4 * (j & 3);
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)q);
    const i16x4 hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)(q + 4 * P));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// fp32: k = k0 + 8 (l / 32) + s for step s of 16 values of k.
template <class C, bool KC, int R>
__device__ __forceinline__ void frag(float (&f)[8], const float* lds, int row, int k0) {
  const int lane = threadIdx.x & 63;
  const int r = row + (lane & 31), k = k0 + (lane >> 5) * 8;
  if constexpr (KC) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(lds + r * C::LDK + k);
    const f32x4_t x = q[0], y = q[1];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      f[s] = x[s];
      f[4 + s] = y[s];
    }
  } else {
#pragma unroll
    for (int s = 0; s < 8; ++s) f[s] = lds[(k + s) * C::pitch(R) + r];
  }
}

// acc += the staged k tile.
template <class C, int FORM>
__device__ __forceinline__ void multiply(f32x16 (&acc)[C::FM][C::FN], const typename C::E* sa,
                                         const typename C::E* sb, int wm, int wn) {
  if constexpr (sizeof(typename C::E) == 2) {
    constexpr int STEPS = C::BK / 16;
    bf16x8 fa[2][C::FM], fb[2][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i) fa[0][i] = frag<C, a_kc(FORM), C::BM>(sa, wm + 32 * i, 0);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) fb[0][j] = frag<C, b_kc(FORM), C::BN>(sb, wn + 32 * j, 0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int c = s & 1, n = c ^ 1;
      if (s + 1 < STEPS) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i) fa[n][i] = frag<C, a_kc(FORM), C::BM>(sa, wm + 32 * i, s + 1);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) fb[n][j] = frag<C, b_kc(FORM), C::BN>(sb, wn + 32 * j, s + 1);
      }
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[c][j], fa[c][i], acc[i][j], 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int k0 = 0; k0 < C::BK; k0 += 16) {
      float fa[C::FM][8], fb[C::FN][8];
#pragma unroll
      for (int i = 0; i < C::FM; ++i) frag<C, a_kc(FORM), C::BM>(fa[i], sa, wm + 32 * i, k0);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) frag<C, b_kc(FORM), C::BN>(fb[j], sb, wn + 32 * j, k0);
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j][s], fa[i][s], acc[i][j], 0, 0, 0);
    }
  }
}

// fp32 sums over long contractions: what has come together over kFold values of k
// goes to a second sum, so a result passes through kFold / 2 + K / kFold roundings
// instead of K / 2 (a matrix instruction adds two products).  64 rows, 64 experts
// of 1024 x 4096: 1.1e-6 relative in one chain, 2.3e-7 so.  The second sum's
// registers cost the 64 x 64 tile one of five waves a SIMD where it matters most,
// the weight gradient (8192 rows, 8 experts of 1024 x 1024: 147 -> 153 us; the
// products 152 -> 153 and 154 -> 155); folding every 256 takes as long, every 64
// 2% more.
constexpr int kFold = 128;
template <class C>
struct Fold {
  static constexpr bool ON = sizeof(typename C::E) == 4;
  f32x16 sum[ON ? C::FM : 1][ON ? C::FN : 1];
  __device__ __forceinline__ Fold() {
    if constexpr (ON)
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) sum[i][j][v] = 0.f;
  }
  // before k tile `n` of a block's share
  __device__ __forceinline__ void step(f32x16 (&acc)[C::FM][C::FN], int n) {
    if constexpr (ON)
      if (n > 0 && n % (kFold / C::BK) == 0)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              sum[i][j][v] += acc[i][j][v];
              acc[i][j][v] = 0.f;
            }
  }
  __device__ __forceinline__ void end(f32x16 (&acc)[C::FM][C::FN]) const {
    if constexpr (ON)
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] += sum[i][j][v];
  }
};

// Product of one tile over k tiles [kb, ke) of a contraction of `K`.
template <class C, int FORM, bool EDGE>
__device__ __forceinline__ void mainloop(f32x16 (&acc)[C::FM][C::FN], typename C::E* smem,
                                         const Operand<C, a_kc(FORM), C::BM>& A,
                                         const Operand<C, b_kc(FORM), C::BN>& B, int kb, int ke, int K,
                                         int wm, int wn) {
  constexpr int SA = C::size(a_kc(FORM), C::BM), SB = C::size(b_kc(FORM), C::BN);
  constexpr int ST = SA + SB;
  u32x4_t va[Operand<C, a_kc(FORM), C::BM>::N], vb[Operand<C, b_kc(FORM), C::BN>::N];
  const int nfull = EDGE ? 0 : K / C::BK;
  auto load = [&](int kt) {
    if (kt < nfull) {
      A.load(va, kt * C::BK);
      B.load(vb, kt * C::BK);
    } else {
      A.load_edge(va, kt * C::BK, K);
      B.load_edge(vb, kt * C::BK, K);
    }
  };
  load(kb);
  A.store(smem, va);
  B.store(smem + SA, vb);
  if (kb + 1 < ke) load(kb + 1);
  __syncthreads();
  Fold<C> fold;
  for (int kt = kb; kt < ke; ++kt) {
    fold.step(acc, kt - kb);
    const int cur = (kt - kb) & 1;
    typename C::E* s = smem + cur * ST;
    typename C::E* d = smem + (cur ^ 1) * ST;
    multiply<C, FORM>(acc, s, s + SA, wm, wn);
    if (kt + 1 < ke) {
      A.store(d, va);
      B.store(d + SA, vb);
      if (kt + 2 < ke) load(kt + 2);
    }
    __syncthreads();
  }
  fold.end(acc);
}

// ------------------------------------------------------------ pipelined tiles
// The middle and large tiles.  Operand pieces are a base that is the same for
// the block and a 32-bit offset a piece; a k tile's whole pieces only (the rest
// of the contraction follows by itself), k rows and tile rows in range.
template <class C, bool KC, int R>
struct Stream {
  typedef typename C::E E;
  typedef Operand<C, KC, R> O;
  static constexpr int N = O::N, PER = O::PER, VEC = C::VEC;
  const E* base;
  int64_t step;      // elements a k tile
  uint32_t off[N];
  int r0, limit;     // as Operand
  int64_t ld;

  // limit >= VEC when not KC: the piece over the last column is read as the
  // last VEC columns
  __device__ __forceinline__ void init(const E* b, int64_t ld_, int r0_, int limit_) {
    r0 = r0_;
    limit = limit_;
    ld = ld_;
    base = KC ? b + (int64_t)r0 * ld : b;
    step = KC ? C::BK : (int64_t)C::BK * ld;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + C::THREADS * i, s = idx / PER, c = idx % PER * VEC;
      off[i] = KC ? (uint32_t)(min(s, limit - 1 - r0) * (int)ld + c)
                  : (uint32_t)(s * (int)ld + min(r0 + c, limit - VEC));
    }
  }
  __device__ __forceinline__ void load(u32x4_t (&v)[N], int kt) const {
    const E* p = base + kt * step;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = load16(p + off[i]);
  }
  // EDGE: a piece that was moved down to the last VEC columns goes to their
  // places by element (columns past the last hold anything)
  template <bool EDGE>
  __device__ __forceinline__ void store(E* lds, const u32x4_t (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + C::THREADS * i, s = idx / PER, c = idx % PER * VEC;
      E* d = lds + s * (KC ? C::LDK : C::pitch(R)) + c;
      if (!EDGE || KC || r0 + c + VEC <= limit) {
        *reinterpret_cast<u32x4_t*>(d) = v[i];
      } else if (r0 + c < limit) {
        const int sh = r0 + c + VEC - limit;  // 1 .. VEC - 1
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c - sh + j >= 0) {
            if constexpr (sizeof(E) == 2) d[j - sh] = (E)(v[i][j >> 1] >> (16 * (j & 1)));
            else d[j - sh] = __uint_as_float(v[i][j]);
          }
      }
    }
  }
  // the last k tile: zeros at k >= kend, piece by piece
  __device__ __forceinline__ void tail(E* lds, int k0, int kend) const {
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + C::THREADS * i, s = idx / PER, c = idx % PER * VEC;
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (KC) v = load_win(base + (int64_t)min(s, limit - 1 - r0) * ld, k0 + c, kend);
      else if (k0 + s < kend) v = load_win(base + (int64_t)(k0 + s) * ld, r0 + c, limit);
      *reinterpret_cast<u32x4_t*>(lds + s * (KC ? C::LDK : C::pitch(R)) + c) = v;
    }
  }
};

// Scheduling groups: MF MFMAs, each followed by up to PER instructions of class
// MASK (0x100 LDS read, 0x200 LDS write) until OPS are placed.
template <int MF, int OPS, int MASK, int PER>
__device__ __forceinline__ void interleave() {
  if constexpr (MF > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    constexpr int k = OPS < PER ? OPS : PER;
    if constexpr (k > 0) __builtin_amdgcn_sched_group_barrier(MASK, k, 0);
    interleave<MF - 1, OPS - k, MASK, PER>();
  } else if constexpr (OPS > 0) {
    __builtin_amdgcn_sched_group_barrier(MASK, OPS, 0);
  }
}

// k tiles [kb, ke) of whole pieces; on entry va[d], vb[d] hold k tile kb + d (the
// last one where there are fewer).  A k tile is one block of instructions: its
// fragments are read a 16-wide step ahead of the MFMAs, the next tile goes from
// the registers to the other LDS buffer under the last step's, and the loads of
// the tile D after that are issued before the barrier.
template <class C, int FORM, bool EDGE, int D>
__device__ __forceinline__ void stream_loop(f32x16 (&acc)[C::FM][C::FN], typename C::E* smem,
                                            const Stream<C, a_kc(FORM), C::BM>& A,
                                            const Stream<C, b_kc(FORM), C::BN>& B,
                                            u32x4_t (&va)[D][Stream<C, a_kc(FORM), C::BM>::N],
                                            u32x4_t (&vb)[D][Stream<C, b_kc(FORM), C::BN>::N], int kb, int ke,
                                            int wm, int wn) {
  constexpr int SA = C::size(a_kc(FORM), C::BM), ST = SA + C::size(b_kc(FORM), C::BN);
  constexpr int NA = Stream<C, a_kc(FORM), C::BM>::N, NB = Stream<C, b_kc(FORM), C::BN>::N;
  A.template store<EDGE>(smem, va[0]);
  B.template store<EDGE>(smem + SA, vb[0]);
  A.load(va[0], min(kb + D, ke - 1));  // past the last tile: the last one again
  B.load(vb[0], min(kb + D, ke - 1));
  __syncthreads();
  static_assert(!Fold<C>::ON || kFold / C::BK % D == 0, "folds between steps");
  Fold<C> fold;
  for (int k0 = kb; k0 < ke; k0 += D) {
    fold.step(acc, k0 - kb);
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (i > 0 && k0 + i >= ke) break;
      const int n = (i + 1) % D;
      const int cur = D % 2 ? (k0 - kb) & 1 : i & 1;
      typename C::E* s = smem + cur * ST;
      typename C::E* d = smem + (cur ^ 1) * ST;
      multiply<C, FORM>(acc, s, s + SA, wm, wn);
      A.template store<EDGE>(d, va[n]);
      B.template store<EDGE>(d + SA, vb[n]);
      const int kn = min(k0 + i + 1 + D, ke - 1);
      A.load(va[n], kn);
      B.load(vb[n], kn);
      if constexpr (!EDGE && sizeof(typename C::E) == 2) {
        constexpr int MF = C::FM * C::FN, STEPS = C::BK / 16;
        constexpr int NF = C::FM * (a_kc(FORM) ? 1 : 2) + C::FN * (b_kc(FORM) ? 1 : 2);
        __builtin_amdgcn_sched_group_barrier(0x100, NF, 0);
#pragma unroll
        for (int st = 0; st + 1 < STEPS; ++st) interleave<MF, NF, 0x100, (NF + MF - 1) / MF>();
        interleave<MF, NA + NB, 0x200, (NA + NB + MF - 1) / MF>();
        __builtin_amdgcn_sched_group_barrier(0x020, NA + NB, 0);
      }
      __syncthreads();
    }
  }
  fold.end(acc);
}

// The same for the large bf16 tile, whose 8 waves are two to a SIMD: the two
// groups of four waves take turns.  While one runs the MFMAs of half a k tile
// (16 a wave, all operands in registers), the other reads its next half's
// fragments from LDS, puts its pieces of the next k tile there and issues its
// global loads; a barrier ends each turn.  The matrix cores of a SIMD thus
// have one wave's MFMAs to issue at any time, instead of both waves waiting for
// LDS at the same place.
template <class C, int FORM, bool EDGE>
__device__ __forceinline__ void turns_loop(f32x16 (&acc)[C::FM][C::FN], typename C::E* smem,
                                           const Stream<C, a_kc(FORM), C::BM>& A,
                                           const Stream<C, b_kc(FORM), C::BN>& B,
                                           u32x4_t (&va)[Stream<C, a_kc(FORM), C::BM>::N],
                                           u32x4_t (&vb)[Stream<C, b_kc(FORM), C::BN>::N], int kb, int ke,
                                           int wm, int wn, int group) {
  constexpr int SA = C::size(a_kc(FORM), C::BM), ST = SA + C::size(b_kc(FORM), C::BN);
  static_assert(C::WAVES == 8 && C::BK == 64 && sizeof(typename C::E) == 2, "two waves a SIMD");
  A.template store<EDGE>(smem, va);
  B.template store<EDGE>(smem + SA, vb);
  {
    const int k1 = min(kb + 1, ke - 1);  // past the last tile: the last one again
    A.load(va, k1);
    B.load(vb, k1);
  }
  __syncthreads();
  // the second group is one turn behind
  if (group) __builtin_amdgcn_s_barrier();
  for (int kt = kb; kt < ke; ++kt) {
    const int cur = (kt - kb) & 1;
    const typename C::E* s = smem + cur * ST;
    typename C::E* d = smem + (cur ^ 1) * ST;
    const int k2 = min(kt + 2, ke - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // this turn's operands; half of the next k tile on its way.  (The other
      // buffer's last reader, the second group's turn before the first group's
      // present one, is done; its next reader is four turns away.)
      bf16x8 fa[2][C::FM], fb[2][C::FN];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i) fa[t][i] = frag<C, a_kc(FORM), C::BM>(s, wm + 32 * i, 2 * h + t);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) fb[t][j] = frag<C, b_kc(FORM), C::BN>(s + SA, wn + 32 * j, 2 * h + t);
      }
      if (h == 0) {
        A.template store<EDGE>(d, va);
        A.load(va, k2);
      } else {
        B.template store<EDGE>(d + SA, vb);
        B.load(vb, k2);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[t][j], fa[t][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (!group) __builtin_amdgcn_s_barrier();
}

// Four columns of a row of C at c (row length n): plain, or added to.
template <typename O>
__device__ __forceinline__ void put4(O* row, int c, int n, f32x4_t v, bool add) {
  if (c + 4 <= n) {
    if constexpr (sizeof(O) == 4) {
      typedef f32x4_t f32x4_a4 __attribute__((aligned(4)));
      f32x4_a4* q = reinterpret_cast<f32x4_a4*>(row + c);
      if (add) v += *q;
      *q = v;
    } else {
      typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
      u32x2_a2* q = reinterpret_cast<u32x2_a2*>(row + c);
      if (add) {
        const u32x2_t o = *q;
        v += f32x4_t{bf16_lo(o[0]), bf16_hi(o[0]), bf16_lo(o[1]), bf16_hi(o[1])};
      }
      *q = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (c + j < n) {
        if constexpr (sizeof(O) == 4) row[c + j] = add ? row[c + j] + v[j] : v[j];
        else
          row[c + j] = (O)pack_bf16(add ? v[j] + __uint_as_float((uint32_t)row[c + j] << 16) : v[j], 0.f);
      }
  }
}

// Rows of no group are zeros.
template <class C, typename O, bool SPLIT>
__device__ __forceinline__ void zero_outside(const Table& T, const GroupedParams& p, int splits) {
  const int b0 = T.begin[0], b1 = T.begin[p.groups], outside = b0 + (int)p.rows - b1;
  for (int i = blockIdx.x; i < outside; i += gridDim.x) {
    const int64_t row = i < b0 ? i : b1 + (i - b0);
    for (int c = threadIdx.x * 4; c < p.n; c += C::THREADS * 4) {
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
      if constexpr (SPLIT) {
        for (int s = 0; s < splits; ++s)
          put4<float>(p.part + ((int64_t)s * p.rows + row) * p.n, c, p.n, zero, false);
      } else {
        put4<O>(reinterpret_cast<O*>(p.c) + row * p.ldc, c, p.n, zero, false);
      }
    }
  }
}

// O: element of C (float or bf16 bits); SPLIT: fp32 partial results to p.part.
template <class C, int FORM, typename O, bool SPLIT>
__global__ __launch_bounds__(C::THREADS, C::MINB) void grouped_kernel(GroupedParams p) {
  typedef typename C::E E;
  constexpr int ST = C::size(a_kc(FORM), C::BM) + C::size(b_kc(FORM), C::BN);
  __shared__ __attribute__((aligned(16))) E smem[2 * ST];
  __shared__ Table T;
  const int tiles_n = (p.n + C::BN - 1) / C::BN;
  const int tiles_m = FORM == TN ? (p.m + C::BM - 1) / C::BM : 0;
  build_table(T, p, C::BM, tiles_n, FORM == TN ? tiles_m * tiles_n : 0);
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  constexpr int WGN = C::BN / C::WN;
  const int wm = wid / WGN * C::WM, wn = wid % WGN * C::WN;
  const int splits = SPLIT ? p.splits : 1;
  const int64_t part_ld = p.n;

  if constexpr (FORM != TN) zero_outside<C, O, SPLIT>(T, p, splits);

  // Blocks are dealt to the 8 XCDs round-robin: XCD x takes a contiguous range
  // of the items, so neighbouring tiles share its L2.
  const int items = T.tile[p.groups] * splits;
  const int per = (items + 7) >> 3, x = blockIdx.x & 7, step = gridDim.x >> 3;
  for (int jx = blockIdx.x >> 3; jx < per; jx += step) {
    const int it = x * per + jx;
    if (it >= items) break;
    const int t = SPLIT ? it / splits : it, sp = SPLIT ? it - t * splits : 0;
    const int e = group_of(T, p.groups, t);
    const int r0 = T.begin[e], nr = T.begin[e + 1] - r0;
    int tm, tn;
    tile_of(t - T.tile[e], FORM == TN ? tiles_m : (nr + C::BM - 1) / C::BM, tiles_n, tm, tn);
    const int m0 = tm * C::BM, n0 = tn * C::BN;
    const int K = FORM == TN ? nr : p.k;
    const int M = FORM == TN ? p.m : nr;
    const int nk = (K + C::BK - 1) / C::BK;
    const int kb = SPLIT ? (int)((int64_t)nk * sp / splits) : 0;
    const int ke = SPLIT ? (int)((int64_t)nk * (sp + 1) / splits) : nk;
    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    if (kb < ke) {
      const E* a = reinterpret_cast<const E*>(p.a) + (int64_t)r0 * p.lda;
      const E* b = reinterpret_cast<const E*>(p.b) +
                   (FORM == TN ? (int64_t)r0 * p.ldb : (int64_t)e * p.stride_b);
      Operand<C, a_kc(FORM), C::BM> A;
      Operand<C, b_kc(FORM), C::BN> B;
      A.init(a, p.lda, m0, M);
      B.init(b, p.ldb, n0, p.n);
      // columns of an operand that is not k-contiguous past its end
      const bool edge = (!a_kc(FORM) && m0 + C::BM > M) || (!b_kc(FORM) && n0 + C::BN > p.n);
      if (edge) mainloop<C, FORM, true>(acc, smem, A, B, kb, ke, K, wm, wn);
      else mainloop<C, FORM, false>(acc, smem, A, B, kb, ke, K, wm, wn);
    }
    // lane l has row l % 32; register v column 8 (v / 4) + 4 (l / 32) + v % 4
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int row = m0 + wm + 32 * i + (lane & 31);
      if (row >= M) continue;
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int col = n0 + wn + 32 * j + 8 * g + 4 * (lane >> 5);
          if (col >= p.n) continue;
          const f32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                             acc[i][j][4 * g + 3]};
          if constexpr (SPLIT) {
            float* q = FORM == TN ? p.part + (((int64_t)sp * p.groups + e) * M + row) * part_ld
                                  : p.part + ((int64_t)sp * p.rows + r0 + row) * part_ld;
            put4<float>(q, col, p.n, v, false);
          } else {
            O* q = reinterpret_cast<O*>(p.c) +
                   (FORM == TN ? (int64_t)e * p.stride_c + (int64_t)row * p.ldc
                               : (int64_t)(r0 + row) * p.ldc);
            put4<O>(q, col, p.n, v, FORM == TN && p.accumulate);
          }
        }
    }
  }
}

// k tiles on their way in registers.  The tiles up to 64 rows keep two; the
// middle one has no registers left for a second: 112 us instead of 101 (5075
// bf16 rows, 17 experts of 1075 x 289, a step).
template <class C>
constexpr int kDepth = C::BM <= 64 ? 2 : 1;

// Blocks a compute unit, and items of a window (0: as many as blocks).  The
// larger tiles are persistent.  Of the others two to five fit a unit, the
// hardware deals out more as they end, and windows of 256 items keep groups of
// unequal length from piling up on one XCD.  (fp32, 8 experts of 1024 x 1024,
// 8192 rows, weight gradient: 183 us, 309 with one window; bf16, 32 of 4096 x
// 1024, 256 rows, input gradient: 50 us, 66 with three persistent blocks a unit.)
template <class C>
constexpr int kBlocks = C::BM <= 64 ? 8 : C::MINB;
template <class C>
constexpr int kWindow = C::BM <= 64 ? 256 : 0;

template <class C>
constexpr bool kTurns = C::WAVES == 8 && C::BK == 64 && sizeof(typename C::E) == 2;

// The large tiles that the large tiles' launch runs: whole rounds of them where
// quarters of the rest find a unit each, which a second launch gives them, and
// the contraction is long enough to pay for that.  (16384 rows, 8 experts of
// 2048 x 2048, 2.16 rounds: forward 160 -> 149 us, input gradient 180 -> 162;
// 32768 rows, 32 of 4096 x 1024: input gradient, k = 4096, 2.23 rounds, 343 -> 304,
// but forward, k = 1024, 9.06 rounds, 327 -> 338.)
constexpr int kLarge = 256, kQuartersK = 2048;
__device__ __forceinline__ int whole_rounds(int items, int round, int k) {
  const int rest = items % round;
  return k >= kQuartersK && rest * 4 <= round ? items - rest : items;
}

// The same products on pipelined tiles.  Blocks are persistent: the first k
// tile of a block's next item is loaded before the item's results are stored.
// QUARTERS: the large tiles after the whole rounds, as 128 x 128 ones, a block a
// unit with four k tiles on their way (two blocks a unit and two k tiles: 165 and
// 178 us where this takes 150 and 161).
template <class C, int FORM, typename O, bool SPLIT, bool QUARTERS = false>
__global__ __launch_bounds__(C::THREADS, C::MINB * C::WAVES / 4) void grouped_tile_kernel(GroupedParams p) {
  typedef typename C::E E;
  constexpr bool AK = a_kc(FORM), BK_ = b_kc(FORM);
  constexpr int SA = C::size(AK, C::BM), ST = SA + C::size(BK_, C::BN);
  // two k tiles; the waves' 32-row stages of C take their place
  constexpr int STAGE = 32 * (C::WN + 16 / (int)sizeof(O)) * (int)sizeof(O);
  constexpr int LDS = STAGE * C::WAVES / (int)sizeof(E) > 2 * ST ? STAGE * C::WAVES / (int)sizeof(E) : 2 * ST;
  __shared__ __attribute__((aligned(16))) E smem[LDS];
  __shared__ Table T;
  constexpr int TM = QUARTERS ? kLarge : C::BM, TN_ = QUARTERS ? kLarge : C::BN;  // of the table's tiles
  const int tiles_n = (p.n + TN_ - 1) / TN_;
  const int tiles_m = FORM == TN ? (p.m + TM - 1) / TM : 0;
  build_table(T, p, TM, tiles_n, FORM == TN ? tiles_m * tiles_n : 0);
  const int wid = threadIdx.x >> 6;
  constexpr int WGN = C::BN / C::WN;
  const int wm = wid / WGN * C::WM, wn = wid % WGN * C::WN;
  const int splits = SPLIT ? p.splits : 1;
  if constexpr (FORM != TN && !QUARTERS) zero_outside<C, O, SPLIT>(T, p, splits);

  // Blocks are dealt to the 8 XCDs round-robin.  Each window of items gives every
  // XCD a contiguous share, neighbouring tiles for its L2, and the windows spread
  // long and short groups over all of them.
  int items = T.tile[p.groups] * splits, first = 0;
  if constexpr (QUARTERS) {
    first = whole_rounds(items, p.round, p.k);
    items = (items - first) * 4;
  } else if constexpr (C::BM == kLarge && FORM != TN) {
    items = whole_rounds(items, gridDim.x, p.k);
  }
  const int window = kWindow<C> ? kWindow<C> : (int)gridDim.x, w0 = (int)blockIdx.x / window * window;
  const int size = min(window, (int)gridDim.x - w0), in = (int)blockIdx.x - w0;
  int q0 = w0 + (in & 7) * (size >> 3) + (in >> 3);
  struct Item {
    int e, r0, m0, n0, K, M, kb, ke, sp;
  };
  auto next = [&](Item& it) -> bool {
    if (q0 >= items) return false;
    const int q = q0;
    q0 += gridDim.x;
    const int t = QUARTERS ? first + q / 4 : SPLIT ? q / splits : q;
    it.sp = SPLIT ? q - t * splits : 0;
    it.e = group_of(T, p.groups, t);
    it.r0 = T.begin[it.e];
    const int nr = T.begin[it.e + 1] - it.r0;
    int tm, tn;
    tile_of(t - T.tile[it.e], FORM == TN ? tiles_m : (nr + TM - 1) / TM, tiles_n, tm, tn);
    it.m0 = tm * TM + (QUARTERS ? (q >> 1 & 1) * C::BM : 0);
    it.n0 = tn * TN_ + (QUARTERS ? (q & 1) * C::BN : 0);
    it.K = FORM == TN ? nr : p.k;
    it.M = FORM == TN ? p.m : nr;
    if (QUARTERS && (it.m0 >= it.M || it.n0 >= p.n)) return false;  // a block has no second one
    const int nk = (it.K + C::BK - 1) / C::BK;
    it.kb = SPLIT ? (int)((int64_t)nk * it.sp / splits) : 0;
    it.ke = SPLIT ? (int)((int64_t)nk * (it.sp + 1) / splits) : nk;
    return true;
  };
  Stream<C, AK, C::BM> A;
  Stream<C, BK_, C::BN> B;
  constexpr int D = QUARTERS ? 4 : kDepth<C>;
  u32x4_t va[D][Stream<C, AK, C::BM>::N], vb[D][Stream<C, BK_, C::BN>::N];
  // the item's operands, and its first whole k tiles on the way
  auto start = [&](const Item& it) {
    const E* a = reinterpret_cast<const E*>(p.a) + (int64_t)it.r0 * p.lda;
    const E* b = reinterpret_cast<const E*>(p.b) +
                 (FORM == TN ? (int64_t)it.r0 * p.ldb : (int64_t)it.e * p.stride_b);
    A.init(a, p.lda, it.m0, it.M);
    B.init(b, p.ldb, it.n0, p.n);
    const int kw = min(it.ke, it.K / C::BK);
    if (it.kb < kw) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        A.load(va[d], min(it.kb + d, kw - 1));
        B.load(vb[d], min(it.kb + d, kw - 1));
      }
    }
  };
  Item it;
  if (!next(it)) return;
  start(it);
  for (;;) {
    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int kw = min(it.ke, it.K / C::BK);  // end of the whole k tiles
    if (it.kb < kw) {
      const bool edge = (!AK && it.m0 + C::BM > it.M) || (!BK_ && it.n0 + C::BN > p.n);
      if constexpr (kTurns<C>) {
        const int group = __builtin_amdgcn_readfirstlane(wid >> 2);
        if (edge) turns_loop<C, FORM, true>(acc, smem, A, B, va[0], vb[0], it.kb, kw, wm, wn, group);
        else turns_loop<C, FORM, false>(acc, smem, A, B, va[0], vb[0], it.kb, kw, wm, wn, group);
      } else {
        if (edge) stream_loop<C, FORM, true, D>(acc, smem, A, B, va, vb, it.kb, kw, wm, wn);
        else stream_loop<C, FORM, false, D>(acc, smem, A, B, va, vb, it.kb, kw, wm, wn);
      }
    }
    if (kw < it.ke) {  // the rest of the contraction
      const int k0 = (it.ke - 1) * C::BK;
      A.tail(smem, k0, it.K);
      B.tail(smem + SA, k0, it.K);
      __syncthreads();
      multiply<C, FORM>(acc, smem, smem + SA, wm, wn);
      __syncthreads();
    }
    const Item done = it;
    const bool more = next(it);
    if (more) start(it);
    const int lane = threadIdx.x & 63;
    if (FORM == TN && !SPLIT && p.accumulate) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int row = done.m0 + wm + 32 * i + (lane & 31);
        if (row >= done.M) continue;
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int col = done.n0 + wn + 32 * j + 8 * g + 4 * (lane >> 5);
            if (col >= p.n) continue;
            const f32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            put4<O>(reinterpret_cast<O*>(p.c) + (int64_t)done.e * p.stride_c + (int64_t)row * p.ldc, col, p.n, v, true);
          }
      }
    } else {
      O* c;
      int64_t ldc;
      if constexpr (SPLIT) {
        ldc = p.n;
        c = reinterpret_cast<O*>(p.part) +
            (FORM == TN ? ((int64_t)done.sp * p.groups + done.e) * done.M : (int64_t)done.sp * p.rows + done.r0) * ldc;
      } else {
        ldc = p.ldc;
        c = reinterpret_cast<O*>(p.c) + (FORM == TN ? (int64_t)done.e * p.stride_c : (int64_t)done.r0 * ldc);
      }
      O* stage = reinterpret_cast<O*>(reinterpret_cast<char*>(smem) + wid * STAGE);
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
        store_rows<C::WN, O>(acc[i], stage, c, ldc, done.m0 + wm + 32 * i, done.M, done.n0 + wn, p.n);
    }
    if (!more) return;
    __syncthreads();  // the buffers are free
  }
}

// ------------------------------------------------------------ outer form, large tile, aligned operands
// 256 x 256 tiles of the outer form, 8 waves of 128 x 64, k tiles of 32 rows that
// go from memory to a ring of 4 LDS stages without passing through registers (a
// load instruction writes its wave's 64 x 16 bytes in lane order: two k rows of
// 512 bytes).  The turns are those of turns_loop, one k tile each; a stage is
// refilled three k tiles ahead, six turns before it is read.  LDS is not
// padded; the 32-byte block c of k row k lies at c ^ 2 (k & 3), which puts the
// four k rows and two blocks of a transpose read's 32 lanes on distinct banks.
// (The product forms have operands with 64 bytes a row and k tile; loaded like
// this, by half lines, they were slower than through registers: 333 against 292
// us forward, 378 against 328 us input gradient, 32768 rows, 32 experts of 4096 x
// 1024.  The outer form took 357 us, 393 through registers.)
constexpr int kStage = 32 * 1024, kStageB = 16 * 1024;  // bytes of a stage, of A's part
typedef __attribute__((address_space(3))) void* lds_ptr;

struct Dma {
  const uint16_t* base;
  int64_t step;
  uint32_t off[2];  // of this lane's piece, for the wave's two instructions
  // columns r0 .. of `limit` (a multiple of 8), read past the end from the last 8
  __device__ __forceinline__ void init(const uint16_t* b, int64_t ld, int r0, int limit, int wid) {
    base = b;
    step = 32 * ld;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      off[j] = (uint32_t)(row(j, wid) * (int)ld + min(r0 + column(j, wid), limit - 8));
  }
  // k row and column of this lane's piece of instruction j
  static __device__ __forceinline__ int row(int j, int wid) { return 2 * (2 * wid + j) + ((threadIdx.x & 63) >> 5); }
  static __device__ __forceinline__ int column(int j, int wid) {
    const int pc = threadIdx.x & 31;
    return (((pc >> 1) ^ (2 * (row(j, wid) & 3))) * 2 + (pc & 1)) * 8;
  }
  __device__ __forceinline__ void issue(char* part, int kt, int wid) const {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_amdgcn_global_load_lds((const void*)(base + kt * step + off[j]), (lds_ptr)(part + (2 * wid + j) * 1024),
                                       16, 0, 0);
  }
};

// A wave's fragments of one k tile of a stage, F of 32 rows and two 16-wide
// steps.  The reads are written out, with their wait in the same block: the
// compiler takes any LDS read it sees to depend on the loads to LDS under way
// and would wait for all of them.
__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
__device__ __forceinline__ bf16x8 join(i16x4 lo, i16x4 hi) {
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int F>
struct DmaFrag {
  uint32_t at[F];  // of each fragment in step 0
  __device__ __forceinline__ DmaFrag(int row) {
    const int lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
#pragma unroll
    for (int i = 0; i < F; ++i)
      at[i] = (8 * (g >> 1) + (j >> 2)) * 512 + ((((row >> 4) + 2 * i + (g & 1)) ^ (2 * (j >> 2))) * 32) + 8 * (j & 3);
  }
};

// Two fragments of both steps; k rows 0 .. 3 and 4 .. 7 of a step are 2048 bytes
// apart, the steps 8192.
__device__ __forceinline__ void read_frags_tr(bf16x8 (&f)[2][2], uint32_t a0, uint32_t a1) {
  i16x4 x[8];
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8\n\t"
      "ds_read_b64_tr_b16 %1, %8 offset:2048\n\t"
      "ds_read_b64_tr_b16 %2, %9\n\t"
      "ds_read_b64_tr_b16 %3, %9 offset:2048\n\t"
      "ds_read_b64_tr_b16 %4, %8 offset:8192\n\t"
      "ds_read_b64_tr_b16 %5, %8 offset:10240\n\t"
      "ds_read_b64_tr_b16 %6, %9 offset:8192\n\t"
      "ds_read_b64_tr_b16 %7, %9 offset:10240\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(x[6]), "=&v"(x[7])
      : "v"(a0), "v"(a1)
      : "memory");
  f[0][0] = join(x[0], x[1]);
  f[0][1] = join(x[2], x[3]);
  f[1][0] = join(x[4], x[5]);
  f[1][1] = join(x[6], x[7]);
}
__device__ __forceinline__ void read_frags(bf16x8 (&f)[2][2], const DmaFrag<2>& F, uint32_t p) {
  read_frags_tr(f, p + F.at[0], p + F.at[1]);
}
__device__ __forceinline__ void read_frags(bf16x8 (&f)[2][4], const DmaFrag<4>& F, uint32_t p) {
  bf16x8 g[2][2];
  read_frags_tr(g, p + F.at[0], p + F.at[1]);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    f[s][0] = g[s][0];
    f[s][1] = g[s][1];
  }
  read_frags_tr(g, p + F.at[2], p + F.at[3]);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    f[s][2] = g[s][0];
    f[s][3] = g[s][1];
  }
}

template <typename O>
__global__ __launch_bounds__(512, 2) void grouped_dma_kernel(GroupedParams p) {
  __shared__ __attribute__((aligned(1024))) char smem[4 * kStage];
  __shared__ Table T;
  __shared__ int order[64];  // the groups, the longest first
  const int tiles_n = (p.n + 255) / 256;
  const int tiles_m = (p.m + 255) / 256;
  build_table(T, p, 256, tiles_n, tiles_m * tiles_n);
  order_groups(order, T, p.groups);
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = wid >> 2;
  const int wm = (wid >> 2) * 128, wn = (wid & 3) * 64;
  const int items = T.tile[p.groups];
  const int place = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  int round = 0;
  struct Item {
    int e, r0, m0, n0, K;
  };
  auto next = [&](Item& it) -> bool {
    const int q = round * gridDim.x + (round & 1 ? gridDim.x - 1 - place : place);
    if (q >= items) return false;
    ++round;
    const int slot = q / (tiles_m * tiles_n);
    it.e = __builtin_amdgcn_readfirstlane(p.groups <= 64 ? order[slot] : slot);
    it.r0 = __builtin_amdgcn_readfirstlane(T.begin[it.e]);
    it.K = __builtin_amdgcn_readfirstlane(T.begin[it.e + 1]) - it.r0;
    int tm, tn;
    tile_of(q - slot * tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
    it.m0 = tm * 256;
    it.n0 = tn * 256;
    return true;
  };
  Dma A, B;
  const uint32_t lds0 = lds_address(smem);
  const DmaFrag<4> FA(wm);
  const DmaFrag<2> FB(wn);
  // k tile kt into its stage (past the item's last whole k tile: the last one again)
  auto issue = [&](const Item& it, int kt) {
    char* st = smem + (kt & 3) * kStage;
    const int k = min(kt, it.K / 32 - 1);
    A.issue(st, k, wid);
    B.issue(st + kStageB, k, wid);
  };
  // the item's operands and its first two k tiles on the way (stages 0 and 1)
  auto start = [&](const Item& it) {
    A.init(reinterpret_cast<const uint16_t*>(p.a) + (int64_t)it.r0 * p.lda, p.lda, it.m0, p.m, wid);
    B.init(reinterpret_cast<const uint16_t*>(p.b) + (int64_t)it.r0 * p.ldb, p.ldb, it.n0, p.n, wid);
    if (it.K >= 32) {
      issue(it, 0);
      issue(it, 1);
    }
  };
  Item it;
  if (!next(it)) return;
  start(it);
  for (;;) {
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int kw = it.K / 32;
    if (kw > 0) {
      issue(it, 2);
      // k tile 0 has landed for this wave (the 8 loads of k tiles 1 and 2 may be
      // under way), then for every wave
      asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      if (group) __builtin_amdgcn_s_barrier();  // the second group is one turn behind
      for (int kt = 0; kt < kw; ++kt) {
        const uint32_t st = lds0 + (kt & 3) * kStage;
        issue(it, kt + 3);  // the stage of k tile kt - 1, whose last reader (the second group) is done
        bf16x8 fa[2][4], fb[2][2];
        read_frags(fb, FB, st + kStageB);
        read_frags(fa, FA, st);
        // k tile kt + 1 has landed before the first group's next turn: the second
        // group waits for its loads here, the first after its MFMAs
        if (group) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[s][j], fa[s][i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        if (!group) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      if (!group) __builtin_amdgcn_s_barrier();
      // the loads past the last k tile have landed before the stages are used again
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
    }
    if (kw * 32 < it.K) {  // the rest of the contraction, zeros past its end
      const int k0 = kw * 32;
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        const bool isa = j < 2;
        const int k = Dma::row(j & 1, wid), c = Dma::column(j & 1, wid);
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (k0 + k < it.K)
          v = load_win((isa ? A.base : B.base) + (int64_t)(k0 + k) * (isa ? p.lda : p.ldb), (isa ? it.m0 : it.n0) + c,
                       isa ? p.m : p.n);
        *reinterpret_cast<u32x4_t*>(smem + (isa ? 0 : kStageB) + (2 * wid + (j & 1)) * 1024 + 16 * (threadIdx.x & 63)) = v;
      }
      __syncthreads();
      bf16x8 fa[2][4], fb[2][2];
      read_frags(fb, FB, lds0 + kStageB);
      read_frags(fa, FA, lds0);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[s][j], fa[s][i], acc[i][j], 0, 0, 0);
      __syncthreads();
    }
    const Item done = it;
    const bool more = next(it);
    if (more) start(it);  // stages 0 and 1; the results leave through the others
    const int lane = threadIdx.x & 63;
    if (p.accumulate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = done.m0 + wm + 32 * i + (lane & 31);
        if (row >= p.m) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int col = done.n0 + wn + 32 * j + 8 * g + 4 * (lane >> 5);
            if (col >= p.n) continue;
            const f32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            put4<O>(reinterpret_cast<O*>(p.c) + (int64_t)done.e * p.stride_c + (int64_t)row * p.ldc, col, p.n, v, true);
          }
      }
    } else {
      O* c = reinterpret_cast<O*>(p.c) + (int64_t)done.e * p.stride_c;
      // 128 bytes of a row at a time: 64 columns of bf16, 32 of fp32
      constexpr int COLS = 128 / (int)sizeof(O), PASS = COLS / 32;
      constexpr int STAGE = 32 * (COLS + 16 / (int)sizeof(O)) * (int)sizeof(O);
      static_assert(8 * STAGE <= 2 * kStage, "the waves' stages fit two of the ring's");
      O* stage = reinterpret_cast<O*>(smem + 2 * kStage + wid * STAGE);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; j += PASS)
          store_rows<COLS, O>(&acc[i][j], stage, c, p.ldc, done.m0 + wm + 32 * i, p.m, done.n0 + wn + 32 * j, p.n);
    }
    if (!more) return;
    __syncthreads();  // the stages are free
  }
}

// C = (C +) the sum of the splits' partial results, in their order.  `rows`
// rows of n in all; row r of C is at (r / m) stride_c + (r % m) ldc.
template <typename O>
__global__ __launch_bounds__(256) void grouped_join_kernel(GroupedParams p, int64_t rows, int m) {
  const int quads = (p.n + 3) / 4;
  const int64_t total = rows * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / quads;
    const int c = (int)(i - r * quads) * 4;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < p.splits; ++s) {
      const float* q = p.part + ((int64_t)s * rows + r) * p.n + c;
      if (c + 4 <= p.n) {
        typedef f32x4_t f32x4_a4 __attribute__((aligned(4)));
        v += *reinterpret_cast<const f32x4_a4*>(q);
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (c + j < p.n) v[j] += q[j];
      }
    }
    const int64_t e = r / m;
    put4<O>(reinterpret_cast<O*>(p.c) + e * p.stride_c + (r - e * m) * p.ldc, c, p.n, v, p.accumulate);
  }
}

// ------------------------------------------------------------ launchers
using BLarge = Cfg<uint16_t, 256, 256, 64, 128, 64, 1>;  // 8 waves
using BMid = Cfg<uint16_t, 128, 128, 64, 64, 64, 2>;     // 4 waves
using BSmall = Cfg<uint16_t, 32, 128, 64, 32, 32, 3>;    // 4 waves
using BHalf = Cfg<uint16_t, 64, 64, 64, 32, 32, 2>;      // 4 waves
using FHalf = Cfg<float, 64, 64, 16, 32, 32, 4>;
using FSmall = Cfg<float, 32, 128, 32, 32, 32, 3>;

// Tile sizes: 0 small (32 x 128), 1 half (64 x 64), 2 middle (128 x 128, bf16),
// 3 large (256 x 256, bf16).  The small tile is for groups of few rows, and has
// the sides under a 16-byte piece.  fp32's matrix instructions take 16 times as
// long a product as bf16's, so its 64 x 64 tiles ask little enough of LDS and
// L2, and their number is worth more: 7 experts of 1001 x 500, 2011 rows, 44
// (forward), 52 and 44 us (gradients), with 128 x 128 ones 61, 56 and 74; 8 of
// 2048 x 2048, 16384 rows, 1200 and 1290; the one loss 8192 rows, 64 of 2048 x
// 1024, weight gradient, 407 and 390.  bf16 takes them where fewer than three
// in four units would have a 128 x 128 one: 1907 rows, 11 of 144 x 1357, forward,
// 52 such tiles, 24 us instead of 31; 5075 rows, 17 of 1075 x 289, input
// gradient, 171, 32 instead of 45; but 23489 rows, 13 of 165 x 432, forward, 392,
// 29 instead of 25.
//
// The host knows the mean of the groups' rows only, so the rules go by it.
// Small tile up to 48 rows, forward and input gradient, small and wider tiles:
// bf16, 32 experts of 4096 x 1024, 12 rows 44, 41 and 48, 68 us; 40 rows 57, 54 and
// 47, 71; 56 rows 68, 83 and 48, 73.  fp32, 64 of 768 x 2048, 12 rows 91, 85 and
// 121, 117; 40 rows 130, 122 and 145, 134; 100 rows 227, 222 and 242, 232.
// Large tile from 256 rows, large and 128 x 128: 32 of 4096 x 1024, forward, 200
// rows 96 and 106, 300 rows 122 and 134; 64 of 768 x 2048, input gradient, 140 rows
// 83 and 62, 250 rows 95 and 91, 300 rows 122 and 106.
// In the outer form from 64 rows, large and 128 x 128, fp32 results: 32 of 4096 x
// 1024, 72 rows 137 and 168, 140 rows 165 and 204; aligned operands gain below that
// too (8 rows 114 and 126, 32 rows 125 and 150), others do not (8 rows 124 and
// 128, 60 rows 183 and 178), nor do results of one tile (300 of 256 x 256, 32 rows,
// 28 and 27).
struct Choice {
  int cfg, bm, bn, bk;
};
Choice choose_wide(int64_t tiles128, bool large, int dtype) {
  if (dtype == PMX_F32) return {1, 64, 64, 16};
  if (large) return {3, 256, 256, 64};
  if (tiles128 * 4 < kCU * 3) return {1, 64, 64, 64};
  return {2, 128, 128, 64};
}
Choice choose_product(int64_t rows, int k, int n, int groups, int dtype) {
  const int64_t avg = rows / groups;
  if (avg <= 48 || k < 8 || n < 8) return {0, 32, 128, dtype == PMX_BF16 ? 64 : 32};
  return choose_wide((rows / 128 + groups) * ((n + 127) / 128),
                     avg >= 256 && n >= 256 && (rows / 256) * ((n + 255) / 256) >= kCU, dtype);
}
Choice choose_outer(int64_t rows, int m, int n, int groups, int dtype) {
  if (m < 8 || n < 8) return {0, 32, 128, dtype == PMX_BF16 ? 64 : 32};
  auto tiles = [&](int side) { return (int64_t)groups * ((m + side - 1) / side) * ((n + side - 1) / side); };
  return choose_wide(tiles(128), m >= 256 && n >= 256 && tiles(256) >= kCU && rows / groups >= 64, dtype);
}

// Splits so that the items come to at most `unit` a compute unit, a split
// keeping at least `least` k tiles.  (8289 fp32 rows, 11 experts of 152 x 848, a
// step: 170 us, 242 with nothing split from 129 tiles on.  Four a unit for the
// small tile: 51 instead of 47 for 16 bf16 rows, 32 experts of 4096 x 1024.  The
// 64 x 64 tile takes four, in the outer form from 8 k tiles on: 23489 bf16 rows,
// 13 of 165 x 432, 41 us, 62 with two; 21648 fp32 rows, 7 of 184 x 648, 95 and
// 139.  In the products, whose partial results are many, from 16: 3384 bf16
// rows, 2 of 1925 x 328, input gradient, 34 us, 41 from 8 on.)  The large tile's
// kernels write whole results only: it is chosen where there are tiles enough.
int splits_for(const Choice& c, int64_t tiles, int64_t nk, int unit, int least) {
  if (tiles == 0 || c.cfg == 3) return 1;
  const int64_t want = unit * kCU / tiles, most = nk / least;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), 64));
}

int64_t max_tiles_product(const Choice& c, int64_t rows, int n, int groups) {
  return (rows / c.bm + std::min<int64_t>(groups, rows)) * ((n + c.bn - 1) / c.bn);
}

// Every 16-byte piece of the outer form's operands aligned and whole: what the
// direct loads to LDS take.
bool dma_ok(const GroupedParams& p) {
  return !(((uintptr_t)p.a | (uintptr_t)p.b) & 15) && p.lda % 8 == 0 && p.ldb % 8 == 0 && p.m % 8 == 0 && p.n % 8 == 0;
}

hipError_t launch_dma(const GroupedParams& p, dim3 grid, hipStream_t s) {
  if (p.out_dtype == PMX_F32) hipLaunchKernelGGL(grouped_dma_kernel<float>, grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL(grouped_dma_kernel<uint16_t>, grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

#define PMX_LAUNCH(KERNEL)                                                                       \
  if (p.splits > 1) { /* never with the large tile (splits_for) */                               \
    if constexpr (C::BM != 256)                                                                  \
      hipLaunchKernelGGL((KERNEL<C, FORM, float, true>), grid, block, 0, s, p);                  \
    else return hipErrorInvalidValue;                                                            \
  } else if (p.out_dtype == PMX_F32) {                                                           \
    hipLaunchKernelGGL((KERNEL<C, FORM, float, false>), grid, block, 0, s, p);                   \
  } else {                                                                                       \
    if constexpr (sizeof(typename C::E) == 2)                                                    \
      hipLaunchKernelGGL((KERNEL<C, FORM, uint16_t, false>), grid, block, 0, s, p);              \
    else return hipErrorInvalidValue;                                                            \
  }

// Blocks of a launch over `items` items, a multiple of 8.
template <class C>
int64_t grid_of(const GroupedParams& p, int64_t items) {
  const int64_t g = (std::min(items, (int64_t)p.num_cu * kBlocks<C>) + 7) / 8 * 8;
  return g < 8 ? 8 : g;
}

template <class C, int FORM>
hipError_t launch_form(const GroupedParams& p, int64_t items, hipStream_t s, bool any_side = false) {
  const int64_t g = grid_of<C>(p, items);
  const dim3 grid((unsigned)g), block(C::THREADS);
  if constexpr (C::BM == 256 && FORM == TN) {
    if (p.splits == 1 && dma_ok(p)) return launch_dma(p, grid, s);
  }
  if constexpr (C::BM == 32) {
    if (any_side) {
      PMX_LAUNCH(grouped_kernel)
      return hipGetLastError();
    }
  }
  if constexpr (C::BM != 32 || FORM != TN) {
    PMX_LAUNCH(grouped_tile_kernel)
  }
  return hipGetLastError();
}

using BQuarter = Cfg<uint16_t, 128, 128, 64, 64, 64, 1>;
template <int FORM>
hipError_t launch_quarters(GroupedParams p, int64_t items, hipStream_t s) {
  p.round = (int)grid_of<BLarge>(p, items);
  const dim3 grid((unsigned)p.round), block(BQuarter::THREADS);
  if (p.out_dtype == PMX_F32) hipLaunchKernelGGL((grouped_tile_kernel<BQuarter, FORM, float, false, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((grouped_tile_kernel<BQuarter, FORM, uint16_t, false, true>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <class C>
hipError_t launch_product_cfg(const GroupedParams& p, int64_t items, hipStream_t s, bool any_side = false) {
  return p.trans_b ? launch_form<C, NT>(p, items, s, any_side) : launch_form<C, NN>(p, items, s, any_side);
}

hipError_t launch_join(const GroupedParams& p, int64_t rows, int m, hipStream_t s) {
  const int64_t total = rows * ((p.n + 3) / 4);
  const dim3 grid((unsigned)std::min<int64_t>((total + 255) / 256, 2048));
  if (p.out_dtype == PMX_F32) hipLaunchKernelGGL(grouped_join_kernel<float>, grid, dim3(256), 0, s, p, rows, m);
  else hipLaunchKernelGGL(grouped_join_kernel<uint16_t>, grid, dim3(256), 0, s, p, rows, m);
  return hipGetLastError();
}

}  // namespace

int grouped_product_splits(int64_t rows, int k, int n, int groups, int dtype) {
  const Choice c = choose_product(rows, k, n, groups, dtype);
  return splits_for(c, max_tiles_product(c, rows, n, groups), (k + c.bk - 1) / c.bk,
                    c.cfg == 1 ? 4 : 2, c.cfg == 1 ? 16 : 8);
}

int grouped_outer_splits(int64_t rows, int m, int n, int groups, int dtype) {
  const Choice c = choose_outer(rows, m, n, groups, dtype);
  const int64_t tiles = (int64_t)groups * ((m + c.bm - 1) / c.bm) * ((n + c.bn - 1) / c.bn);
  return splits_for(c, tiles, rows / groups / c.bk, c.cfg == 1 ? 4 : 2, 8);
}

hipError_t launch_grouped_product(const GroupedParams& p, hipStream_t s) {
  if (p.rows == 0) return hipSuccess;
  const Choice c = choose_product(p.rows, p.k, p.n, p.groups, p.dtype);
  const int64_t items = max_tiles_product(c, p.rows, p.n, p.groups) * p.splits;
  hipError_t e;
  if (p.dtype == PMX_BF16) {
    e = c.cfg == 0   ? launch_product_cfg<BSmall>(p, items, s, p.k < 8 || p.n < 8)
        : c.cfg == 1 ? launch_product_cfg<BHalf>(p, items, s)
        : c.cfg == 2 ? launch_product_cfg<BMid>(p, items, s)
                     : launch_product_cfg<BLarge>(p, items, s);
  } else {
    e = c.cfg == 0 ? launch_product_cfg<FSmall>(p, items, s, p.k < 8 || p.n < 8)
                   : launch_product_cfg<FHalf>(p, items, s);
  }
  if (e == hipSuccess && c.cfg == 3 && p.k >= kQuartersK) e = p.trans_b ? launch_quarters<NT>(p, items, s) : launch_quarters<NN>(p, items, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join(p, p.rows, (int)p.rows, s);
}

hipError_t launch_grouped_outer(const GroupedParams& p, hipStream_t s) {
  const Choice c = choose_outer(p.rows, p.m, p.n, p.groups, p.dtype);
  const int64_t items =
      (int64_t)p.groups * ((p.m + c.bm - 1) / c.bm) * ((p.n + c.bn - 1) / c.bn) * p.splits;
  hipError_t e;
  if (p.dtype == PMX_BF16)
    e = c.cfg == 0   ? launch_form<BSmall, TN>(p, items, s, true)
        : c.cfg == 1 ? launch_form<BHalf, TN>(p, items, s)
        : c.cfg == 2 ? launch_form<BMid, TN>(p, items, s)
                     : launch_form<BLarge, TN>(p, items, s);
  else
    e = c.cfg == 0 ? launch_form<FSmall, TN>(p, items, s, true)
                   : launch_form<FHalf, TN>(p, items, s);
  if (e != hipSuccess || p.splits == 1) return e;
  return launch_join(p, (int64_t)p.groups * p.m, p.m, s);
}

}  // namespace pmx
