// Token embedding: Y[t] = scale W[id_t], and the gradient of the table,
//   dW[v] (+)= scale sum_{t : id_t = v, v != padding_idx} dY[t].
//
// The gradient sorts the tokens by id (stable, least significant digit first,
// one or two passes) and sums runs of equal ids over fixed chunks of the sorted
// order, so every row of dW is written once and every sum has a fixed order:
// no floating atomics, the same bits on every call.  Sums are fp32.
//
// Bound: HBM, tokens x dim read and vocab x dim written; the sort moves 8
// bytes a token and pass and is all latency.  So the sort's launches also clear
// dW: their other blocks write zeros to every row, the rows that have tokens
// are written again afterwards.  Up to kSmallSort tokens one block sorts them
// in LDS in one launch; up to kFew tokens one launch does everything.
//
// Measured, 32768 tokens of 1024 bf16 into 50000 fp32 rows (272 MB, 53 us at a
// copy's rate): 95 us, digit counts 10 and 9, scatters 15 and 15 (the clearing
// under these four), sums 31, joins 9.  4097 tokens of 515 fp32 into 10007 rows:
// sort and clearing 15, sums 4, joins 9.  A lookup of 8 rows takes 2.2 us, one of
// 32768 rows of 1024 bf16 21 (134 MB).
#include <algorithm>

#include "pmx_train.h"

namespace pmx {
namespace {

constexpr int kSortThreads = 256, kSortItems = 8, kSortTile = kSortThreads * kSortItems;
constexpr int kSortMaxBlocks = 256;  // a block sorts several tiles beyond 2^19 tokens
constexpr int kMaxDigits = 2048;     // 11 bits a pass
constexpr int kFew = 256;            // tokens up to which one launch does it all
constexpr int kFewBits = 10, kFewRows = 1 << kFewBits;  // rows one of its blocks owns at most
constexpr int kFewGroup = 3;         // they come in groups of 8
constexpr int kTeamRun = 16;         // tokens of a row that one team sums by itself
// Tokens one block sorts in LDS, which holds no more.  One block and the sort's
// launches, into 10007 x 515: 600 tokens 19 and 36 us, 4096 28 and 42, 8192 42 and
// 48; into 50000 x 1024: 8192 tokens 44 and 63.
constexpr int kSmallSort = 8192;

struct SortPlan {
  int bits;     // key bits: keys 0 .. vocab (vocab: tokens without a row)
  int passes;   // 1 or 2
  int dbits;    // bits a pass
  int span;     // tokens a block
  int blocks;
  int chunk;    // sorted positions summed by one block
  int chunks;
};

SortPlan sort_plan(int64_t tokens, int vocab) {
  SortPlan s;
  s.bits = 1;
  while ((int64_t)vocab >> s.bits) ++s.bits;
  s.passes = s.bits <= 11 ? 1 : 2;
  s.dbits = (s.bits + s.passes - 1) / s.passes;
  const int64_t tiles = (tokens + kSortTile - 1) / kSortTile;
  const int64_t per = (tiles + kSortMaxBlocks - 1) / kSortMaxBlocks;
  s.span = (int)(per * kSortTile);
  s.blocks = s.span ? (int)((tokens + s.span - 1) / s.span) : 0;
  // chunks of 8 to 32 tokens, about 1024 of them; longer ones once there are 4096
  const int64_t c = tokens <= 32768 ? (tokens + 1023) / 1024 : std::max<int64_t>(32, (tokens + 4095) / 4096);
  s.chunk = (int)std::max<int64_t>(8, (c + 7) / 8 * 8);
  s.chunks = (int)((tokens + s.chunk - 1) / s.chunk);
  return s;
}

struct EmbedWs {
  int* cnt;       // [blocks][digits]
  uint2* a;       // key, position
  uint2* b;
  float* part;    // [chunks][2][dim]
  size_t bytes;
};

EmbedWs embed_ws(void* base, const SortPlan& s, int64_t tokens, int dim) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  EmbedWs w;
  char* p = reinterpret_cast<char*>(base);
  size_t o = 0;
  w.cnt = reinterpret_cast<int*>(p + o);
  o += up((size_t)s.blocks * ((size_t)1 << s.dbits) * sizeof(int));
  w.a = reinterpret_cast<uint2*>(p + o);
  o += up((size_t)tokens * sizeof(uint2));
  w.b = reinterpret_cast<uint2*>(p + o);
  o += up((size_t)tokens * sizeof(uint2));
  w.part = reinterpret_cast<float*>(p + o);
  o += up((size_t)s.chunks * 2 * (size_t)dim * sizeof(float));
  w.bytes = o;
  return w;
}

// ---------------------------------------------------------------- lookup
// VB bytes a thread and step: the largest power of two up to 16 that divides
// the row length, both row strides and both addresses.  threadIdx.x walks a
// row, threadIdx.y the rows.  A grid has fewer than 2^32 threads in x, so blocks
// beyond kLookupBlocks go on in y.
constexpr int64_t kLookupBlocks = 1 << 23;

template <int VB>
struct Raw;
template <> struct Raw<16> { typedef u32x4_t type; };
template <> struct Raw<8> { typedef u32x2_t type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<2> { typedef uint16_t type; };

template <typename T, int VB>
__global__ __launch_bounds__(256) void embed_lookup_kernel(EmbedParams p) {
  typedef typename Raw<VB>::type R;
  constexpr int NE = VB / (int)sizeof(T);
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.tokens) return;
  const int64_t id = load_index(p.ids, t, p.ids64);
  const bool row = id >= 0 && id < p.vocab;  // an id outside the table reads nothing: zeros
  const T* src = reinterpret_cast<const T*>(p.table) + (row ? id : 0) * p.ld_table;
  T* dst = reinterpret_cast<T*>(p.out) + t * p.ld_out;
  const int n = p.dim / NE;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    R r = {};
    if (row) {
      r = reinterpret_cast<const R*>(src)[c];
      if (p.scale != 1.f) {
        T x[NE];
        __builtin_memcpy(x, &r, VB);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int j = 0; j < NE; ++j) x[j] *= p.scale;
        } else {
#pragma unroll
          for (int j = 0; j < NE; ++j)
            x[j] = (T)pack_bf16(__uint_as_float((uint32_t)x[j] << 16) * p.scale, 0.f);
        }
        __builtin_memcpy(&r, x, VB);
      }
    }
    reinterpret_cast<R*>(dst)[c] = r;
  }
}

// ---------------------------------------------------------------- sort
__device__ __forceinline__ uint32_t key_of(const EmbedParams& p, int64_t t) {
  const int64_t id = load_index(p.ids, t, p.ids64);
  return id < 0 || id >= p.vocab || id == p.padding_idx ? (uint32_t)p.vocab : (uint32_t)id;
}

// Rows [r0, r1) of dW to be cleared by the blocks of a launch from
// `first_block` on.
struct Clear {
  int r0, r1, first_block;
};

template <typename O>
__device__ __forceinline__ void store_zero4(O* d, int left);

// A block clears as many rows at a time as its threads cover.
template <typename O>
__device__ __forceinline__ void clear_rows(const EmbedParams& p, const Clear& z) {
  const int quads = (p.dim + 3) / 4, nt = blockDim.x;
  const int each = nt > quads ? nt / quads : 1;  // rows at a time
  const int r = nt > quads ? threadIdx.x / quads : 0, q0 = nt > quads ? threadIdx.x % quads : threadIdx.x;
  const int blocks = (int)gridDim.x - z.first_block;
  if (r >= each) return;
  for (int v = z.r0 + ((int)blockIdx.x - z.first_block) * each + r; v < z.r1; v += blocks * each) {
    O* d = reinterpret_cast<O*>(p.out) + (int64_t)v * p.ld_out;
    for (int q = q0; q < quads; q += nt) store_zero4<O>(d + 4 * q, p.dim - 4 * q);
  }
}
__device__ __forceinline__ void clear_any(const EmbedParams& p, const Clear& z) {
  if (p.out_dtype == PMX_F32) clear_rows<float>(p, z);
  else clear_rows<uint16_t>(p, z);
}

// All of the sort in one block, for up to kSmallSort tokens: LDS holds the
// (key, position) pairs, a pass ranks them (in registers) and puts them back
// in the new order.
__global__ __launch_bounds__(1024) void embed_sort_small_kernel(EmbedParams p, SortPlan s, uint2* out, Clear z) {
  constexpr int W = 16, N = kSmallSort / 1024;
  __shared__ uint2 pair[kSmallSort];
  __shared__ uint16_t wcnt[W][kMaxDigits];
  __shared__ int wsum[W];
  if ((int)blockIdx.x >= z.first_block) {
    clear_any(p, z);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6, tokens = (int)p.tokens;
  const int nd = 1 << s.dbits;
  // wave w has tokens w per .. of `per`, a multiple of 64
  const int steps = (tokens + 1023) / 1024, base = wid * steps * 64;
  uint2 kp[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = base + i * 64 + lane;
    kp[i] = i < steps && t < tokens ? make_uint2(key_of(p, t), (uint32_t)t) : make_uint2(0, 0);
  }
  for (int pass = 0; pass < s.passes; ++pass) {
    const int shift = pass * s.dbits;
    if (pass) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int t = base + i * 64 + lane;
        if (i < steps && t < tokens) kp[i] = pair[t];
      }
    }
    for (int d = tid; d < nd; d += 1024)
#pragma unroll
      for (int w = 0; w < W; ++w) wcnt[w][d] = 0;
    __syncthreads();
    int rank[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      rank[i] = 0;
      if (i < steps) {
        const bool live = base + i * 64 + lane < tokens;
        const int d = (kp[i].x >> shift) & (nd - 1);
        uint64_t m = __ballot(live);
        for (int bit = 0; bit < s.dbits; ++bit) {
          const uint64_t v = __ballot((d >> bit) & 1);
          m &= ((d >> bit) & 1) ? v : ~v;
        }
        const int first = m ? __builtin_ctzll(m) : 0;
        // one wave's counters: the first lane of each digit reads and adds
        int old = 0;
        if (live && lane == first) {
          old = wcnt[wid][d];
          wcnt[wid][d] = (uint16_t)(old + __popcll(m));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the next step's lanes see it
        old = __shfl(old, first);
        rank[i] = old + __popcll(m & ((1ull << lane) - 1));
      }
    }
    __syncthreads();
    // digits' totals, their exclusive sum, then every wave's start
    const int each = (nd + 1023) / 1024;  // 1 or 2 digits a thread
    int total = 0;
    for (int e = 0; e < each; ++e) {
      const int d = tid * each + e;
      if (d < nd)
#pragma unroll
        for (int w = 0; w < W; ++w) total += wcnt[w][d];
    }
    int incl = total;
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 63) wsum[wid] = incl;
    __syncthreads();
    int o = incl - total;
    for (int w = 0; w < wid; ++w) o += wsum[w];
    for (int e = 0; e < each; ++e) {
      const int d = tid * each + e;
      if (d < nd)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int x = wcnt[w][d];
          wcnt[w][d] = (uint16_t)o;
          o += x;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < steps && base + i * 64 + lane < tokens)
        pair[wcnt[wid][(kp[i].x >> shift) & (nd - 1)] + rank[i]] = kp[i];
    __syncthreads();
  }
  for (int t = tid; t < tokens; t += 1024) out[t] = pair[t];
}

// Digit counts of a pass per block, [blocks][digits].  (Counting pass 2 with
// global atomics while pass 1 scatters took 24 us for 32768 tokens, of which a
// frequent id's atomics on one counter were half.)
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void embed_hist_kernel(EmbedParams p, SortPlan s, int* cnt,
                                                                  const uint2* in, Clear z) {
  __shared__ int h[kMaxDigits];
  if ((int)blockIdx.x >= z.first_block) {
    clear_any(p, z);
    return;
  }
  const int nd = 1 << s.dbits;
  for (int d = threadIdx.x; d < nd; d += kSortThreads) h[d] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * s.span;
  const int64_t t1 = t0 + s.span < p.tokens ? t0 + s.span : p.tokens;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kSortThreads)
    atomicAdd(&h[((FIRST ? key_of(p, t) : in[t].x) >> (FIRST ? 0 : s.dbits)) & (nd - 1)], 1);
  __syncthreads();
  for (int d = threadIdx.x; d < nd; d += kSortThreads) cnt[(int64_t)blockIdx.x * nd + d] = h[d];
}

// One stable scatter pass.  A wave ranks 64 consecutive tokens at a time by
// matching digits with ballots; waves and tiles follow each other in order.
template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void embed_scatter_kernel(EmbedParams p, SortPlan s, const int* c,
                                                                     const uint2* in, uint2* out, Clear z) {
  constexpr int W = kSortThreads / 64;
  __shared__ int wcnt[W][kMaxDigits];
  __shared__ int base[kMaxDigits];
  __shared__ int part[kSortThreads];
  if ((int)blockIdx.x >= z.first_block) {
    clear_any(p, z);
    return;
  }
  const int nd = 1 << s.dbits, shift = FIRST ? 0 : s.dbits;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  // where each digit's tokens of this block begin: the digit's place in the
  // whole order plus what earlier blocks hold of it
  const int each = nd > kSortThreads ? nd / kSortThreads : 1;  // digits a thread
  int total = 0;
  for (int i = 0; i < each; ++i) {
    const int d = tid * each + i;
    if (d < nd) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int b = 0; b < s.blocks; ++b) {
        const int x = c[(int64_t)b * nd + d];
        if (b < (int)blockIdx.x) before += x;
        all += x;
      }
      base[d] = total + before;
      total += all;
    }
  }
  part[tid] = total;
  __syncthreads();
  for (int o = 1; o < kSortThreads; o <<= 1) {
    const int x = tid >= o ? part[tid - o] : 0;
    __syncthreads();
    part[tid] += x;
    __syncthreads();
  }
  const int excl = part[tid] - total;
  for (int i = 0; i < each; ++i) {
    const int d = tid * each + i;
    if (d < nd) base[d] += excl;
  }
  const int64_t t0 = (int64_t)blockIdx.x * s.span;
  const int64_t t1 = t0 + s.span < p.tokens ? t0 + s.span : p.tokens;
  for (int64_t tile = t0; tile < t1; tile += kSortTile) {
    __syncthreads();
    for (int d = tid; d < nd; d += kSortThreads)
#pragma unroll
      for (int w = 0; w < W; ++w) wcnt[w][d] = 0;
    __syncthreads();
    uint32_t key[kSortItems], pos[kSortItems];
    int rank[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t t = tile + wid * (64 * kSortItems) + i * 64 + lane;
      key[i] = 0;
      pos[i] = 0;
      if (t < t1) {
        if (FIRST) {
          key[i] = key_of(p, t);
          pos[i] = (uint32_t)t;
        } else {
          const uint2 v = in[t];
          key[i] = v.x;
          pos[i] = v.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t t = tile + wid * (64 * kSortItems) + i * 64 + lane;
      const bool live = t < t1;
      const int d = (key[i] >> shift) & (nd - 1);
      uint64_t m = __ballot(live);
      for (int bit = 0; bit < s.dbits; ++bit) {
        const uint64_t v = __ballot((d >> bit) & 1);
        m &= ((d >> bit) & 1) ? v : ~v;
      }
      // m: the live lanes with this lane's digit
      const int first = m ? __builtin_ctzll(m) : 0;
      int old = 0;
      if (live && lane == first) old = atomicAdd(&wcnt[wid][d], __popcll(m));
      old = __shfl(old, first);
      rank[i] = old + __popcll(m & ((1ull << lane) - 1));
    }
    __syncthreads();
    for (int d = tid; d < nd; d += kSortThreads) {
      int o = base[d];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int x = wcnt[w][d];
        wcnt[w][d] = o;
        o += x;
      }
      base[d] = o;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t t = tile + wid * (64 * kSortItems) + i * 64 + lane;
      if (t < t1) {
        const int dst = wcnt[wid][(key[i] >> shift) & (nd - 1)] + rank[i];
        out[dst] = make_uint2(key[i], pos[i]);
      }
    }
  }
}

// ---------------------------------------------------------------- sums
// Four columns of a row (fewer at its end), at any element alignment.
typedef float f32x4a_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2a_t __attribute__((ext_vector_type(2), aligned(2)));

template <typename T>
__device__ __forceinline__ f32x4_t load4(const T* p, int left) {
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  if (left >= 4) {
    if constexpr (sizeof(T) == 4) {
      v = *reinterpret_cast<const f32x4a_t*>(p);
    } else {
      const u32x2_t r = *reinterpret_cast<const u32x2a_t*>(p);
      v = {bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < left) {
        if constexpr (sizeof(T) == 4) v[j] = p[j];
        else v[j] = __uint_as_float((uint32_t)p[j] << 16);
      }
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int left, f32x4_t v) {
  if (left >= 4) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<f32x4a_t*>(p) = v;
    } else {
      const u32x2_t r = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      *reinterpret_cast<u32x2a_t*>(p) = r;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < left) {
        if constexpr (sizeof(T) == 4) p[j] = v[j];
        else p[j] = (T)pack_bf16(v[j], 0.f);
      }
  }
}

template <typename O>
__device__ __forceinline__ void store_zero4(O* d, int left) {
  store4<O>(d, left, f32x4_t{0.f, 0.f, 0.f, 0.f});
}

// A finished row: four of its columns.
template <typename O>
__device__ __forceinline__ void put_row(const EmbedParams& p, uint32_t key, int col, f32x4_t acc) {
  O* d = reinterpret_cast<O*>(p.out) + (int64_t)key * p.ld_out + col;
  const int left = p.dim - col;
  f32x4_t v = acc * p.scale;
  if (p.accumulate) v += load4<O>(d, left);
  store4<O>(d, left, v);
}

// Sums of runs of equal keys.  Sub-block (blockIdx, threadIdx.y) has one chunk
// of the sorted order and 4 blockDim.x columns; a run inside the chunk is
// finished here, a run that reaches over its ends leaves a partial sum (slot 0:
// the run that enters the chunk, slot 1: the run that leaves it), joined by
// embed_join_kernel.  WAVE: blockDim.x is a multiple of 64, so a wave has one
// chunk and reads its keys through the scalar cache.
template <typename T, typename O, bool WAVE>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedParams p, SortPlan s,
                                                        const uint2* __restrict__ sorted,
                                                        float* __restrict__ part, int slabs) {
  const int tokens = (int)p.tokens;
  const int ty = WAVE ? __builtin_amdgcn_readfirstlane(threadIdx.y) : threadIdx.y;
  const int cg = (int)blockIdx.x / slabs, slab = (int)blockIdx.x % slabs;
  const int64_t chunk = (int64_t)cg * blockDim.y + ty;
  const int col = (slab * (int)blockDim.x + (int)threadIdx.x) * 4;
  if (chunk >= s.chunks || col >= p.dim) return;
  const int c0 = (int)(chunk * s.chunk);
  const int c1 = c0 + s.chunk < tokens ? c0 + s.chunk : tokens;
  const int left = p.dim - col;
  const T* dy = reinterpret_cast<const T*>(p.dy) + col;
  const uint32_t none = (uint32_t)p.vocab;
  const uint32_t before = c0 > 0 ? sorted[c0 - 1].x : none;
  const uint32_t after = c1 < tokens ? sorted[c1].x : none;
  uint32_t cur = sorted[c0].x;
  bool entered = cur == before;  // the run began in an earlier chunk
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto slot = [&](int k) { return part + ((int64_t)chunk * 2 + k) * p.dim + col; };
  constexpr int U = 8;
  for (int i0 = c0; i0 < c1; i0 += U) {
    uint2 kp[U];
    f32x4_t v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) kp[j] = i0 + j < c1 ? sorted[i0 + j] : make_uint2(none, 0);
#pragma unroll
    for (int j = 0; j < U; ++j)
      v[j] = kp[j].x != none ? load4<T>(dy + (int64_t)kp[j].y * p.ld_dy, left) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (i0 + j < c1) {
        if (kp[j].x != cur) {
          if (cur != none) {
            if (entered) store4<float>(slot(0), left, acc);
            else put_row<O>(p, cur, col, acc);
          }
          cur = kp[j].x;
          entered = false;
          acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        acc += v[j];
      }
    }
  }
  if (cur == none) return;
  if (entered) store4<float>(slot(0), left, acc);
  else if (cur == after) store4<float>(slot(1), left, acc);
  else put_row<O>(p, cur, col, acc);
}

// Runs over chunk ends: one block a chunk (and slab of columns); the chunk a
// run begins in adds the partial sums of the chunks it goes through.  Their
// number comes from one look at the chunks' first keys by all threads; then
// threadIdx.y deals them out in contiguous shares, joined in order.  (Partial
// sums come from other XCDs' caches, about 2 us a dependent load: one thread
// walking a frequent id's 65 chunks took 50 us.)
template <typename O>
__global__ __launch_bounds__(1024) void embed_join_kernel(EmbedParams p, SortPlan s, const uint2* __restrict__ sorted,
                                                          const float* __restrict__ part, int slabs) {
  __shared__ f32x4_t sums[1024];
  const int tokens = (int)p.tokens;
  const int slab = (int)blockIdx.x % slabs;
  const int64_t chunk = (int)blockIdx.x / slabs;
  const int col = (slab * (int)blockDim.x + (int)threadIdx.x) * 4;
  const int64_t c0 = chunk * s.chunk, c1 = c0 + s.chunk;
  if (c1 >= tokens) return;  // nothing follows
  const uint32_t key = sorted[c1 - 1].x;
  if (key == (uint32_t)p.vocab || sorted[c1].x != key) return;
  if (c0 > 0 && sorted[c0].x == key && sorted[c0 - 1].x == key) return;  // began earlier
  const int nt = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  int n = 0;  // chunks after this one that the run enters
  for (;;) {
    const int64_t c = chunk + 1 + n + tid;
    const int k = __syncthreads_count(c < s.chunks && sorted[c * s.chunk].x == key);
    n += k;
    if (k < nt) break;
  }
  const int left = p.dim - col;
  // this thread's share of the slots 1 of `chunk`, then 0 of chunk + 1 .. + n
  const int ny = blockDim.y, i0 = (int)((int64_t)(n + 1) * threadIdx.y / ny),
            i1 = (int)((int64_t)(n + 1) * (threadIdx.y + 1) / ny);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  if (left > 0) {
    constexpr int U = 8;
    for (int i = i0; i < i1; i += U) {
      f32x4_t v[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t at = i + j < i1 ? i + j : i;  // past the share: read, not added
        v[j] = load4<float>(part + ((chunk + at) * 2 + (at == 0)) * p.dim + col, left);
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i + j < i1) acc += v[j];
    }
  }
  sums[tid] = acc;
  __syncthreads();
  if (threadIdx.y == 0 && left > 0) {
    for (int y = 1; y < ny; ++y) acc += sums[y * blockDim.x + tid];
    put_row<O>(p, key, col, acc);
  }
}

// The whole gradient in one launch, for up to kFew tokens: three launches that
// wait for each other cost more than the work.  Block (range, slab) owns every
// ranges-th group of 8 rows and 4 blockDim.x of their columns.  It reads every
// id, lists its own in token order, sorts the list by row (one wave, ballots)
// and writes each of its rows once: the sum of the row's tokens, or zeros.  A
// team (one threadIdx.y) takes a row of up to kTeamRun tokens; the block shares
// out a longer run and joins it in order.
//
// 13 tokens into 3000 x 200: 7.4 us, with the sort's launches 15; 200 into
// 20000 x 512: 15.6 and 24.6.  One block reads a whole run, about 30 GB/s: 500
// tokens of one id took 65 us here and 28 with the sort, hence the 256.
template <typename T, typename O>
__global__ __launch_bounds__(kFew) void embed_few_kernel(EmbedParams p, int ranges, int slabs) {
  constexpr int W = kFew / 64, U = 8;
  __shared__ uint32_t list[kFew];     // row << 16 | token, in token order
  __shared__ uint16_t token[kFew];    // by row
  __shared__ int head[kFewRows];      // tokens of a row, then where they begin, then where they end
  __shared__ int wsum[W], longs;
  __shared__ uint16_t long_row[kFew / kTeamRun];
  __shared__ f32x4_t sums[kFew];
  const int tx = blockDim.x, ny = blockDim.y;
  const int tid = threadIdx.y * tx + threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int range = (int)blockIdx.x % ranges, slab = (int)blockIdx.x / ranges;
  const int shift = 31 - __clz(ranges), tokens = (int)p.tokens;
  // the range's rows, at most kFewRows, some of its last group past the table
  const int rows = (((p.vocab - 1) >> kFewGroup) - range + ranges) >> shift << kFewGroup;
  auto row_of = [&](int j) {
    return (((j >> kFewGroup) << shift) + range) << kFewGroup | (j & ((1 << kFewGroup) - 1));
  };
  for (int j = tid; j < kFewRows; j += kFew) head[j] = 0;
  if (tid == 0) longs = 0;
  int key = -1;
  if (tid < tokens) {
    const uint32_t k = key_of(p, tid);
    if (k != (uint32_t)p.vocab && (int)(k >> kFewGroup & (ranges - 1)) == range)
      key = (int)(k >> kFewGroup >> shift << kFewGroup | (k & ((1 << kFewGroup) - 1)));
  }
  const uint64_t mine = __ballot(key >= 0);
  if (lane == 0) wsum[wid] = __popcll(mine);
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wid) at += wsum[w];
    all += wsum[w];
  }
  if (key >= 0) {
    list[at + __popcll(mine & ((1ull << lane) - 1))] = (uint32_t)key << 16 | (uint32_t)tid;
    atomicAdd(&head[key], 1);
  }
  __syncthreads();
  if (wid == 0 && all > 0) {
    // where each row's tokens begin
    int before = 0;
    for (int j0 = 0; j0 < rows; j0 += 64) {
      const int c = head[j0 + lane];  // 0 past the range's rows
      int incl = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(incl, o);
        if (lane >= o) incl += x;
      }
      head[j0 + lane] = before + incl - c;
      before += __shfl(incl, 63);
    }
    // the list in order, 64 at a time, each behind those of its row before it
    for (int i0 = 0; i0 < all; i0 += 64) {
      const bool live = i0 + lane < all;
      const uint32_t e = live ? list[i0 + lane] : 0;
      const int j = (int)(e >> 16);
      uint64_t m = __ballot(live);
#pragma unroll
      for (int bit = 0; bit < kFewBits; ++bit) {
        const uint64_t v = __ballot((j >> bit) & 1);
        m &= ((j >> bit) & 1) ? v : ~v;
      }
      const int first = m ? __builtin_ctzll(m) : 0;
      int o = 0;
      if (live && lane == first) o = atomicAdd(&head[j], __popcll(m));
      o = __shfl(o, first);
      if (live) token[o + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(e & 0xFFFF);
    }
  }
  __syncthreads();
  // head[j] is now where row j's tokens end
  const int col = (slab * tx + (int)threadIdx.x) * 4, left = p.dim - col;
  const T* dy = reinterpret_cast<const T*>(p.dy) + col;
  auto run = [&](int a, int b) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int i = a; i < b; i += U) {
      f32x4_t v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = load4<T>(dy + (int64_t)token[i + u < b ? i + u : a] * p.ld_dy, left);  // past the run: read, not added
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u < b) acc += v[u];
    }
    return acc;
  };
  for (int j = threadIdx.y; j < rows; j += ny) {
    const int a = j ? head[j - 1] : 0, b = head[j];
    if (all == 0 || a == b) {
      if (!p.accumulate && left > 0 && row_of(j) < p.vocab)
        store_zero4<O>(reinterpret_cast<O*>(p.out) + (int64_t)(row_of(j)) * p.ld_out + col, left);
    } else if (b - a > kTeamRun) {
      if (threadIdx.x == 0) long_row[atomicAdd(&longs, 1)] = (uint16_t)j;
    } else if (left > 0) {
      put_row<O>(p, (uint32_t)(row_of(j)), col, run(a, b));
    }
  }
  __syncthreads();
  for (int l = 0; l < longs; ++l) {
    const int j = long_row[l];
    const int a = j ? head[j - 1] : 0, len = head[j] - a;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    if (left > 0) acc = run(a + len * (int)threadIdx.y / ny, a + len * ((int)threadIdx.y + 1) / ny);
    sums[tid] = acc;
    __syncthreads();
    if (threadIdx.y == 0 && left > 0) {
      for (int y = 1; y < ny; ++y) acc += sums[y * tx + tid];
      put_row<O>(p, (uint32_t)(row_of(j)), col, acc);
    }
    __syncthreads();
  }
}

int pow2_up(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

template <typename T>
hipError_t lookup_t(const EmbedParams& p, int vb, hipStream_t s) {
  const int n = (int)(p.dim * sizeof(T) / vb);
  int tx = pow2_up(n < 256 ? n : 256);
  if (tx < 16) tx = 16;
  const dim3 block(tx, 256 / tx);
  const int64_t blocks = (p.tokens + block.y - 1) / block.y, gx = std::min(blocks, kLookupBlocks);
  const dim3 grid((unsigned)gx, (unsigned)((blocks + gx - 1) / gx));
  switch (vb) {
    case 16: hipLaunchKernelGGL((embed_lookup_kernel<T, 16>), grid, block, 0, s, p); break;
    case 8: hipLaunchKernelGGL((embed_lookup_kernel<T, 8>), grid, block, 0, s, p); break;
    case 4: hipLaunchKernelGGL((embed_lookup_kernel<T, 4>), grid, block, 0, s, p); break;
    default:
      if constexpr (sizeof(T) == 2) hipLaunchKernelGGL((embed_lookup_kernel<T, 2>), grid, block, 0, s, p);
      else return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// `blocks` sorting blocks and, unless dW is added to, blocks that clear its
// rows [from, to) of `tenths` tenths, `most` at most.
dim3 with_clear(const EmbedParams& p, int blocks, int from, int to, int tenths, Clear* z, int most = 2048) {
  z->r0 = (int)((int64_t)p.vocab * from / tenths);
  z->r1 = (int)((int64_t)p.vocab * to / tenths);
  z->first_block = blocks;
  const int rows = p.accumulate ? 0 : z->r1 - z->r0;
  return dim3((unsigned)(blocks + std::min(rows, most)));
}

template <typename T, typename O>
hipError_t few_t(const EmbedParams& p, hipStream_t st) {
  const int quads = (p.dim + 3) / 4;
  int tx = pow2_up(quads < 64 ? quads : 64);
  if (tx < 16) tx = 16;
  const int slabs = (quads + tx - 1) / tx, groups = ((p.vocab - 1) >> kFewGroup) + 1;
  // about 1024 blocks; more where a block would own too many rows
  int ranges = 1;
  while (ranges < groups && (ranges * slabs < 1024 || (int64_t)ranges * (kFewRows >> kFewGroup) < groups)) ranges <<= 1;
  hipLaunchKernelGGL((embed_few_kernel<T, O>), dim3((unsigned)ranges * slabs), dim3(tx, kFew / tx), 0, st, p, ranges,
                     slabs);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t grad_t(const EmbedParams& p, hipStream_t st) {
  if (p.tokens == 0 && p.accumulate) return hipSuccess;
  if (p.tokens <= kFew) return few_t<T, O>(p, st);
  const SortPlan s = sort_plan(p.tokens, p.vocab);
  const EmbedWs w = embed_ws(p.ws, s, p.tokens, p.dim);
  const uint2* sorted = w.a;
  hipError_t e;
  Clear z;
  const dim3 b(kSortThreads);
  if (p.tokens <= kSmallSort) {
    // one of these blocks fits a unit, and each is 16 waves to start (1000 tokens
    // into 10007 x 515: 28 us, 31 with up to 2048 blocks)
    const dim3 g = with_clear(p, 1, 0, 1, 1, &z, 512);
    hipLaunchKernelGGL(embed_sort_small_kernel, g, dim3(1024), 0, st, p, s, w.a, z);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    // the clearing is dealt out over the launches by the sort's share of them
    const bool two = s.passes > 1;
    dim3 g = with_clear(p, s.blocks, 0, two ? 2 : 4, 10, &z);
    hipLaunchKernelGGL((embed_hist_kernel<true>), g, b, 0, st, p, s, w.cnt, (const uint2*)nullptr, z);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    g = with_clear(p, s.blocks, two ? 2 : 4, two ? 5 : 10, 10, &z);
    hipLaunchKernelGGL((embed_scatter_kernel<true>), g, b, 0, st, p, s, (const int*)w.cnt, (const uint2*)nullptr,
                       w.a, z);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (two) {
      g = with_clear(p, s.blocks, 5, 7, 10, &z);
      hipLaunchKernelGGL((embed_hist_kernel<false>), g, b, 0, st, p, s, w.cnt, (const uint2*)w.a, z);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      g = with_clear(p, s.blocks, 7, 10, 10, &z);
      hipLaunchKernelGGL((embed_scatter_kernel<false>), g, b, 0, st, p, s, (const int*)w.cnt, (const uint2*)w.a,
                         w.b, z);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      sorted = w.b;
    }
  }
  const int quads = (p.dim + 3) / 4;
  int tx = pow2_up(quads < 256 ? quads : 256);
  if (tx < 16) tx = 16;
  const dim3 block(tx, 256 / tx);
  const int slabs = (quads + tx - 1) / tx;
  const dim3 grid((unsigned)((s.chunks + block.y - 1) / block.y * slabs));
  if (tx >= 64)
    hipLaunchKernelGGL((embed_sum_kernel<T, O, true>), grid, block, 0, st, p, s, sorted, w.part, slabs);
  else
    hipLaunchKernelGGL((embed_sum_kernel<T, O, false>), grid, block, 0, st, p, s, sorted, w.part, slabs);
  if ((e = hipGetLastError()) != hipSuccess || s.chunks < 2) return e;
  hipLaunchKernelGGL((embed_join_kernel<O>), dim3((unsigned)(s.chunks * slabs)), dim3(tx, 1024 / tx), 0, st, p, s,
                     sorted, (const float*)w.part, slabs);
  return hipGetLastError();
}

}  // namespace

size_t embed_grad_workspace(int64_t tokens, int vocab, int dim) {
  // few tokens need none; asking for the smallest one all the same keeps a
  // program that passes null from being refused only once its batch grows
  return tokens <= kFew ? 256 : embed_ws(nullptr, sort_plan(tokens, vocab), tokens, dim).bytes;
}

hipError_t launch_embed_lookup(const EmbedParams& p, hipStream_t s) {
  if (p.tokens == 0) return hipSuccess;
  const int es = p.dtype == PMX_F32 ? 4 : 2;
  const uint64_t all = (uint64_t)(uintptr_t)p.table | (uint64_t)(uintptr_t)p.out | (uint64_t)p.dim * es |
                       (uint64_t)p.ld_table * es | (uint64_t)p.ld_out * es;
  const int vb = !(all & 15) ? 16 : !(all & 7) ? 8 : !(all & 3) ? 4 : 2;
  return es == 4 ? lookup_t<float>(p, vb, s) : lookup_t<uint16_t>(p, vb, s);
}

hipError_t launch_embed_grad(const EmbedParams& p, hipStream_t s) {
  if (p.dtype == PMX_F32)
    return p.out_dtype == PMX_F32 ? grad_t<float, float>(p, s) : grad_t<float, uint16_t>(p, s);
  return p.out_dtype == PMX_F32 ? grad_t<uint16_t, float>(p, s) : grad_t<uint16_t, uint16_t>(p, s);
}

}  // namespace pmx
