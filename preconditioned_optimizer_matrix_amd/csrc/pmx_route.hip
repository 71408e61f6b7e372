// Router of an expert layer: softmax, the top k experts of each token, their
// gates, counts, the order of the pairs by expert, and the balance loss with
// its gradient.  Formulas and edge cases: include/pmx.h.
//
// Design: a block takes a chunk of tokens (chunk_of).  A team of 4 to 64 lanes holds a
// token's row in registers, a lane neighbouring experts, so among equal logits the
// lowest lane with a match and its first match are the lowest index.  A chunk's choice
// of an expert is one 64-bit mask in LDS: its count is the mask's bits, a pair's rank the
// bits below its token, whatever order they were set in.  So the pairs are sorted by
// (expert, token) without a sort:
//   1. rows:    ids, gates, masks -> counts a chunk; sums of p and lse^2 a chunk
//   2. scatter: each block adds up the counts of the chunks before its own and of all
//               (a byte each), so offsets and each pair's row; the first blocks sum p
//               over the chunks, the last of them to finish writes the loss
// With many chunks a launch between the two adds the counts up instead.  One chunk
// does everything in one launch.  Every sum has a fixed order.
//
// Bound: launches and latency; the logits are read once forward and once in the
// gradient.  32768 x 64 fp32 (8 MB each time), top 4: 8.5 and 6.7 us for the two launches,
// 7.6 for the gradient; 16 tokens of 32: 4.8 us in one launch.  With many tokens the
// instructions themselves: 262144 x 128 bf16, top 4, 61 a logit forward and 42 in the
// gradient keep the units busy for 50 and 43 us.
#include <algorithm>

#include "pmx_layer.h"

namespace pmx {
namespace {

constexpr int kMaxE = PMX_MAX_GROUPS, kMaxTop = PMX_MAX_ROUTE_TOP;

constexpr int kScatter = 512;  // threads of the second launch: four blocks a unit
// Tokens a block.  Above 256 experts a token a team, in blocks of half the size once
// there is more than one a unit: 500 experts, 4097 fp32 tokens, the whole forward 25.2 us
// with 32 a block and 27.1 with 16, 32768 bf16 tokens 81 and 73; 1000 experts, 16 and 8 a
// block, 4096 tokens 33.6 and 33.5, 32768 180 and 158.
int chunk_of(int64_t rows, int experts) {
  if (experts <= 256) return 64;
  if (experts <= 512) return rows <= 8192 ? 32 : 16;
  return rows <= 16 ? 16 : 8;
}
// One launch where one block takes a token a team: 64 tokens of 1000 experts in it 49 us,
// in two launches 22.
bool one_launch(int64_t rows, int experts) { return rows <= chunk_of(rows, experts); }
int64_t chunks_of(int64_t rows, int experts) { return (rows + chunk_of(rows, experts) - 1) / chunk_of(rows, experts); }
// Every block reads all counts while that is at most 32 MB in all: a launch less
// (32768 tokens, 64 experts: one launch of 6.9 us for two of 7.2 and 4.1).
bool counts_in_scatter(int64_t chunks, int experts) { return chunks * chunks * ((experts + 3) / 4 * 4) <= (32 << 20); }

struct RouteWs {
  uint8_t* count;   // [chunks][experts, up to a multiple of 4]
  float* share;     // [chunks][experts] sums of p
  float* zsum;      // [chunks] sums of lse^2
  int32_t* live;    // [chunks]
  double* part;     // [experts / 16] of the loss
  int32_t* done;    // blocks that have written theirs
  int32_t* before;  // [chunks][experts] pairs of earlier chunks, from the launch between
  size_t bytes;
};
__host__ __device__ __forceinline__ RouteWs route_ws(void* base, int64_t chunks, int experts, bool between) {
  RouteWs w;
  char* p = reinterpret_cast<char*>(base);
  w.part = reinterpret_cast<double*>(p);
  p += (experts + 15) / 16 * 8;
  w.done = reinterpret_cast<int32_t*>(p);
  p += 8;
  w.share = reinterpret_cast<float*>(p);
  p += chunks * experts * 4;
  w.zsum = reinterpret_cast<float*>(p);
  p += chunks * 4;
  w.live = reinterpret_cast<int32_t*>(p);
  p += chunks * 4;
  w.before = reinterpret_cast<int32_t*>(p);
  if (between) p += chunks * experts * 4;
  w.count = reinterpret_cast<uint8_t*>(p);
  p += chunks * ((experts + 3) / 4 * 4);
  w.bytes = (size_t)(p - reinterpret_cast<char*>(base));
  return w;
}

// T lanes a token, V experts a lane, TEAMS tokens a block (the gradient: 256 threads).
template <typename E_, int T_, int V_, int TEAMS_>
struct RCfg {
  typedef E_ E;
  static constexpr int T = T_, V = V_, MAXE = T_ * V_ < kMaxE ? T_ * V_ : kMaxE;
  static constexpr int TEAMS = TEAMS_, THREADS = T_ * TEAMS_, WAVES = THREADS / 64;
};

template <int T>
__device__ __forceinline__ float team_max(float v) {
  v = fmaxf(v, dpp<kXor1>(v));
  v = fmaxf(v, dpp<kXor2>(v));
  if constexpr (T >= 8) v = fmaxf(v, dpp<kHalfMirror>(v));
  if constexpr (T >= 16) v = fmaxf(v, dpp<kMirror>(v));
  if constexpr (T >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  if constexpr (T >= 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
template <int T>
__device__ __forceinline__ float team_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  if constexpr (T >= 8) v += dpp<kHalfMirror>(v);
  if constexpr (T >= 16) v += dpp<kMirror>(v);
  if constexpr (T >= 32) v += __shfl_xor(v, 16);
  if constexpr (T >= 64) v += __shfl_xor(v, 32);
  return v;
}
// Over the wave's teams: what lanes of one place in their teams hold.
template <int T>
__device__ __forceinline__ float over_teams(float v) {
  if constexpr (T <= 4) v += dpp<0x124>(v);  // row_ror:4
  if constexpr (T <= 8) v += dpp<0x128>(v);  // row_ror:8
  if constexpr (T <= 16) v += __shfl_xor(v, 16);
  if constexpr (T <= 32) v += __shfl_xor(v, 32);
  return v;
}
template <int T>
__device__ __forceinline__ uint64_t team_bits(uint64_t votes) {  // of this lane's team, from bit 0
  if constexpr (T == 64) return votes;
  else return (votes >> ((threadIdx.x & 63) & ~(T - 1))) & ((1ull << T) - 1);
}

// A lane's logits, -inf past the last expert.
template <class C>
__device__ __forceinline__ void load_logits(float (&z)[C::V], const RouteParams& p, int64_t row, int lane) {
  typedef typename C::E E;
  const E* r = reinterpret_cast<const E*>(p.z) + row * p.ldz;
  const int e0 = lane * C::V;
  typedef uint32_t vec __attribute__((ext_vector_type(C::V * (int)sizeof(E) / 4), aligned(sizeof(E))));
  if (e0 + C::V <= p.experts) {
    const vec v = *reinterpret_cast<const vec*>(r + e0);
#pragma unroll
    for (int j = 0; j < C::V; ++j) {
      if constexpr (sizeof(E) == 2) z[j] = j & 1 ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
      else z[j] = __uint_as_float(v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < C::V; ++j) {
      z[j] = -__builtin_inff();
      if (e0 + j < p.experts) {
        if constexpr (sizeof(E) == 2) z[j] = __uint_as_float((uint32_t)r[e0 + j] << 16);
        else z[j] = r[e0 + j];
      }
    }
  }
}

template <class C>
__device__ __forceinline__ void store_logits(void* dz, int64_t ld, int64_t row, int experts, int lane, const float (&z)[C::V]) {
  typedef typename C::E E;
  E* r = reinterpret_cast<E*>(dz) + row * ld;
  const int e0 = lane * C::V;
  typedef uint32_t vec __attribute__((ext_vector_type(C::V * (int)sizeof(E) / 4), aligned(sizeof(E))));
  vec v;
#pragma unroll
  for (int j = 0; j < C::V * (int)sizeof(E) / 4; ++j) {
    if constexpr (sizeof(E) == 2) v[j] = pack_bf16(z[2 * j], z[2 * j + 1]);
    else v[j] = __float_as_uint(z[j]);
  }
  if (e0 + C::V <= experts) {
    *reinterpret_cast<vec*>(r + e0) = v;
  } else {
#pragma unroll
    for (int j = 0; j < C::V; ++j)
      if (e0 + j < experts) {
        if constexpr (sizeof(E) == 2) r[e0 + j] = (E)(v[j >> 1] >> (16 * (j & 1)));
        else r[e0 + j] = z[j];
      }
  }
}

struct RowStat {
  float high, sum, inv;  // inv: e inv are the probabilities, 0 in dead and NaN in bad rows
  bool dead, bad;  // nothing to choose from; NaN or +inf
};
// e: exp(z - max), always finite (0 for NaN and where the largest is infinite).
template <class C>
__device__ __forceinline__ RowStat softmax_row(float (&e)[C::V], const float (&z)[C::V], bool live) {
  RowStat s;
  float m = z[0];
#pragma unroll
  for (int j = 1; j < C::V; ++j) m = fmaxf(m, z[j]);
  s.high = team_max<C::T>(m);
  float t = 0.f;
#pragma unroll
  for (int j = 0; j < C::V; ++j) {
    e[j] = exp_acc(z[j] - s.high);
    t += e[j];
  }
  s.sum = team_sum<C::T>(t);
  bool nan = false;
#pragma unroll
  for (int j = 0; j < C::V; ++j) nan |= !(z[j] < __builtin_inff());
  s.bad = live && team_bits<C::T>(__ballot(nan)) != 0;
  s.dead = !live || (!s.bad && s.high == -__builtin_inff());
  s.inv = s.dead ? 0.f : s.bad ? __builtin_nanf("") : 1.f / s.sum;
  return s;
}

struct Masks {
  uint64_t bits[kMaxE];
};
// A chunk's choices: index (-1: none left) and logit; its tokens' largest logit and
// what a gate is divided by (NaN: a bad row).
struct Chosen {
  int16_t id[64][kMaxTop];
  float z[64][kMaxTop];
  float high[64], den[64];
};

// Rows of one chunk: choices to LDS, sums of p to registers.
template <class C>
__device__ __forceinline__ void route_rows(const RouteParams& p, int64_t first, int count, Chosen& S, float (&share)[C::V],
                                           float& zsum, int& live_count) {
  const int team = threadIdx.x / C::T, lane = threadIdx.x % C::T;
  const int rounds = (count + C::TEAMS - 1) / C::TEAMS;
  for (int i = 0; i < rounds; ++i) {
    const int at = i * C::TEAMS + team;
    const bool inside = at < count;
    const int64_t row = first + (inside ? at : count - 1);
    float z[C::V], e[C::V];
    load_logits<C>(z, p, row, lane);
    const bool live = inside && (!p.live || p.live[row] != 0);
    const RowStat s = softmax_row<C>(e, z, live);
#pragma unroll
    for (int j = 0; j < C::V; ++j) share[j] += e[j] * s.inv;
    const float lse = s.bad ? __builtin_nanf("") : s.high + logf(s.sum);
    if (!s.dead && lane == 0) {
      zsum += lse * lse;
      ++live_count;
    }
    const float none = -__builtin_inff();
    const bool routed = !s.dead && !s.bad;
    float chosen_sum = 0.f;
    for (int k = 0; k < p.top; ++k) {
      float m = z[0];
#pragma unroll
      for (int j = 1; j < C::V; ++j) m = fmaxf(m, z[j]);
      const float best = team_max<C::T>(m);
      const uint64_t match = team_bits<C::T>(__ballot(m == best));
      const bool ok = routed && best != none;
      if (ok) chosen_sum += exp_acc(best - s.high);
      // the first lane with a match, its first match
      int v = C::V - 1;
#pragma unroll
      for (int j = C::V - 2; j >= 0; --j) v = z[j] == best ? j : v;
      const bool mine = ok && lane == __ffsll((unsigned long long)match) - 1;
      if (inside && (mine || (!ok && lane == 0))) {
        S.id[at][k] = (int16_t)(ok ? lane * C::V + v : -1);
        S.z[at][k] = best;
      }
#pragma unroll
      for (int j = 0; j < C::V; ++j) z[j] = mine && j == v ? none : z[j];
    }
    if (inside && lane == 0) {
      S.high[at] = s.high;
      S.den[at] = s.bad ? __builtin_nanf("") : p.normalize ? chosen_sum : s.sum;
    }
  }
}

// Ids and gates of a chunk to memory, the chosen to the masks.
template <class C>
__device__ __forceinline__ void route_pairs(const RouteParams& p, int64_t first, int count, Masks& M, const Chosen& S) {
  for (int i = threadIdx.x; i < count * p.top; i += C::THREADS) {
    const int t = i / p.top, k = i - t * p.top, id = S.id[t][k];
    const float den = S.den[t];
    p.ids[first * p.top + i] = id;
    p.gates[first * p.top + i] = id >= 0 ? exp_acc(S.z[t][k] - S.high[t]) / den : den != den ? den : 0.f;
    if (id >= 0) atomicOr((unsigned long long*)&M.bits[id], 1ull << t);
  }
}

template <class C>
struct Join {
  static constexpr int ROWS = C::WAVES < 8 ? C::WAVES : 8;
  float sums[C::MAXE], stage[ROWS][C::MAXE], z[C::WAVES];
  int n[C::WAVES];
};
// Sums over the teams, in a fixed order, of what each lane holds of its experts (J.sums),
// and of lse^2 and live tokens, which all threads get.
template <class C>
__device__ __forceinline__ void join_teams(Join<C>& J, const float (&share)[C::V], float& z, int& n, int experts) {
  constexpr int ROWS = Join<C>::ROWS;
  const int wid = threadIdx.x >> 6, lane = threadIdx.x % C::T;
  float v[C::V];
#pragma unroll
  for (int j = 0; j < C::V; ++j) v[j] = over_teams<C::T>(share[j]);
  z = over_teams<C::T>(z);
  n = (int)over_teams<C::T>((float)n);  // 64 at most
  if ((threadIdx.x & 63) == 0) {
    J.z[wid] = z;
    J.n[wid] = n;
  }
  for (int part = 0; part < C::WAVES / ROWS; ++part) {
    if (wid / ROWS == part && (int)(threadIdx.x & 63) < C::T)
#pragma unroll
      for (int j = 0; j < C::V; ++j) {
        const int e = lane * C::V + j;
        float* q = &J.stage[wid % ROWS][e];
        if (e < experts) *q = part ? *q + v[j] : v[j];
      }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < experts; e += C::THREADS) {
    float t = J.stage[0][e];
#pragma unroll
    for (int w = 1; w < ROWS; ++w) t += J.stage[w][e];
    J.sums[e] = t;
  }
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < C::WAVES; ++w) {
    z += J.z[w];
    n += J.n[w];
  }
  __syncthreads();
}

// Exclusive sums of `n` counts by the first wave, the total last.
__device__ __forceinline__ void scan_offsets(int* off, const int* counts, int n) {
  if (threadIdx.x < 64) {
    int carry = 0;
    for (int b = 0; b < n; b += 64) {
      const int i = b + threadIdx.x, c = i < n ? counts[i] : 0;
      int v = c;
      for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(v, d);
        if ((int)threadIdx.x >= d) v += x;
      }
      if (i < n) off[i] = carry + v - c;
      carry += __shfl(v, 63);
    }
    if (threadIdx.x == 0) off[n] = carry;
  }
  __syncthreads();
}

// loss = balance E / (top n) sum_e c_e P_e / n + zloss / n sum lse^2, from the sum of c_e n P_e.
// A bad row makes zsum NaN, and the loss whatever its terms; a zsum that is infinite only
// counts where it has a weight.
__device__ __forceinline__ void write_loss(const RouteParams& p, double dot, double zsum, int n) {
  const double nn = n;
  const double balance = p.balance != 0.f ? (double)p.balance * p.experts / (p.top * nn * nn) * dot : 0.0;
  const double z = p.zloss != 0.f ? (double)p.zloss / nn * zsum : 0.0;
  *p.loss = n == 0 ? 0.f : zsum != zsum ? __builtin_nanf("") : (float)(balance + z);
}
__device__ __forceinline__ double wave_sum_double(double v) {
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Everything, for one chunk of tokens (or none).
template <class C>
__global__ __launch_bounds__(C::THREADS) void route_one_kernel(RouteParams p) {
  __shared__ Masks M;
  __shared__ Chosen S;
  __shared__ Join<C> J;
  __shared__ int counts[C::MAXE], off[C::MAXE + 1];
  const int count = (int)p.rows;
  for (int e = threadIdx.x; e < p.experts; e += C::THREADS) M.bits[e] = 0;
  float share[C::V], z = 0.f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < C::V; ++j) share[j] = 0.f;
  if (count) route_rows<C>(p, 0, count, S, share, z, n);
  join_teams<C>(J, share, z, n, p.experts);  // its barriers: the choices are whole
  route_pairs<C>(p, 0, count, M, S);
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += C::THREADS) counts[e] = __popcll(M.bits[e]);
  __syncthreads();
  scan_offsets(off, counts, p.experts);
  for (int e = threadIdx.x; e <= p.experts; e += C::THREADS) {
    p.counts[e] = e < p.experts ? counts[e] : n;
    p.offsets[e] = off[e];
  }
  if (threadIdx.x < 64) {
    double dot = 0.0;
    for (int e = threadIdx.x; e < p.experts; e += 64) dot += (double)counts[e] * (double)J.sums[e];
    dot = wave_sum_double(dot);
    if (threadIdx.x == 0) write_loss(p, dot, z, n);
  }
  if (!p.slots) return;
  for (int i = threadIdx.x; i < count * p.top; i += C::THREADS) {
    const int t = i / p.top, e = S.id[t][i - t * p.top];
    int slot = -1;
    if (e >= 0) {
      slot = off[e] + __popcll(M.bits[e] & ((1ull << t) - 1));
      p.tokens[slot] = t;
    }
    p.slots[i] = slot;
    if (i >= off[p.experts]) p.tokens[i] = -1;
  }
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void route_rows_kernel(RouteParams p, int64_t chunks, bool between) {
  __shared__ Masks M;
  __shared__ Chosen S;
  __shared__ Join<C> J;
  const RouteWs w = route_ws(p.ws, chunks, p.experts, between);
  const int64_t b = blockIdx.x, first = b * C::TEAMS;
  const int count = (int)min((int64_t)C::TEAMS, p.rows - first);
  for (int e = threadIdx.x; e < p.experts; e += C::THREADS) M.bits[e] = 0;
  float share[C::V], z = 0.f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < C::V; ++j) share[j] = 0.f;
  route_rows<C>(p, first, count, S, share, z, n);
  join_teams<C>(J, share, z, n, p.experts);
  route_pairs<C>(p, first, count, M, S);
  __syncthreads();
  const int wide = (p.experts + 3) / 4 * 4;
  for (int e = threadIdx.x; e < wide; e += C::THREADS) w.count[b * wide + e] = e < p.experts ? (uint8_t)__popcll(M.bits[e]) : 0;
  for (int e = threadIdx.x; e < p.experts; e += C::THREADS) w.share[b * p.experts + e] = J.sums[e];
  if (threadIdx.x == 0) {
    w.zsum[b] = z;
    w.live[b] = n;
    if (b == 0) *w.done = 0;
  }
}

// Between: 16 experts a block, 64 segments of the chunks each.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteParams p, int64_t chunks) {
  __shared__ int part[64][17];
  const RouteWs w = route_ws(p.ws, chunks, p.experts, true);
  const int in = threadIdx.x & 15, seg = threadIdx.x >> 4, e = blockIdx.x * 16 + in, wide = (p.experts + 3) / 4 * 4;
  const int64_t per = (chunks + 63) / 64, c0 = min(seg * per, chunks), c1 = min(c0 + per, chunks);
  int n = 0;
  if (e < p.experts)
#pragma unroll 8
    for (int64_t c = c0; c < c1; ++c) n += w.count[c * wide + e];
  part[seg][in] = n;
  __syncthreads();
  int before = 0;
  for (int s = 0; s < seg; ++s) before += part[s][in];
  if (e >= p.experts) return;
#pragma unroll 8
  for (int64_t c = c0; c < c1; ++c) {
    w.before[c * p.experts + e] = before;
    before += w.count[c * wide + e];
  }
  if (seg == 63) p.counts[e] = before;
}

// The loss from the chunks' sums: 16 experts a block, the chunks in 32 segments; the
// last block to finish adds the parts up.
__device__ __forceinline__ void route_loss(const RouteParams& p, const RouteWs& w, int q, int64_t chunks) {
  __shared__ double seg[32][17];
  __shared__ int part[32][17];
  __shared__ double zs[8];
  __shared__ int ns[8], last;
  const int parts = (p.experts + 15) / 16, wide = (p.experts + 3) / 4 * 4;
  const int in = threadIdx.x & 15, s = threadIdx.x >> 4, e = q * 16 + in;
  const int64_t per = (chunks + 31) / 32, c0 = min(s * per, chunks), c1 = min(c0 + per, chunks);
  double t = 0.0;  // up to 2^17 chunks a segment
  int c_e = 0;
  if (e < p.experts)
#pragma unroll 8
    for (int64_t c = c0; c < c1; ++c) {
      t += (double)w.share[c * p.experts + e];
      c_e += w.count[c * wide + e];
    }
  seg[s][in] = t;
  part[s][in] = c_e;
  __syncthreads();
  if (threadIdx.x < 64) {  // four quarters of the segments
    double d = 0.0;
    int c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d += seg[8 * s + i][in];
      c += part[8 * s + i][in];
    }
    d += __shfl_xor(d, 16);
    d += __shfl_xor(d, 32);
    c += __shfl_xor(c, 16);
    c += __shfl_xor(c, 32);
    d *= (double)c;
    for (int k = 8; k > 0; k >>= 1) d += __shfl_xor(d, k);
    if (threadIdx.x == 0) {
      w.part[q] = d;
      __threadfence();
      last = atomicAdd(w.done, 1) == parts - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!last) return;
  double z = 0.0;
  int n = 0;
  for (int64_t c = threadIdx.x; c < chunks; c += kScatter) {
    z += (double)w.zsum[c];
    n += w.live[c];
  }
  z = wave_sum_double(z);
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
  if ((threadIdx.x & 63) == 0) {
    zs[threadIdx.x >> 6] = z;
    ns[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    double dot = 0.0;
    if ((int)threadIdx.x < parts) dot = __hip_atomic_load(&w.part[threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    dot = wave_sum_double(dot);
    if (threadIdx.x == 0) {
      z = 0.0;
      n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z += zs[i];
        n += ns[i];
      }
      p.counts[p.experts] = n;
      write_loss(p, dot, z, n);
    }
  }
}

// Blocks past the chunks: the loss.
__global__ __launch_bounds__(kScatter) void route_scatter_kernel(RouteParams p, int chunk, int64_t chunks, bool between) {
  __shared__ Masks M;
  __shared__ int counts[kMaxE], before[kMaxE], off[kMaxE + 1];
  const RouteWs w = route_ws(p.ws, chunks, p.experts, between);
  const int64_t b = blockIdx.x;
  const int losses = (p.experts + 15) / 16;  // first: theirs is the longer way
  if (b < losses) {
    route_loss(p, w, (int)b, chunks);
    return;
  }
  const int64_t at = b - losses, first = at * chunk;
  const int count = (int)min((int64_t)chunk, p.rows - first);
  const int pairs = p.slots ? count * p.top : 0;  // 1024 at most: two a thread
  int chosen[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = threadIdx.x + k * kScatter;
    chosen[k] = i < pairs ? p.ids[first * p.top + i] : -1;
  }
  for (int e = threadIdx.x; e < p.experts; e += kScatter) {
    M.bits[e] = 0;
    counts[e] = between ? p.counts[e] : 0;
    before[e] = between ? w.before[at * p.experts + e] : 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (chosen[k] >= 0) atomicOr((unsigned long long*)&M.bits[chosen[k]], 1ull << (((int)threadIdx.x + k * kScatter) / p.top));
  if (!between) {  // four experts a thread, its share of the chunks
    const int words = (p.experts + 3) / 4, segs = kScatter / words, s = (int)threadIdx.x / words;
    const uint32_t* c = reinterpret_cast<const uint32_t*>(w.count) + ((int)threadIdx.x - s * words);
    int all[4] = {0, 0, 0, 0}, low[4] = {0, 0, 0, 0};
    if (s < segs) {
#pragma unroll 8
      for (int i = s; i < (int)chunks; i += segs) {
        const uint32_t v = c[(int64_t)i * words];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = v >> (8 * j) & 255;
          all[j] += x;
          low[j] += i < at ? x : 0;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 4 * ((int)threadIdx.x - s * words) + j;
        if (e < p.experts) {  // whole numbers: in any order
          atomicAdd(&counts[e], all[j]);
          atomicAdd(&before[e], low[j]);
        }
      }
    }
  }
  __syncthreads();
  scan_offsets(off, counts, p.experts);
  if (at == 0)
    for (int e = threadIdx.x; e <= p.experts; e += kScatter) {
      p.offsets[e] = off[e];
      if (e < p.experts) p.counts[e] = counts[e];
    }
  if (!p.slots) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = threadIdx.x + k * kScatter, e = chosen[k], in = i / p.top;
    if (i >= pairs) continue;
    int slot = -1;
    if (e >= 0) {
      slot = off[e] + before[e] + __popcll(M.bits[e] & ((1ull << in) - 1));
      p.tokens[slot] = (int32_t)(first + in);
    }
    p.slots[first * p.top + i] = slot;
  }
  // rows behind the last pair
  const int64_t all = p.rows * p.top;
  for (int64_t i = off[p.experts] + at * kScatter + threadIdx.x; i < all; i += chunks * kScatter) p.tokens[i] = -1;
}

// dz = p (a - sum p a) + u zloss 2 lse / n p + the gates' part.
template <class C>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteParams p) {
  constexpr int TEAMS = 256 / C::T;
  const int team = threadIdx.x / C::T, lane = threadIdx.x % C::T, shift = (threadIdx.x & 63) & ~(C::T - 1);
  const int64_t step = (int64_t)gridDim.x * TEAMS;
  int64_t base = (int64_t)blockIdx.x * TEAMS;
  // a row's data, loaded ahead of what the row before it computes
  constexpr int NK = (kMaxTop + C::T - 1) / C::T;  // choices a lane holds: lane, lane + T, ..
  float nz[C::V], ng[NK] = {}, nd[NK] = {};
  int nid[NK];
#pragma unroll
  for (int i = 0; i < NK; ++i) nid[i] = -1;
  bool nlive = false;
  auto fetch = [&](int64_t b) {
    const int64_t row = min(b + team, p.rows - 1);
    load_logits<C>(nz, p, row, lane);
#pragma unroll
    for (int i = 0; i < NK; ++i)
      if (p.dgates && lane + i * C::T < p.top) {
        nid[i] = p.ids[row * p.top + lane + i * C::T];
        ng[i] = p.gates[row * p.top + lane + i * C::T];
        nd[i] = p.dgates[row * p.top + lane + i * C::T];
      }
    nlive = !p.live || p.live[row] != 0;
  };
  fetch(base);
  const float n = (float)p.counts[p.experts], u = p.upstream ? *p.upstream : 1.f;
  int c[C::V];
#pragma unroll
  for (int j = 0; j < C::V; ++j) c[j] = p.counts[min(lane * C::V + j, p.experts)];
  const float cb = n > 0.f ? u * p.balance * (float)p.experts / ((float)p.top * n) / n : 0.f;
  const float cz = n > 0.f ? u * p.zloss * 2.f / n : 0.f;
  float a[C::V];
#pragma unroll
  for (int j = 0; j < C::V; ++j) a[j] = lane * C::V + j < p.experts ? cb * (float)c[j] : 0.f;
  for (; base < p.rows; base += step) {
    const bool inside = base + team < p.rows, live = nlive && inside;
    const int64_t row = base + team;
    float z[C::V], e[C::V];
#pragma unroll
    for (int j = 0; j < C::V; ++j) z[j] = nz[j];
    int my_id[NK];
    float my_g[NK], my_d[NK], gd = 0.f;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      my_id[i] = nid[i];
      my_g[i] = nid[i] < 0 ? 0.f : ng[i];
      my_d[i] = nid[i] < 0 ? 0.f : nd[i];
      gd += my_g[i] * my_d[i];
    }
    if (base + step < p.rows) fetch(base + step);
    const RowStat s = softmax_row<C>(e, z, live);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < C::V; ++j) {
      e[j] *= s.inv;
      dot += e[j] * a[j];
    }
    dot = team_sum<C::T>(dot);
    gd = team_sum<C::T>(gd);
    // p's factor: the balance and z parts, and without normalisation the gates' own
    const float lse = s.high + logf(s.sum);
    const float all = s.dead ? 0.f : cz * lse - dot - (p.normalize ? 0.f : gd);
#pragma unroll
    for (int j = 0; j < C::V; ++j) z[j] = e[j] * (a[j] + all);
    if (p.dgates) {
      // the chosen ones': normalised g (dg - sum g dg), else g dg
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const float mine = s.dead ? 0.f : my_g[i] * (my_d[i] - (p.normalize ? gd : 0.f));
#pragma unroll
        for (int k = 0; k < (C::T < kMaxTop ? C::T : kMaxTop); ++k) {
          if (k + i * C::T >= p.top) continue;
          const int id = __shfl(my_id[i], shift + k) - lane * C::V;
          const float d = __shfl(mine, shift + k);
#pragma unroll
          for (int j = 0; j < C::V; ++j) z[j] += j == id ? d : 0.f;
        }
      }
    }
    if (inside) store_logits<C>(p.dz, p.lddz, row, p.experts, lane, z);
  }
}

// Few lanes a token, many experts a lane: the instructions of a reduction serve as
// many tokens as a wave has teams, until too few waves are left to hide their latency
// (32768 fp32 tokens, 64 experts, forward's first launch and the gradient: 16 lanes of 4
// 11.5 and 8.3 us, 8 of 8 9.8 and 8.1, 4 of 16 9.6 and 9.2; 262144 bf16 tokens, 128
// experts, the whole forward and the gradient: 16 lanes of 8 142 and 47 us, 8 of 16 97 and
// 43; the same tokens of 64 fp32: 8 of 8 72 and 27, 4 of 16 66 and 35).  Twelve a lane where
// that is enough: the 262144 of 96 bf16 103 and 47, 94 and 36; 32768 of 384 69 and 33, 62
// and 24; of 640 133 and 53, 123 and 44.
template <typename E, typename F>
hipError_t with_cfg(int chunk, int experts, F&& f) {
  if (experts <= 16) return f(RCfg<E, 4, 4, 64>());
  if (experts <= 32) return f(RCfg<E, 4, 8, 64>());
  if (experts <= 64) return f(RCfg<E, 8, 8, 64>());
  if (experts <= 96) return f(RCfg<E, 8, 12, 64>());
  if (experts <= 128) return f(RCfg<E, 8, 16, 64>());
  if (experts <= 192) return f(RCfg<E, 16, 12, 64>());
  if (experts <= 256) return f(RCfg<E, 16, 16, 64>());
  if (experts <= 384) return chunk == 32 ? f(RCfg<E, 32, 12, 32>()) : f(RCfg<E, 32, 12, 16>());
  if (experts <= 512) return chunk == 32 ? f(RCfg<E, 32, 16, 32>()) : f(RCfg<E, 32, 16, 16>());
  if (experts <= 768) return chunk == 16 ? f(RCfg<E, 64, 12, 16>()) : f(RCfg<E, 64, 12, 8>());
  return chunk == 16 ? f(RCfg<E, 64, 16, 16>()) : f(RCfg<E, 64, 16, 8>());
}
template <typename F>
hipError_t with_cfg(const RouteParams& p, F&& f) {
  const int chunk = chunk_of(p.rows, p.experts);
  return p.dtype == PMX_BF16 ? with_cfg<uint16_t>(chunk, p.experts, f) : with_cfg<float>(chunk, p.experts, f);
}

}  // namespace

size_t route_workspace(int64_t rows, int experts) {
  if (one_launch(rows, experts)) return 0;
  const int64_t c = chunks_of(rows, experts);
  return route_ws(nullptr, c, experts, !counts_in_scatter(c, experts)).bytes;
}

hipError_t launch_route(const RouteParams& p, hipStream_t s) {
  const int64_t chunks = chunks_of(p.rows, p.experts);
  const bool between = !counts_in_scatter(chunks, p.experts), one = one_launch(p.rows, p.experts);
  hipError_t e = with_cfg(p, [&](auto c) {
    typedef decltype(c) C;
    if (one) route_one_kernel<C><<<1, C::THREADS, 0, s>>>(p);
    else route_rows_kernel<C><<<dim3((unsigned)chunks), C::THREADS, 0, s>>>(p, chunks, between);
    return hipGetLastError();
  });
  if (e != hipSuccess || one) return e;
  if (between) {
    route_scan_kernel<<<dim3((p.experts + 15) / 16), 1024, 0, s>>>(p, chunks);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  route_scatter_kernel<<<dim3((unsigned)(chunks + (p.experts + 15) / 16)), kScatter, 0, s>>>(p, chunk_of(p.rows, p.experts), chunks, between);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteParams& p, hipStream_t s) {
  return with_cfg(p, [&](auto c) {
    typedef decltype(c) C;
    const int64_t blocks = std::min<int64_t>((p.rows + 256 / C::T - 1) / (256 / C::T), (int64_t)p.num_cu * 8);
    route_grad_kernel<C><<<dim3((unsigned)blocks), 256, 0, s>>>(p);
    return hipGetLastError();
  });
}

}  // namespace pmx
