// Router of an expert layer: softmax, the top k experts of each token, their
// gates, counts, the order of the pairs by expert, and the balance loss with
// its gradient.  Formulas and edge cases: include/pmx.h.
//
// Design: the tokens are cut into chunks of up to 64, a block each.  A team of 16
// lanes (up to 128 experts) or a wave holds a token's row in registers, a lane
// neighbouring experts, so among equal logits the lowest lane with a match and
// its first match are the lowest index.  A chunk's choice of an expert is one
// 64-bit mask in LDS: its count is the mask's bits, a pair's rank the bits below
// its token, whatever order they were set in.  So the pairs are sorted by
// (expert, token) without a sort:
//   1. rows:    ids, gates, masks -> counts a chunk; sums of p and lse^2 a chunk
//   2. scan:    each expert's counts over the chunks, its total, its mean of p
//   3. scatter: offsets from the totals, each pair's row from its rank, the loss
// One chunk does everything in one launch.  Every sum has a fixed order.
//
// Bound: launches and latency; the logits are read once forward and once in the
// gradient (32768 x 64 fp32: 8 MB each).
#include <algorithm>

#include "pmx_layer.h"

namespace pmx {
namespace {

constexpr int kMaxE = PMX_MAX_GROUPS;
constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147180559945309f;

// exp(x) for x <= 0: the product's rounding error goes back in as a factor.
__device__ __forceinline__ float exp_acc(float x) {
  const float y = x * kLog2e;
  const float r = fmaf(x, kLog2e, -y) + x * kLog2eLow;
  const float e = __builtin_amdgcn_exp2f(y);
  return y > -200.f ? fmaf(e, r * kLn2, e) : 0.f;  // x = -inf: r is NaN
}

// Up to 64 tokens a chunk; shorter ones until there is one for every unit.
int chunk_of(int64_t rows) { return rows <= 64 || rows >= 16384 ? 64 : 16; }
int64_t chunks_of(int64_t rows) { return rows ? (rows + chunk_of(rows) - 1) / chunk_of(rows) : 1; }

struct RouteWs {
  int32_t* count;  // [chunks][experts]; after the scan: pairs of earlier chunks
  float* share;    // [chunks][experts] sums of p
  float* zsum;     // [chunks] sums of lse^2
  int32_t* live;   // [chunks]
  float* mean;     // [experts] sums of p over all chunks
  float* total;    // [1] sum of lse^2
};
__host__ __device__ __forceinline__ RouteWs route_ws(void* base, int64_t chunks, int experts) {
  RouteWs w;
  w.count = reinterpret_cast<int32_t*>(base);
  w.share = reinterpret_cast<float*>(w.count + chunks * experts);
  w.zsum = w.share + chunks * experts;
  w.live = reinterpret_cast<int32_t*>(w.zsum + chunks);
  w.mean = reinterpret_cast<float*>(w.live + chunks);
  w.total = w.mean + experts;
  return w;
}

// T lanes a token, V experts a lane.
template <typename E_, int T_, int V_>
struct RCfg {
  typedef E_ E;
  static constexpr int T = T_, V = V_, TEAMS = 256 / T_;
};

template <int T>
__device__ __forceinline__ float team_max(float v) {
  return T == 16 ? row_max(v) : wave_max(v);
}
template <int T>
__device__ __forceinline__ float team_sum(float v) {
  return T == 16 ? row_sum(v) : wave_sum(v);
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

struct RowStat {
  float high, sum;
  bool dead, bad;  // nothing to choose from; NaN or +inf
};
// Turns z into exp(z - max).
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
    const float d = z[j] - s.high;
    // NaN (also inf - inf, where the row holds +inf) stays
    e[j] = d == d ? exp_acc(d) : d;
  }
#pragma unroll
  for (int j = 0; j < C::V; ++j) t += e[j];
  s.sum = team_sum<C::T>(t);
  // a row of -inf gives NaN as well, but one that holds NaN beside them is bad
  bool nan = false;
#pragma unroll
  for (int j = 0; j < C::V; ++j) nan |= z[j] != z[j] || z[j] == __builtin_inff();
  const uint64_t votes = __ballot(nan);
  const int shift = (threadIdx.x & 63) & ~(C::T - 1);
  const uint64_t mine = C::T == 64 ? votes : (votes >> shift) & ((1ull << (C::T & 63)) - 1);
  s.bad = live && mine != 0;
  s.dead = !live || (!s.bad && s.high == -__builtin_inff());
  return s;
}

struct Masks {
  uint64_t bits[kMaxE];
};

// Rows of one chunk: ids and gates to memory, the chosen to the masks, sums of p
// to registers.
template <class C>
__device__ __forceinline__ void route_rows(const RouteParams& p, int64_t first, int count, Masks& M, float (&share)[C::V],
                                           float& zsum, int& live_count) {
  const int team = threadIdx.x / C::T, lane = threadIdx.x % C::T, shift = (threadIdx.x & 63) & ~(C::T - 1);
  const int rounds = (count + C::TEAMS - 1) / C::TEAMS;
  for (int i = 0; i < rounds; ++i) {
    const int at = i * C::TEAMS + team;
    const bool inside = at < count;
    const int64_t row = first + (inside ? at : count - 1);
    float z[C::V], e[C::V];
    load_logits<C>(z, p, row, lane);
    const bool live = inside && (!p.live || p.live[row] != 0);
    const RowStat s = softmax_row<C>(e, z, live);
    if (!s.dead) {
      const float inv = 1.f / s.sum;
#pragma unroll
      for (int j = 0; j < C::V; ++j) share[j] += e[j] * inv;
      if (lane == 0) {
        const float lse = s.bad ? __builtin_nanf("") : s.high + logf(s.sum);
        zsum += lse * lse;
        ++live_count;
      }
    }
    // the chosen: `mine` keeps the choices of this lane's turn (choice j of lane j)
    int my_id = -1;
    float my_gate = 0.f, chosen_sum = 0.f;
    const float none = -__builtin_inff();
    for (int k = 0; k < p.top; ++k) {
      float m = z[0];
#pragma unroll
      for (int j = 1; j < C::V; ++j) m = fmaxf(m, z[j]);
      const float best = team_max<C::T>(m);
      const uint64_t votes = __ballot(m == best);
      const uint64_t mine = C::T == 64 ? votes : (votes >> shift) & ((1ull << (C::T & 63)) - 1);
      const bool ok = best != none && !s.dead && !s.bad && mine != 0;
      const int win = ok ? __ffsll((unsigned long long)mine) - 1 : 0;
      int v = 0;
      float ev = 0.f;
      bool found = false;
#pragma unroll
      for (int j = 0; j < C::V; ++j)
        if (!found && z[j] == best) {
          found = true;
          v = j;
          ev = e[j];
        }
      if (ok && lane == win) {
#pragma unroll
        for (int j = 0; j < C::V; ++j)
          if (j == v) z[j] = none;
      }
      const int id = __shfl(lane * C::V + v, shift + win);
      const float ge = __shfl(ev, shift + win);
      if (ok) chosen_sum += ge;
      if (lane == k) {
        my_id = ok ? id : -1;
        my_gate = ok ? ge : 0.f;
      }
    }
    if (inside && lane < p.top) {
      const float gate = my_gate / (p.normalize ? chosen_sum : s.sum);
      p.ids[row * p.top + lane] = my_id;
      p.gates[row * p.top + lane] = s.dead ? 0.f : s.bad ? __builtin_nanf("") : my_id < 0 ? 0.f : gate;
      if (my_id >= 0) atomicOr((unsigned long long*)&M.bits[my_id], 1ull << at);
    }
  }
}

// Sums over the teams, in their order, of what each lane holds of its experts:
// into LDS [experts].
template <class C>
__device__ __forceinline__ void join_share(float* out, const float (&share)[C::V], int experts) {
  const int team = threadIdx.x / C::T, lane = threadIdx.x % C::T;
  for (int t = 0; t < C::TEAMS; ++t) {
    if (team == t)
#pragma unroll
      for (int j = 0; j < C::V; ++j) {
        const int e = lane * C::V + j;
        if (e < experts) out[e] = t ? out[e] + share[j] : share[j];
      }
    __syncthreads();
  }
}
__device__ __forceinline__ void join_teams(float& z, int& n, float* zs, int* ns, int teams, int lanes) {
  if (threadIdx.x % lanes == 0) {
    zs[threadIdx.x / lanes] = z;
    ns[threadIdx.x / lanes] = n;
  }
  __syncthreads();
  z = 0.f;
  n = 0;
  for (int t = 0; t < teams; ++t) {
    z += zs[t];
    n += ns[t];
  }
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

// loss = balance E / (top n) sum_e c_e P_e / n + zloss / n sum lse^2, by the first wave.
__device__ __forceinline__ void write_loss(const RouteParams& p, const int* counts, const float* sums, float zsum, int n) {
  if (threadIdx.x < 64) {
    double b = 0.0;
    for (int e = threadIdx.x; e < p.experts; e += 64) b += (double)counts[e] * (double)sums[e];
    for (int d = 32; d > 0; d >>= 1) b += __shfl_xor(b, d);
    if (threadIdx.x == 0) {
      const double nn = n;
      *p.loss = n == 0 ? 0.f
                       : (float)((p.balance != 0.f ? (double)p.balance * p.experts / (p.top * nn * nn) * b : 0.0) +
                                 (p.zloss != 0.f ? (double)p.zloss / nn * (double)zsum : 0.0));
    }
  }
}

// Rows of the pairs of a chunk: base[e] is the row of its first pair of expert e.
template <typename Base>
__device__ __forceinline__ void scatter_chunk(const RouteParams& p, int64_t first, int count, const Masks& M, Base&& base) {
  for (int i = threadIdx.x; i < count * p.top; i += blockDim.x) {
    const int at = i / p.top;
    const int64_t pair = first * p.top + i;
    const int e = p.ids[pair];
    int slot = -1;
    if (e >= 0) {
      slot = base(e) + __popcll(M.bits[e] & ((1ull << at) - 1));
      p.tokens[slot] = (int32_t)(first + at);
    }
    p.slots[pair] = slot;
  }
}

// Everything, for up to one chunk of tokens (or none).
template <class C>
__global__ __launch_bounds__(256) void route_one_kernel(RouteParams p) {
  __shared__ Masks M;
  __shared__ float sums[kMaxE];
  __shared__ int counts[kMaxE], off[kMaxE + 1];
  __shared__ float zs[C::TEAMS];
  __shared__ int ns[C::TEAMS];
  const int count = (int)p.rows;
  for (int e = threadIdx.x; e < p.experts; e += 256) M.bits[e] = 0;
  __syncthreads();
  float share[C::V], z = 0.f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < C::V; ++j) share[j] = 0.f;
  if (count) route_rows<C>(p, 0, count, M, share, z, n);
  join_share<C>(sums, share, p.experts);  // its barriers: the masks are whole, ids written
  join_teams(z, n, zs, ns, C::TEAMS, C::T);
  for (int e = threadIdx.x; e < p.experts; e += 256) counts[e] = __popcll(M.bits[e]);
  __syncthreads();
  scan_offsets(off, counts, p.experts);
  for (int e = threadIdx.x; e <= p.experts; e += 256) {
    p.counts[e] = e < p.experts ? counts[e] : n;
    p.offsets[e] = off[e];
  }
  write_loss(p, counts, sums, z, n);
  if (p.slots) {
    __threadfence_block();
    scatter_chunk(p, 0, count, M, [&](int e) { return off[e]; });
    for (int i = off[p.experts] + threadIdx.x; i < count * p.top; i += 256) p.tokens[i] = -1;
  }
}

template <class C>
__global__ __launch_bounds__(256) void route_rows_kernel(RouteParams p, int chunk, int64_t chunks) {
  __shared__ Masks M;
  __shared__ float sums[kMaxE];
  __shared__ float zs[C::TEAMS];
  __shared__ int ns[C::TEAMS];
  const RouteWs w = route_ws(p.ws, chunks, p.experts);
  const int64_t b = blockIdx.x, first = b * chunk;
  const int count = (int)min((int64_t)chunk, p.rows - first);
  for (int e = threadIdx.x; e < p.experts; e += 256) M.bits[e] = 0;
  __syncthreads();
  float share[C::V], z = 0.f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < C::V; ++j) share[j] = 0.f;
  route_rows<C>(p, first, count, M, share, z, n);
  join_share<C>(sums, share, p.experts);
  join_teams(z, n, zs, ns, C::TEAMS, C::T);
  for (int e = threadIdx.x; e < p.experts; e += 256) {
    w.count[b * p.experts + e] = __popcll(M.bits[e]);
    w.share[b * p.experts + e] = sums[e];
  }
  if (threadIdx.x == 0) {
    w.zsum[b] = z;
    w.live[b] = n;
  }
}

// 16 experts a block, 64 segments of the chunks each.
__global__ __launch_bounds__(1024) void route_scan_kernel(RouteParams p, int64_t chunks) {
  __shared__ int part[64][17];
  __shared__ float fpart[64][17];
  const RouteWs w = route_ws(p.ws, chunks, p.experts);
  const int in = threadIdx.x & 15, seg = threadIdx.x >> 4, e = blockIdx.x * 16 + in;
  const int64_t per = (chunks + 63) / 64, c0 = min(seg * per, chunks), c1 = min(c0 + per, chunks);
  int n = 0;
  float f = 0.f;
  if (e < p.experts)
    for (int64_t c = c0; c < c1; ++c) {
      n += w.count[c * p.experts + e];
      f += w.share[c * p.experts + e];
    }
  part[seg][in] = n;
  fpart[seg][in] = f;
  __syncthreads();
  int before = 0;
  for (int s = 0; s < seg; ++s) before += part[s][in];
  if (e < p.experts) {
    for (int64_t c = c0; c < c1; ++c) {
      const int64_t i = c * p.experts + e;
      const int v = w.count[i];
      w.count[i] = before;
      before += v;
    }
    if (seg == 63) p.counts[e] = before;
    if (seg == 0) {
      float t = 0.f;
      for (int s = 0; s < 64; ++s) t += fpart[s][in];
      w.mean[e] = t;
    }
  }
  if (blockIdx.x) return;
  // the chunks' sums of lse^2 and live tokens
  __syncthreads();
  const int64_t per1 = (chunks + 1023) / 1024, k0 = min((int64_t)threadIdx.x * per1, chunks), k1 = min(k0 + per1, chunks);
  f = 0.f;
  n = 0;
  for (int64_t c = k0; c < k1; ++c) {
    f += w.zsum[c];
    n += w.live[c];
  }
  f = wave_sum(f);
  for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d);
  if ((threadIdx.x & 63) == 0) {
    fpart[threadIdx.x >> 6][0] = f;
    part[threadIdx.x >> 6][0] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    f = 0.f;
    n = 0;
    for (int s = 0; s < 16; ++s) {
      f += fpart[s][0];
      n += part[s][0];
    }
    *w.total = f;
    p.counts[p.experts] = n;
  }
}

__global__ __launch_bounds__(256) void route_scatter_kernel(RouteParams p, int chunk, int64_t chunks) {
  __shared__ Masks M;
  __shared__ int counts[kMaxE], off[kMaxE + 1];
  const RouteWs w = route_ws(p.ws, chunks, p.experts);
  const int64_t b = blockIdx.x, first = b * chunk;
  const int count = (int)min((int64_t)chunk, p.rows - first);
  for (int e = threadIdx.x; e < p.experts; e += 256) {
    M.bits[e] = 0;
    counts[e] = p.counts[e];
  }
  __syncthreads();
  if (p.slots)
    for (int i = threadIdx.x; i < count * p.top; i += 256) {
      const int e = p.ids[first * p.top + i];
      if (e >= 0) atomicOr((unsigned long long*)&M.bits[e], 1ull << (i / p.top));
    }
  scan_offsets(off, counts, p.experts);
  if (b == 0) {
    for (int e = threadIdx.x; e <= p.experts; e += 256) p.offsets[e] = off[e];
    write_loss(p, counts, w.mean, *w.total, p.counts[p.experts]);
  }
  if (!p.slots) return;
  const int32_t* base = w.count + b * p.experts;
  scatter_chunk(p, first, count, M, [&](int e) { return off[e] + base[e]; });
  // rows behind the last pair
  const int64_t all = p.rows * p.top;
  for (int64_t i = off[p.experts] + b * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) p.tokens[i] = -1;
}

// dz = p (a - sum p a) + u zloss 2 lse / n p + the gates' part.
template <class C>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteParams p) {
  typedef typename C::E E;
  const int team = threadIdx.x / C::T, lane = threadIdx.x % C::T, shift = (threadIdx.x & 63) & ~(C::T - 1);
  const float n = (float)p.counts[p.experts], u = p.upstream ? *p.upstream : 1.f;
  const float cb = n > 0.f ? u * p.balance * (float)p.experts / ((float)p.top * n) / n : 0.f;
  const float cz = n > 0.f ? u * p.zloss * 2.f / n : 0.f;
  float a[C::V];
#pragma unroll
  for (int j = 0; j < C::V; ++j) {
    const int e = lane * C::V + j;
    a[j] = e < p.experts ? cb * (float)p.counts[e] : 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * C::TEAMS;
  for (int64_t base = (int64_t)blockIdx.x * C::TEAMS; base < p.rows; base += step) {
    const bool inside = base + team < p.rows;
    const int64_t row = inside ? base + team : p.rows - 1;
    float z[C::V], e[C::V];
    load_logits<C>(z, p, row, lane);
    int my_id = -1;
    float my_g = 0.f, my_d = 0.f;
    if (p.dgates && lane < p.top) {
      my_id = p.ids[row * p.top + lane];
      my_g = p.gates[row * p.top + lane];
      my_d = p.dgates[row * p.top + lane];
      if (my_id < 0) my_g = my_d = 0.f;
    }
    const RowStat s = softmax_row<C>(e, z, inside && (!p.live || p.live[row] != 0));
    const float inv = 1.f / s.sum;
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < C::V; ++j) {
      e[j] *= inv;
      dot += e[j] * a[j];
    }
    dot = team_sum<C::T>(dot);
    const float gd = p.dgates ? team_sum<C::T>(my_g * my_d) : 0.f;
    // p's factor: the balance and z parts, and without normalisation the gates' own
    const float lse = s.high + logf(s.sum);
    const float all = cz * lse - dot - (p.normalize ? 0.f : gd);
#pragma unroll
    for (int j = 0; j < C::V; ++j) z[j] = e[j] * (a[j] + all);
    if (p.dgates) {
      // the chosen ones': normalised g (dg - sum g dg), else g dg
      const float mine = my_g * (my_d - (p.normalize ? gd : 0.f));
      for (int k = 0; k < p.top; ++k) {
        const int id = __shfl(my_id, shift + k);
        const float d = __shfl(mine, shift + k);
#pragma unroll
        for (int j = 0; j < C::V; ++j)
          if (lane * C::V + j == id) z[j] += d;
      }
    }
    if (inside) {
      E* dz = reinterpret_cast<E*>(p.dz) + row * p.lddz;
#pragma unroll
      for (int j = 0; j < C::V; ++j) {
        const int i = lane * C::V + j;
        const float v = s.dead ? 0.f : s.bad ? __builtin_nanf("") : z[j];
        if (i < p.experts) {
          if constexpr (sizeof(E) == 2) dz[i] = (E)pack_bf16(v, 0.f);
          else dz[i] = v;
        }
      }
    }
  }
}

template <typename E, typename F>
hipError_t with_cfg(int experts, F&& f) {
  if (experts <= 64) return f(RCfg<E, 16, 4>());
  if (experts <= 128) return f(RCfg<E, 16, 8>());
  if (experts <= 256) return f(RCfg<E, 64, 4>());
  if (experts <= 512) return f(RCfg<E, 64, 8>());
  return f(RCfg<E, 64, 16>());
}
template <typename F>
hipError_t with_cfg(const RouteParams& p, F&& f) {
  return p.dtype == PMX_BF16 ? with_cfg<uint16_t>(p.experts, f) : with_cfg<float>(p.experts, f);
}

}  // namespace

size_t route_workspace(int64_t rows, int experts) {
  if (rows <= 64) return 0;
  const int64_t c = chunks_of(rows);
  return (size_t)(2 * c * experts + 2 * c + experts + 1) * 4;
}

hipError_t launch_route(const RouteParams& p, hipStream_t s) {
  const hipError_t e = with_cfg(p, [&](auto c) {
    typedef decltype(c) C;
    if (p.rows <= 64) route_one_kernel<C><<<1, 256, 0, s>>>(p);
    else route_rows_kernel<C><<<dim3((unsigned)chunks_of(p.rows)), 256, 0, s>>>(p, chunk_of(p.rows), chunks_of(p.rows));
    return hipGetLastError();
  });
  if (e != hipSuccess || p.rows <= 64) return e;
  const int64_t chunks = chunks_of(p.rows);
  route_scan_kernel<<<dim3((p.experts + 15) / 16), 1024, 0, s>>>(p, chunks);
  const hipError_t e1 = hipGetLastError();
  if (e1 != hipSuccess) return e1;
  route_scatter_kernel<<<dim3((unsigned)chunks), 256, 0, s>>>(p, chunk_of(p.rows), chunks);
  return hipGetLastError();
}

hipError_t launch_route_grad(const RouteParams& p, hipStream_t s) {
  return with_cfg(p, [&](auto c) {
    typedef decltype(c) C;
    const int64_t blocks = std::min<int64_t>((p.rows + C::TEAMS - 1) / C::TEAMS, (int64_t)p.num_cu * 8);
    route_grad_kernel<C><<<dim3((unsigned)blocks), 256, 0, s>>>(p);
    return hipGetLastError();
  });
}

}  // namespace pmx
