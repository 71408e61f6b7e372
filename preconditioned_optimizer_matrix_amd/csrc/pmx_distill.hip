// Distillation loss from a teacher's top logits, with its gradient.
//
// Mathematics (pmx_train.h has the formulas).  A row needs the maximum m of
// its logits, S_tau = sum exp((z - m) / tau) and S_1 = sum exp(z - m); with
// e_i = exp((a_i - max a) / tau) over the teacher's listed logits a_i and
// A = sum e_i, the Kullback-Leibler part is
//   (sum e_i (a_i - max a) / tau - sum e_i (z_{id_i} - m) / tau) / A - log A + log S_tau,
// so one reduction for the two maxima and one for the five sums give the
// loss, and the gradient is a multiple of the same exponentials plus a
// correction at the top + 1 listed columns.  All sums are fp32; a row's loss
// terms are O(log vocab), so fp32 holds them to a few 1e-7.
//
// Bound: HBM.  The logits are read once and the gradient written once: the
// row stays in registers between the two (up to 16 16-byte chunks a thread,
// up to 1024 threads: 128 Ki bf16 or 64 Ki fp32 logits), packed as it was
// loaded.  Blocks are persistent: as soon as a chunk's gradient is computed,
// its registers take the load of the block's next row, so the loads run under
// the exponentials and the stores.  Longer rows are read three times, for the
// maximum, the sums and the gradient.  When there are few long rows, a row is cut
// over several blocks: one launch for partial sums, one for the rest.
// exp(z - m) is the tau-th power of exp((z - m) / tau): for tau = 2, 4 or 8 it
// is squared up instead of a second exponential (a quarter-rate instruction).
//
// Measured, 8192 rows of 128000 bf16 with the gradient, tau = 2, a tenth of the
// rows ignored: 927 us for 4.0 GB, 4.3 TB/s where a copy reaches 5.1 (936 to 1038 one
// call at a time under a profiler).  4096 rows of 50000 fp32: 405 us, 4.0 TB/s.
// 1023 rows of 32003 bf16, the loss 19 us, the later gradient 25.  7 rows of 128000
// fp32: 5 us for the partial sums, 8 for the rest.  Rows past the registers, 4096 of
// 151936 bf16: 873 us, all three reads and the write beyond the L2s (5.0 GB, 5.7
// TB/s); 490 would be one read and the write.  A list of many entries costs a
// block entries^2 / threads steps where it corrects the gradient: 1024 rows of 32000
// bf16, 20 entries 37 us, 1023 entries 312.
#include <algorithm>

#include "pmx_train.h"

namespace pmx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;
constexpr int kFewRows = 32;        // at most so many rows are cut over several blocks
constexpr int kMiddleRow = 512 * 16;  // chunks of a row that fit a block's registers without 1024 threads
constexpr int kLongRow = 1024 * 16;   // with them

// exponentials per element: one (a single temperature is in play), two, or one
// and 1, 2 or 3 squarings
enum Exps : int { EXP_ONE = 0, EXP_TWO = 1, EXP_SQ1 = 2, EXP_SQ2 = 3, EXP_SQ3 = 4 };

typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  static constexpr uint32_t NEG = 0xFF800000u;  // -inf
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
  static __device__ __forceinline__ float get(const u32x4_t& v, int j) {
    return __uint_as_float(v[j]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&x)[4]) {
    return {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
            __float_as_uint(x[3])};
  }
};
template <>
struct Elem<uint16_t> {
  static constexpr int VEC = 8;
  static constexpr uint32_t NEG = 0xFF80FF80u;
  static __device__ __forceinline__ float load(const uint16_t* p) {
    return __uint_as_float((uint32_t)*p << 16);
  }
  static __device__ __forceinline__ void store(uint16_t* p, float v) {
    *p = (uint16_t)pack_bf16(v, 0.f);
  }
  static __device__ __forceinline__ float get(const u32x4_t& v, int j) {
    return (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float (&x)[8]) {
    return {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
            pack_bf16(x[6], x[7])};
  }
};

// A row as whole 16-byte aligned chunks and the few elements before and after
// them (fewer than VEC each): element i of those is i < head from the row's
// start, else from the chunks' end.
template <typename T>
struct Row {
  static constexpr int VEC = Elem<T>::VEC;
  int head, chunks, edges;
  __device__ __forceinline__ Row(const T* row, int n) {
    head = (int)((16 - ((uintptr_t)row & 15)) & 15) / (int)sizeof(T);
    if (head > n) head = n;
    chunks = (n - head) / VEC;
    edges = n - chunks * VEC;
  }
  __device__ __forceinline__ int edge(int i) const { return i < head ? i : chunks * VEC + i; }
};

// Chunk `i` from a base that is the same for the whole block: a scalar address
// and a 32-bit offset.
template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const T* base, uint32_t i) {
  return *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(base) + 16u * i);
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* base, uint32_t i, const float (&x)[Elem<T>::VEC]) {
  // the gradient's rows may be aligned otherwise
  *reinterpret_cast<u32x4_a2*>(reinterpret_cast<char*>(base) + 16u * i) = Elem<T>::pack(x);
}

// Exponentials of one logit: et = exp((z - m) / tau), e1 = exp(z - m).  The
// difference comes first: one fused multiply-add with a rounded -m / tau would
// be off by 2^-24 |m / tau| in the exponent, and overflow for rows masked with
// the type's lowest value.
template <int EX>
struct Expo {
  float m, a, rt;
  __device__ __forceinline__ Expo(const DistillParams& p, float m_) {
    m = m_;
    // the only temperature of EXP_ONE: tau, or 1 where only the label counts
    rt = 1.f / (EX == EXP_ONE && p.mix == 0.f ? 1.f : p.tau);
    a = kLog2e * rt;
  }
  __device__ __forceinline__ void operator()(float z, float& et, float& e1) const {
    const float d = z - m;
    et = __builtin_amdgcn_exp2f(d * a);
    if (EX == EXP_ONE) e1 = et;
    if (EX == EXP_TWO) e1 = __builtin_amdgcn_exp2f(d * kLog2e);
    if (EX >= EXP_SQ1) e1 = et * et;
    if (EX >= EXP_SQ2) e1 *= e1;
    if (EX >= EXP_SQ3) e1 *= e1;
  }
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <int NT, int N>
__device__ __forceinline__ void block_max(float (&v)[N], float (*red)[16]) {
  constexpr int W = NT / 64;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_max(v[i]);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][wid] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float m = red[i][lane & (W - 1)];
#pragma unroll
    for (int o = W / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    v[i] = m;
  }
  __syncthreads();
}

template <int NT, int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[16]) {
  constexpr int W = NT / 64;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][wid] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float m = red[i][lane & (W - 1)];
#pragma unroll
    for (int o = W / 2; o; o >>= 1) m += __shfl_xor(m, o);
    v[i] = m;
  }
  __syncthreads();
}

// The listed columns of a row: the teacher's entries and, last, the label.
// Entries outside the vocabulary have id -1.
constexpr int kListed = PMX_MAX_TOP + 1;
struct Listed {
  int id[kListed];
  float e[kListed];  // teacher logit, then exp((... - max) / tau)
  float z[kListed];  // the student's logit there
};

// A thread's listed entries, on the way from memory (fetch, issued under the
// previous row's work) to LDS (put).
template <typename T, int NT>
struct Fetched {
  static constexpr int N = (kListed + NT - 1) / NT;
  int id[N];
  float a[N], z[N];
  // saved: the listed logits as distill_part_kernel kept them, not the row's
  // (which other blocks may be overwriting with the gradient)
  __device__ __forceinline__ void fetch(const DistillParams& p, int64_t t, const float* saved = nullptr) {
    const T* row = reinterpret_cast<const T*>(p.z) + t * p.ldz;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + NT * k;
      int64_t d = -1;
      a[k] = kNegInf;
      z[k] = 0.f;
      if (i < p.top) {
        d = load_index(p.ids, t * p.ld_ids + i, p.ids64);
        if (d >= 0 && d < p.vocab) {
          const int64_t o = t * p.ld_teacher + i;
          a[k] = p.teacher_dtype == PMX_F32 ? reinterpret_cast<const float*>(p.teacher)[o]
                                            : Elem<uint16_t>::load(reinterpret_cast<const uint16_t*>(p.teacher) + o);
        }
      } else if (i == p.top && p.labels) {
        d = load_index(p.labels, t, p.labels64);
      }
      if (d < 0 || d >= p.vocab) d = -1;
      id[k] = (int)d;
      if (d >= 0) z[k] = saved ? saved[i] : Elem<T>::load(row + d);
    }
  }
  __device__ __forceinline__ float put(Listed& L, const DistillParams& p) const {
    float amax = kNegInf;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + NT * k;
      if (i <= p.top) {
        L.id[i] = id[k];
        L.e[i] = a[k];
        L.z[i] = z[k];
        amax = fmaxf(amax, a[k]);
      }
    }
    return amax;
  }
};

// L.e becomes e = exp((a - am) / tau); sum[0] += e, sum[1] += e (a - am) / tau,
// sum[2] += e (z - m) / tau.  The difference comes before the temperature, as in Expo.
template <int NT, int EX>
__device__ __forceinline__ void teacher_sums(Listed& L, const DistillParams& p, const Expo<EX>& ex,
                                             float am, float (&sum)[5]) {
  for (int i = threadIdx.x; i < p.top; i += NT) {
    const float a = (L.e[i] - am) * ex.rt;
    const float e = __builtin_amdgcn_exp2f(a * kLog2e);
    L.e[i] = e;
    sum[0] += e;
    if (e != 0.f) {  // nothing (not NaN) where the teacher gives no weight
      sum[1] += e * a;
      sum[2] += e * (L.z[i] - ex.m) * ex.rt;
    }
  }
}

// The row's loss from its sums.
template <int EX>
__device__ __forceinline__ float row_loss(const DistillParams& p, bool label, float z_label, const Expo<EX>& ex,
                                          const float (&v)[5]) {
  float loss = 0.f;
  if (v[3] != 0.f) {  // a row of nothing but -inf has none
    if (p.mix != 0.f && v[0] != 0.f)
      loss += p.mix * p.tau * p.tau * ((v[1] - v[2]) / v[0] - logf(v[0]) + logf(v[3]));
    if (p.mix != 1.f && label) loss += (1.f - p.mix) * (logf(v[4]) - (z_label - ex.m));
  }
  return loss;
}

// Gradient scales: gt and g1 multiply the exponentials (one temperature: gt
// alone carries both), gp the teacher's e_i, gc the label's one.
struct Scales {
  float gt, g1, gp, gc;
};
template <int EX>
__device__ __forceinline__ Scales grad_scales(const DistillParams& p, float w, float inv_t,
                                              float inv_1, float sum_e, bool label) {
  const bool row = inv_t != 0.f;  // a row of nothing but -inf has no gradient
  const float kd = row && sum_e != 0.f && p.mix != 0.f ? w * p.mix * p.tau : 0.f;
  const float ce = row && label && p.mix != 1.f ? w * (1.f - p.mix) : 0.f;
  Scales s;
  s.gt = kd * inv_t;
  s.g1 = ce * inv_1;
  if (EX == EXP_ONE) s.gt += s.g1;
  s.gp = kd != 0.f ? kd / sum_e : 0.f;
  s.gc = ce;
  return s;
}
__device__ __forceinline__ float inverse(float s) { return s != 0.f ? 1.f / s : 0.f; }

template <int EX>
__device__ __forceinline__ float grad_of(float z, const Expo<EX>& ex, const Scales& s) {
  float et, e1;
  ex(z, et, e1);
  return EX == EXP_ONE ? s.gt * et : s.gt * et + s.g1 * e1;
}

template <typename T, int EX>
__device__ __forceinline__ void add_chunk(const Expo<EX>& ex, const u32x4_t& u, float& st, float& s1) {
#pragma unroll
  for (int j = 0; j < Elem<T>::VEC; ++j) {
    float et, e1;
    ex(Elem<T>::get(u, j), et, e1);
    st += et;
    if (EX != EXP_ONE) s1 += e1;
  }
}
template <typename T, int EX>
__device__ __forceinline__ void grad_chunk(const Expo<EX>& ex, const Scales& s, const u32x4_t& u,
                                           float (&x)[Elem<T>::VEC]) {
#pragma unroll
  for (int j = 0; j < Elem<T>::VEC; ++j) x[j] = grad_of(Elem<T>::get(u, j), ex, s);
}

// Corrections of the gradient at the listed columns [lo, hi), over dense
// values already written by this block.  Every entry naming the same column
// writes the same value.
template <typename T, int NT, int EX>
__device__ __forceinline__ void fix_listed(const Listed& L, const DistillParams& p, T* dz,
                                           const Expo<EX>& ex, const Scales& s, int lo, int hi) {
  for (int i = threadIdx.x; i <= p.top; i += NT) {
    const int id = L.id[i];
    if (id < 0 || id < lo || id >= hi) continue;
    float v = grad_of(L.z[i], ex, s);
    if (p.mix != 0.f) {  // (without the teacher's part its logits may hold anything)
      float ps = 0.f;
      for (int j = 0; j < p.top; ++j) ps += L.id[j] == id ? L.e[j] : 0.f;
      v -= s.gp * ps;
    }
    if (L.id[p.top] == id) v -= s.gc;
    Elem<T>::store(dz + id, v);
  }
}

__device__ __forceinline__ float weight_of(const DistillParams& p, int64_t t) {
  return p.weights ? p.weights[t] : 1.f / (float)p.rows;
}

template <typename T, int NT>
__device__ __forceinline__ void clear_row(T* row, int n) {
  const Row<T> r(row, n);
  const float zero[Elem<T>::VEC] = {};
  for (int c = threadIdx.x; c < r.chunks; c += NT) store_chunk<T>(row + r.head, c, zero);
  for (int i = threadIdx.x; i < r.edges; i += NT) Elem<T>::store(row + r.edge(i), 0.f);
}

// The next row from t on that counts; ignored rows on the way get their zeros.
// p.rows: none.  `after(t)` is the row that follows t for this block.
template <typename T, int NT, bool GRAD, typename F>
__device__ __forceinline__ int64_t next_live(const DistillParams& p, int64_t t, F&& after) {
  while (t < p.rows) {
    if (weight_of(p, t) != 0.f) return t;
    if (threadIdx.x == 0) {
      p.rows_loss[t] = 0.f;
      if (p.stats) p.stats[3 * t] = p.stats[3 * t + 1] = p.stats[3 * t + 2] = 0.f;
    }
    if (GRAD) clear_row<T, NT>(reinterpret_cast<T*>(p.dz) + t * p.lddz, p.vocab);
    t = after(t);
  }
  return p.rows;
}

// First row of the rows that blocks claim (the first gridDim.x are dealt out).
__global__ void distill_claim_kernel(uint32_t* next, uint32_t first) { *next = first; }

// Waves a SIMD for NC chunks a thread: registers for the row (4 NC) and 50
// to 60 more.
constexpr int waves_for(int nc) { return nc <= 4 ? 6 : nc <= 8 ? 5 : 4; }

// Keeps a chunk packed: without it the compiler holds on to the unpacked
// values from one phase to the next, twice the registers for bf16.
__device__ __forceinline__ void stay_packed(u32x4_t& v) { asm volatile("" : "+v"(v)); }

// Rows in registers: NC chunks a thread and one edge element.
template <typename T, int NT, int NC, int EX, bool GRAD>
__global__ __launch_bounds__(NT, waves_for(NC)) void distill_row_kernel(DistillParams p) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ Listed L;
  __shared__ float red[5][16];
  const int n = p.vocab, tid = threadIdx.x;
  u32x4_t v[NC];
  float edge;
  Fetched<T, NT> f;
  // every lane loads, from the row's last chunk where it has none (no branch:
  // a value joined from two paths costs the row's registers twice); `mask`
  // makes such chunks -inf before their first use
  auto load_one = [&](const T* body, int last, int c) {
    int i = tid;
    asm volatile("" : "+v"(i));  // the offset is computed here, not kept from row to row
    v[c] = load_chunk<T>(body, (uint32_t)min(i + c * NT, last));
  };
  auto mask = [&](int last, int c) {
    const bool out = tid > last - c * NT;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[c][k] = out ? Elem<T>::NEG : v[c][k];
  };
  auto load_edge = [&](const T* z, const Row<T>& r) {
    edge = tid < r.edges ? Elem<T>::load(z + r.edge(tid)) : kNegInf;
  };
  // CLAIM: after its first row a block takes the next one nobody has taken, so
  // that blocks with many ignored rows do not finish early (with 10% of 8192
  // rows ignored, the block with most rows to do had 32 where the mean is 28.8)
  constexpr bool CLAIM = NT == 1024;
  __shared__ uint32_t claimed;
  auto after = [&](int64_t t) -> int64_t {
    if constexpr (CLAIM) {
      __syncthreads();
      if (threadIdx.x == 0) claimed = atomicAdd(p.next_row, 1u);
      __syncthreads();
      return claimed;
    } else {
      return t + gridDim.x;
    }
  };
  int64_t t = next_live<T, NT, GRAD>(p, blockIdx.x, after);
  if constexpr (CLAIM) __syncthreads();  // every wave has read `claimed` before the first row's claim overwrites it
  if (t >= p.rows) return;
  {
    const T* z = reinterpret_cast<const T*>(p.z) + t * p.ldz;
    const Row<T> r(z, n);
#pragma unroll
    for (int c = 0; c < NC; ++c) load_one(z + r.head, r.chunks - 1, c);
    load_edge(z, r);
    f.fetch(p, t);
  }
  for (;;) {
    const Row<T> r(reinterpret_cast<const T*>(p.z) + t * p.ldz, n);
    if (CLAIM && tid == 0) claimed = atomicAdd(p.next_row, 1u);  // read after block_max
    float mx[2];
    mx[0] = edge;
    mx[1] = f.put(L, p);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      mask(r.chunks - 1, c);
#pragma unroll
      for (int j = 0; j < VEC; j += 2)
        mx[0] = fmaxf(fmaxf(mx[0], Elem<T>::get(v[c], j)), Elem<T>::get(v[c], j + 1));
      stay_packed(v[c]);
    }
    block_max<NT>(mx, red);
    const float am = mx[1] == kNegInf ? 0.f : mx[1];
    const Expo<EX> ex(p, mx[0] == kNegInf ? 0.f : mx[0]);  // -inf - 0 stays -inf
    const int64_t tn = next_live<T, NT, GRAD>(p, CLAIM ? (int64_t)claimed : t + gridDim.x, after);
    // without a next row every lane loads this row's first chunk again
    const bool more = tn < p.rows;
    const T* zn = reinterpret_cast<const T*>(p.z) + (more ? tn : t) * p.ldz;
    const Row<T> rn(zn, n);
    const T* body = zn + rn.head;
    const int last = more ? rn.chunks - 1 : 0;
    float sum[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    teacher_sums<NT>(L, p, ex, am, sum);
    {
      float et, e1;
      ex(edge, et, e1);
      sum[3] += et;
      if (EX != EXP_ONE) sum[4] += e1;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      add_chunk<T>(ex, v[c], sum[3], sum[4]);
      if (GRAD) {
        stay_packed(v[c]);
      } else {
        // the sums are taken here, before the registers are loaded again
        asm volatile("" : "+v"(sum[3]), "+v"(sum[4]) : : "memory");
        load_one(body, last, c);
      }
    }
    if (EX == EXP_ONE) sum[4] = sum[3];
    asm volatile("" : "+v"(sum[3]), "+v"(sum[4]) : : "memory");
    const float own_edge = edge;
    if (!GRAD) load_edge(zn, rn);
    if (more) f.fetch(p, tn);
    block_sum<NT>(sum, red);
    if (tid == 0) {
      p.rows_loss[t] = row_loss(p, L.id[p.top] >= 0, L.z[p.top], ex, sum);
      if (p.stats) {
        p.stats[3 * t] = ex.m;
        p.stats[3 * t + 1] = inverse(sum[3]);
        p.stats[3 * t + 2] = inverse(sum[4]);
      }
    }
    if constexpr (GRAD) {
      T* dz = reinterpret_cast<T*>(p.dz) + t * p.lddz;
      const Scales s = grad_scales<EX>(p, weight_of(p, t), inverse(sum[3]), inverse(sum[4]), sum[0],
                                       L.id[p.top] >= 0);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float x[VEC];
        grad_chunk<T>(ex, s, v[c], x);
        if (tid < r.chunks - c * NT) store_chunk<T>(dz + r.head + c * NT * VEC, tid, x);
        load_one(body, last, c);
      }
      if (tid < r.edges) Elem<T>::store(dz + r.edge(tid), grad_of(own_edge, ex, s));
      load_edge(zn, rn);
      __syncthreads();
      fix_listed<T, NT>(L, p, dz, ex, s, 0, n);
    }
    if (!more) return;
    __syncthreads();  // L is free
    t = tn;
  }
}

// Rows too long for the registers: read three times.
template <typename T, int EX, bool GRAD>
__global__ __launch_bounds__(1024) void distill_long_kernel(DistillParams p) {
  constexpr int VEC = Elem<T>::VEC, NT = 1024;
  __shared__ Listed L;
  __shared__ float red[5][16];
  const int n = p.vocab, tid = threadIdx.x;
  auto after = [](int64_t t) -> int64_t { return t + gridDim.x; };
  for (int64_t t = blockIdx.x; (t = next_live<T, NT, GRAD>(p, t, after)) < p.rows; t += gridDim.x) {
    const T* z = reinterpret_cast<const T*>(p.z) + t * p.ldz;
    const Row<T> r(z, n);
    const T* body = z + r.head;
    Fetched<T, NT> f;
    f.fetch(p, t);
    float mx[2];
    mx[0] = tid < r.edges ? Elem<T>::load(z + r.edge(tid)) : kNegInf;
    const float edge = mx[0];
    mx[1] = f.put(L, p);
#pragma unroll 4
    for (int c = tid; c < r.chunks; c += NT) {
      const u32x4_t u = load_chunk<T>(body, c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) mx[0] = fmaxf(mx[0], Elem<T>::get(u, j));
    }
    block_max<NT>(mx, red);
    const float am = mx[1] == kNegInf ? 0.f : mx[1];
    const Expo<EX> ex(p, mx[0] == kNegInf ? 0.f : mx[0]);
    float sum[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    teacher_sums<NT>(L, p, ex, am, sum);
    ex(edge, sum[3], sum[4]);
#pragma unroll 4
    for (int c = tid; c < r.chunks; c += NT) {
      const u32x4_t u = load_chunk<T>(body, c);
      add_chunk<T>(ex, u, sum[3], sum[4]);
    }
    if (EX == EXP_ONE) sum[4] = sum[3];
    block_sum<NT>(sum, red);
    if (tid == 0) {
      p.rows_loss[t] = row_loss(p, L.id[p.top] >= 0, L.z[p.top], ex, sum);
      if (p.stats) {
        p.stats[3 * t] = ex.m;
        p.stats[3 * t + 1] = inverse(sum[3]);
        p.stats[3 * t + 2] = inverse(sum[4]);
      }
    }
    if constexpr (GRAD) {
      T* dz = reinterpret_cast<T*>(p.dz) + t * p.lddz;
      const Scales s = grad_scales<EX>(p, weight_of(p, t), inverse(sum[3]), inverse(sum[4]), sum[0],
                                       L.id[p.top] >= 0);
#pragma unroll 4
      for (int c = tid; c < r.chunks; c += NT) {
        const u32x4_t u = load_chunk<T>(body, c);
        float x[VEC];
        grad_chunk<T>(ex, s, u, x);
        store_chunk<T>(dz + r.head, c, x);
      }
      if (tid < r.edges) Elem<T>::store(dz + r.edge(tid), grad_of(edge, ex, s));
      __syncthreads();
      fix_listed<T, NT>(L, p, dz, ex, s, 0, n);
    }
    __syncthreads();
  }
}

// Block (x, y) has slab x of row y.  A slab is a range
// of whole chunks; the row's edges belong to slab 0.
template <typename T>
struct Slab {
  int c0, c1, edges;
  __device__ __forceinline__ Slab(const Row<T>& r, int slabs) {
    const int per = (r.chunks + slabs - 1) / slabs;
    c0 = min((int)blockIdx.x * per, r.chunks);
    c1 = min(c0 + per, r.chunks);
    edges = blockIdx.x == 0 ? r.edges : 0;
  }
};

// The listed logits kept for the second launch, behind the partial sums.
__device__ __forceinline__ float* saved_of(const DistillParams& p, int64_t t) {
  return p.part + p.rows * p.splits * 3 + t * (p.top + 1);
}

// Partial sums of a slab, relative to the slab's own maximum:
// part[row][slab] = {max, S_tau, S_1}.  Slab 0 also keeps the listed logits.
template <typename T, int EX>
__global__ __launch_bounds__(256) void distill_part_kernel(DistillParams p) {
  constexpr int VEC = Elem<T>::VEC, NT = 256;
  __shared__ float red[2][16];
  const int64_t t = blockIdx.y;
  const int tid = threadIdx.x;
  if (weight_of(p, t) == 0.f) return;
  const T* z = reinterpret_cast<const T*>(p.z) + t * p.ldz;
  const Row<T> r(z, p.vocab);
  const Slab<T> b(r, (int)gridDim.x);
  if (blockIdx.x == 0) {
    Fetched<T, NT> f;
    f.fetch(p, t);
#pragma unroll
    for (int k = 0; k < f.N; ++k)
      if (tid + NT * k <= p.top) saved_of(p, t)[tid + NT * k] = f.z[k];
  }
  const float edge = tid < b.edges ? Elem<T>::load(z + r.edge(tid)) : kNegInf;
  float mx[1];
  mx[0] = edge;
#pragma unroll 4
  for (int c = b.c0 + tid; c < b.c1; c += NT) {
    const u32x4_t u = load_chunk<T>(z + r.head, c);
#pragma unroll
    for (int j = 0; j < VEC; ++j) mx[0] = fmaxf(mx[0], Elem<T>::get(u, j));
  }
  block_max<NT>(mx, red);
  const Expo<EX> ex(p, mx[0] == kNegInf ? 0.f : mx[0]);
  float sum[2];
  ex(edge, sum[0], sum[1]);
#pragma unroll 4
  for (int c = b.c0 + tid; c < b.c1; c += NT) {
    const u32x4_t u = load_chunk<T>(z + r.head, c);
    add_chunk<T>(ex, u, sum[0], sum[1]);
  }
  if (EX == EXP_ONE) sum[1] = sum[0];
  block_sum<NT>(sum, red);
  if (tid == 0) {
    float* q = p.part + (t * gridDim.x + blockIdx.x) * 3;
    q[0] = mx[0];
    q[1] = sum[0];
    q[2] = sum[1];
  }
}

// The row's maximum and sums from its slabs' (at most 64, one a lane), in every
// wave.
template <int EX>
__device__ __forceinline__ float join_parts(const DistillParams& p, int64_t t, float& st, float& s1) {
  const int lane = threadIdx.x & 63;
  const float* q = p.part + (t * p.splits + min(lane, p.splits - 1)) * 3;
  const bool in = lane < p.splits;
  const float mi = in ? q[0] : kNegInf, ti = in ? q[1] : 0.f, oi = in ? q[2] : 0.f;
  float m = wave_max(mi);
  if (m == kNegInf) m = 0.f;
  const Expo<EX> ex(p, m);
  // a slab of nothing but -inf has zero sums (NaN ones stay NaN)
  const float d = (mi == kNegInf ? 0.f : mi) - m;
  const float ft = __builtin_amdgcn_exp2f(d * ex.a);
  const float f1 = EX == EXP_ONE ? ft : __builtin_amdgcn_exp2f(d * kLog2e);
  st = wave_sum(ti != 0.f ? ti * ft : 0.f);
  s1 = wave_sum(oi != 0.f ? oi * f1 : 0.f);
  return m;
}

// Losses, statistics and the total of few rows from the slabs' sums: one block,
// a wave a row.
template <int EX>
__device__ void few_rows_loss(const DistillParams& p) {
  __shared__ double part[kFewRows];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int64_t t = wid; t < p.rows; t += waves) {
    const float w = weight_of(p, t);
    float m = 0.f, st = 0.f, s1 = 0.f, loss = 0.f;
    if (w != 0.f) {
      const float* z = saved_of(p, t);
      m = join_parts<EX>(p, t, st, s1);
      const Expo<EX> ex(p, m);
      auto entry = [&](int i) {  // teacher logit, -inf outside the vocabulary
        const int64_t id = load_index(p.ids, t * p.ld_ids + i, p.ids64), o = t * p.ld_teacher + i;
        if (id < 0 || id >= p.vocab) return kNegInf;
        return p.teacher_dtype == PMX_F32 ? reinterpret_cast<const float*>(p.teacher)[o]
                                          : Elem<uint16_t>::load(reinterpret_cast<const uint16_t*>(p.teacher) + o);
      };
      float am = kNegInf;
      for (int i = lane; i < p.top; i += 64) am = fmaxf(am, entry(i));
      am = wave_max(am);
      if (am == kNegInf) am = 0.f;
      float sum[5] = {0.f, 0.f, 0.f, st, s1};
      for (int i = lane; i < p.top; i += 64) {
        const float a = (entry(i) - am) * ex.rt, e = __builtin_amdgcn_exp2f(a * kLog2e);
        sum[0] += e;
        if (e != 0.f) {
          sum[1] += e * a;
          sum[2] += e * (z[i] - m) * ex.rt;
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) sum[i] = wave_sum(sum[i]);
      const int64_t y = p.labels ? load_index(p.labels, t, p.labels64) : -1;
      loss = row_loss(p, y >= 0 && y < p.vocab, z[p.top], ex, sum);
    }
    if (lane == 0) {
      p.rows_loss[t] = loss;
      if (p.stats) {
        p.stats[3 * t] = m;
        p.stats[3 * t + 1] = inverse(st);
        p.stats[3 * t + 2] = inverse(s1);
      }
      part[t] = w != 0.f ? (p.weights ? (double)w : 1.0 / (double)p.rows) * (double)loss : 0.0;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int t = 0; t < (int)p.rows; ++t) s += part[t];
    *p.total = (float)s;
  }
}

// One slab of one row at a time: the gradient from the saved statistics, or
// (JOIN) from the slabs' sums of distill_part_kernel; then one more block has
// the losses.  A thread's first four chunks are loaded before the teacher's
// list is worked through.
template <typename T, int EX, bool JOIN>
__global__ __launch_bounds__(256) void distill_grad_kernel(DistillParams p, int slabs) {
  constexpr int VEC = Elem<T>::VEC, NT = 256, NC = 4;
  __shared__ Listed L;
  __shared__ float red[5][16];
  if (JOIN && (int)blockIdx.x == slabs) {
    if (blockIdx.y == 0) few_rows_loss<EX>(p);
    return;
  }
  const int n = p.vocab, tid = threadIdx.x;
  for (int64_t t = blockIdx.y; t < p.rows; t += gridDim.y) {
    const T* z = reinterpret_cast<const T*>(p.z) + t * p.ldz;
    T* dz = reinterpret_cast<T*>(p.dz) + t * p.lddz;
    const Row<T> r(z, n);
    const Slab<T> b(r, slabs);
    const float wt = weight_of(p, t);
    if (wt == 0.f) {
      const float zero[VEC] = {};
      for (int c = b.c0 + tid; c < b.c1; c += NT) store_chunk<T>(dz + r.head, c, zero);
      if (tid < b.edges) Elem<T>::store(dz + r.edge(tid), 0.f);
      continue;
    }
    Fetched<T, NT> f;
    f.fetch(p, t, JOIN ? saved_of(p, t) : nullptr);
    u32x4_t u[NC];
    auto load = [&](int c0) {
#pragma unroll
      for (int k = 0; k < NC; ++k)
        if (c0 + k * NT < b.c1) u[k] = load_chunk<T>(z + r.head, c0 + k * NT);
    };
    load(b.c0 + tid);
    const float edge = tid < b.edges ? Elem<T>::load(z + r.edge(tid)) : 0.f;
    float m, inv_t, inv_1;
    if (JOIN) {
      m = join_parts<EX>(p, t, inv_t, inv_1);
      inv_t = inverse(inv_t);
      inv_1 = inverse(inv_1);
    } else {
      m = p.stats[3 * t];
      inv_t = p.stats[3 * t + 1];
      inv_1 = p.stats[3 * t + 2];
    }
    const Expo<EX> ex(p, m);
    float am[1], sum[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
    am[0] = f.put(L, p);
    block_max<NT>(am, red);
    teacher_sums<NT>(L, p, ex, am[0] == kNegInf ? 0.f : am[0], sum);
    float sum_e[1] = {sum[0]};
    block_sum<NT>(sum_e, red);
    const float w = wt * (p.upstream ? *p.upstream : 1.f);
    const Scales s = grad_scales<EX>(p, w, inv_t, inv_1, sum_e[0], L.id[p.top] >= 0);
    for (int c0 = b.c0 + tid;;) {
#pragma unroll
      for (int k = 0; k < NC; ++k)
        if (c0 + k * NT < b.c1) {
          float x[VEC];
          grad_chunk<T>(ex, s, u[k], x);
          store_chunk<T>(dz + r.head, c0 + k * NT, x);
        }
      c0 += NC * NT;
      if (c0 >= b.c1) break;
      load(c0);
    }
    if (tid < b.edges) Elem<T>::store(dz + r.edge(tid), grad_of(edge, ex, s));
    __syncthreads();
    if (b.c1 > b.c0) fix_listed<T, NT>(L, p, dz, ex, s, r.head + b.c0 * VEC, r.head + b.c1 * VEC);
    if (b.edges) {
      fix_listed<T, NT>(L, p, dz, ex, s, 0, r.head);
      fix_listed<T, NT>(L, p, dz, ex, s, r.head + r.chunks * VEC, n);
    }
    __syncthreads();
  }
}

// total = sum_t w_t L_t in a fixed order, one block.  Ignored rows hold 0.
__global__ __launch_bounds__(1024) void distill_total_kernel(DistillParams p) {
  __shared__ double red[16];
  double s = 0.0;
  const double uni = 1.0 / (double)p.rows;
  for (int64_t t = threadIdx.x; t < p.rows; t += 1024) {
    const double w = p.weights ? (double)p.weights[t] : uni;
    if (w != 0.0) s += w * (double)p.rows_loss[t];
  }
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) s += red[w];
    *p.total = (float)s;
  }
}

// Slabs of a row when there are few long rows (1: one block a row): about two
// blocks a compute unit, slabs of at least 1024 chunks.  Loss with gradient, cut
// and whole rows: 8 x 128000 bf16 18 and 28 us, 32 of them 26 and 29, 64 of them
// 48 and 30 (one block has all the losses); 8 x 128000 fp32 18 and 27, 32 of them
// 29 and 29.  Rows of up to kMiddleRow chunks: 8 x 32000 bf16 18 and 16, 64 of
// them 42 and 17; 8 x 64000 bf16 18 and 18.
int splits_of(int64_t rows, int vocab, int dtype) {
  const int chunks = vocab / (dtype == PMX_F32 ? 4 : 8);
  if (rows > kFewRows || rows == 0 || chunks <= kMiddleRow) return 1;
  return (int)std::min<int64_t>(std::min<int64_t>(512 / rows, chunks / 1024), 64);
}

// Slabs of a row in distill_grad_kernel: enough for about four blocks a compute
// unit in all, of at least 1024 chunks (four a thread).  A block works through
// the row's list before it writes, so more blocks than run at once cost more
// than they gain (1023 rows of 32003 bf16: 4 slabs 29.2 us, 3 26.5 us).
int grad_slabs(const DistillParams& p) {
  const int64_t chunks = p.vocab / (p.dtype == PMX_F32 ? 4 : 8);
  const int64_t want = (4 * (int64_t)p.num_cu + p.rows - 1) / p.rows;
  return (int)std::max<int64_t>(1, std::min(want, (chunks + 1023) / 1024));
}

template <typename T, int EX, bool GRAD>
hipError_t launch_rows(const DistillParams& p, hipStream_t s) {
  constexpr int VEC = Elem<T>::VEC;
  if (p.splits > 1) {
    hipLaunchKernelGGL((distill_part_kernel<T, EX>), dim3(p.splits, (unsigned)p.rows), dim3(256), 0, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int slabs = GRAD ? grad_slabs(p) : 0;
    hipLaunchKernelGGL((distill_grad_kernel<T, EX, true>), dim3(slabs + 1, GRAD ? (unsigned)p.rows : 1), dim3(256), 0,
                       s, p, slabs);
    return hipGetLastError();
  }
  // the smallest block whose registers hold the row's chunks; a row shorter
  // than two chunks may have no whole one and takes the other kernel
  const int64_t chunks = p.vocab / VEC;
#define PMX_ROWS(NT, NC)                                                                          \
  if (chunks >= 2 && chunks <= (int64_t)NT * NC) {                                                               \
    const int64_t g = std::min<int64_t>(p.rows, (int64_t)p.num_cu * waves_for(NC) * 256 / NT);    \
    if (NT == 1024) {                                                                             \
      hipLaunchKernelGGL(distill_claim_kernel, dim3(1), dim3(1), 0, s, p.next_row, (uint32_t)g);  \
      hipError_t e = hipGetLastError();                                                           \
      if (e != hipSuccess) return e;                                                              \
    }                                                                                             \
    hipLaunchKernelGGL((distill_row_kernel<T, NT, NC, EX, GRAD>), dim3((unsigned)g), dim3(NT), 0, s, p); \
    return hipGetLastError();                                                                     \
  }
  PMX_ROWS(256, 2)
  PMX_ROWS(256, 4)
  PMX_ROWS(256, 8)
  PMX_ROWS(256, 16)
  PMX_ROWS(512, 16)
  PMX_ROWS(1024, 16)
#undef PMX_ROWS
  const int64_t g = std::min<int64_t>(p.rows, (int64_t)p.num_cu * 2);
  hipLaunchKernelGGL((distill_long_kernel<T, EX, GRAD>), dim3((unsigned)g), dim3(1024), 0, s, p);
  return hipGetLastError();
}

int exps_of(const DistillParams& p) {
  if (p.mix == 0.f || p.mix == 1.f || p.tau == 1.f) return EXP_ONE;
  return p.tau == 2.f ? EXP_SQ1 : p.tau == 4.f ? EXP_SQ2 : p.tau == 8.f ? EXP_SQ3 : EXP_TWO;
}

template <typename T, bool GRAD>
hipError_t launch_loss_t(const DistillParams& p, hipStream_t s) {
  switch (exps_of(p)) {
    case EXP_ONE: return launch_rows<T, EXP_ONE, GRAD>(p, s);
    case EXP_TWO: return launch_rows<T, EXP_TWO, GRAD>(p, s);
    case EXP_SQ1: return launch_rows<T, EXP_SQ1, GRAD>(p, s);
    case EXP_SQ2: return launch_rows<T, EXP_SQ2, GRAD>(p, s);
    default: return launch_rows<T, EXP_SQ3, GRAD>(p, s);
  }
}

template <typename T>
hipError_t launch_grad_t(const DistillParams& p, hipStream_t s) {
  // in place one block owns the row: it reads the listed logits before it
  // overwrites them
  const int slabs = p.z == p.dz ? 1 : grad_slabs(p);
  const dim3 grid((unsigned)slabs, (unsigned)(p.rows < 65535 ? p.rows : 65535));
#define PMX_GRAD(EX) \
  case EX: hipLaunchKernelGGL((distill_grad_kernel<T, EX, false>), grid, dim3(256), 0, s, p, slabs); break;
  switch (exps_of(p)) {
    PMX_GRAD(EXP_ONE)
    PMX_GRAD(EXP_TWO)
    PMX_GRAD(EXP_SQ1)
    PMX_GRAD(EXP_SQ2)
    PMX_GRAD(EXP_SQ3)
  }
#undef PMX_GRAD
  return hipGetLastError();
}

}  // namespace

int64_t distill_part_floats(int64_t rows, int vocab, int top, int dtype) {
  const int k = splits_of(rows, vocab, dtype);
  if (k > 1) return rows * (k * 3 + top + 1);
  const int chunks = vocab / (dtype == PMX_F32 ? 4 : 8);
  return rows > 0 && chunks > kMiddleRow && chunks <= kLongRow ? 1 : 0;  // next_row
}

hipError_t launch_distill_loss(DistillParams p, hipStream_t s) {
  p.splits = splits_of(p.rows, p.vocab, p.dtype);
  p.next_row = reinterpret_cast<uint32_t*>(p.part);
  hipError_t e = hipSuccess;
  if (p.rows > 0) {  // (no rows: total = 0)
    if (p.dtype == PMX_F32) e = p.dz ? launch_loss_t<float, true>(p, s) : launch_loss_t<float, false>(p, s);
    else e = p.dz ? launch_loss_t<uint16_t, true>(p, s) : launch_loss_t<uint16_t, false>(p, s);
  }
  if (e != hipSuccess || p.splits > 1) return e;  // (with the losses of rows cut over blocks)
  hipLaunchKernelGGL(distill_total_kernel, dim3(1), dim3(1024), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_distill_grad(const DistillParams& p, hipStream_t s) {
  return p.dtype == PMX_F32 ? launch_grad_t<float>(p, s) : launch_grad_t<uint16_t>(p, s);
}

}  // namespace pmx
