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
// up to 1024 threads: 128 Ki bf16 or 64 Ki fp32 logits).  Longer rows are read
// twice (the second time mostly from the last-level cache).  When there are
// few rows, the row is cut over several blocks: one launch for the partial
// sums, one for the gradient.
// exp(z - m) is the tau-th power of exp((z - m) / tau): for tau = 2, 4 or 8 it
// is squared up instead of a second exponential (a quarter-rate instruction).
#include "pmx_train.h"

namespace pmx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;

// exponentials per element: one (a single temperature is in play), two, or
// one and squarings
enum Exps : int { EXP_ONE = 0, EXP_TWO = 1, EXP_SQ = 2 };

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
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

// Elements from the row's start down to the 16-byte boundary below it: chunk
// c of a row holds elements [c VEC - head, (c + 1) VEC - head).
template <typename T>
__device__ __forceinline__ int head_of(const T* row) {
  return (int)(((uintptr_t)row & 15) / sizeof(T));
}

// Chunk with first element e0 of a row of n elements; places outside the row
// hold -inf (no weight in a maximum or a sum).  Whole chunks are one aligned
// 16-byte load; the row's first and last chunk are read by element.
template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const T* row, int e0, int n) {
  constexpr int VEC = Elem<T>::VEC;
  if (e0 >= 0 && e0 + VEC <= n) return *reinterpret_cast<const u32x4_t*>(row + e0);
  float x[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    x[j] = (e0 + j >= 0 && e0 + j < n) ? Elem<T>::load(row + e0 + j) : kNegInf;
  return Elem<T>::pack(x);
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int e0, int n, bool vec, const float (&x)[Elem<T>::VEC]) {
  constexpr int VEC = Elem<T>::VEC;
  if (vec && e0 >= 0 && e0 + VEC <= n) {
    *reinterpret_cast<u32x4_t*>(row + e0) = Elem<T>::pack(x);
    return;
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (e0 + j >= 0 && e0 + j < n) Elem<T>::store(row + e0 + j, x[j]);
}

// Exponentials of one logit: et = exp((z - m) / tau), e1 = exp(z - m).
template <int EX>
struct Expo {
  float m, ct;  // ct = log2(e) / tau (EXP_ONE: of the only temperature)
  int sq;       // EXP_SQ: tau = 2^sq
  __device__ __forceinline__ void operator()(float z, float& et, float& e1) const {
    const float d = z - m;
    et = __builtin_amdgcn_exp2f(d * ct);
    if (EX == EXP_ONE) e1 = et;
    if (EX == EXP_TWO) e1 = __builtin_amdgcn_exp2f(d * kLog2e);
    if (EX == EXP_SQ) {
      e1 = et * et;
      if (sq > 1) e1 *= e1;
      if (sq > 2) e1 *= e1;
    }
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
    float m = red[i][0];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, red[i][w]);
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
    float m = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) m += red[i][w];
    v[i] = m;
  }
  __syncthreads();
}

// The listed columns of a row: the teacher's entries and, last, the label.
// Entries outside the vocabulary have id -1.
struct Listed {
  int id[PMX_MAX_TOP + 1];
  float e[PMX_MAX_TOP + 1];  // teacher logit / tau, then exp(... - max)
  float z[PMX_MAX_TOP + 1];  // the student's logit there
};

template <typename T, int NT>
__device__ __forceinline__ void load_listed(Listed& L, const DistillParams& p, int64_t t,
                                            const T* z, float& amax) {
  const float rt = 1.f / p.tau;
  amax = kNegInf;
  const int n = p.top + 1;
  for (int i = threadIdx.x; i < n; i += NT) {
    int64_t id = -1;
    float a = kNegInf;
    if (i < p.top) {
      id = load_index(p.ids, t * p.ld_ids + i, p.ids64);
      if (id < 0 || id >= p.vocab) id = -1;
      if (id >= 0) {
        const int64_t o = t * p.ld_teacher + i;
        a = rt * (p.teacher_dtype == PMX_F32
                      ? reinterpret_cast<const float*>(p.teacher)[o]
                      : Elem<uint16_t>::load(reinterpret_cast<const uint16_t*>(p.teacher) + o));
      }
    } else if (p.labels) {
      id = load_index(p.labels, t, p.labels64);
      if (id < 0 || id >= p.vocab) id = -1;
    }
    L.id[i] = (int)id;
    L.e[i] = a;
    L.z[i] = id >= 0 ? Elem<T>::load(z + id) : 0.f;
    amax = fmaxf(amax, a);
  }
}

// Row results: the scale of each exponential in the gradient and the loss.
struct RowOut {
  float m, inv_t, inv_1;  // maximum, 1 / S_tau, 1 / S_1 (0: no logit above -inf)
  float a_inv;            // 1 / A (0: no teacher entry)
  float loss;
};

// sums: A, sum e (a - amax), sum e (z - m) / tau, S_tau, S_1
__device__ __forceinline__ RowOut finish_row(const DistillParams& p, const Listed& L, float m,
                                             const float (&v)[5]) {
  RowOut r;
  r.m = m;
  r.inv_t = v[3] != 0.f ? 1.f / v[3] : 0.f;
  r.inv_1 = v[4] != 0.f ? 1.f / v[4] : 0.f;
  r.a_inv = v[0] != 0.f ? 1.f / v[0] : 0.f;
  r.loss = 0.f;
  if (v[3] != 0.f) {
    if (p.mix != 0.f && v[0] != 0.f)
      r.loss += p.mix * p.tau * p.tau * ((v[1] - v[2]) * r.a_inv - logf(v[0]) + logf(v[3]));
    if (p.mix != 1.f && L.id[p.top] >= 0)
      r.loss += (1.f - p.mix) * (logf(v[4]) - (L.z[p.top] - m));
  }
  return r;
}

// Corrections of the gradient at the listed columns, over dense values already
// written by this block.  Every entry naming the same column writes the same
// value.
template <typename T, int NT, int EX>
__device__ __forceinline__ void fix_listed(const Listed& L, const DistillParams& p, T* dz,
                                           const Expo<EX>& ex, float gt, float g1, float gp,
                                           float gc, int lo, int hi) {
  for (int i = threadIdx.x; i <= p.top; i += NT) {
    const int id = L.id[i];
    if (id < 0 || id < lo || id >= hi) continue;  // lo may lie before the row's start
    float ps = 0.f;
    for (int j = 0; j < p.top; ++j) ps += L.id[j] == id ? L.e[j] : 0.f;
    float et, e1;
    ex(L.z[i], et, e1);
    float v = gt * et + (EX == EXP_ONE ? 0.f : g1 * e1) - gp * ps;
    if (L.id[p.top] == id) v -= gc;
    Elem<T>::store(dz + id, v);
  }
}

// Gradient scales: gt and g1 multiply the exponentials (one temperature: gt
// alone carries both), gp the teacher's e_i, gc the label's one.
struct Scales {
  float gt, g1, gp, gc;
};
template <int EX>
__device__ __forceinline__ Scales grad_scales(const DistillParams& p, float w, float inv_t,
                                              float inv_1, float a_inv, bool label) {
  const bool row = inv_t != 0.f;  // a row of nothing but -inf has no gradient
  const float kd = row && a_inv != 0.f && p.mix != 0.f ? w * p.mix * p.tau : 0.f;
  const float ce = row && label && p.mix != 1.f ? w * (1.f - p.mix) : 0.f;
  Scales s;
  s.gt = kd * inv_t;
  s.g1 = ce * inv_1;
  if (EX == EXP_ONE) s.gt += s.g1;
  s.gp = kd * a_inv;
  s.gc = ce;
  return s;
}

template <int EX>
__device__ __forceinline__ Expo<EX> make_expo(const DistillParams& p, float m) {
  Expo<EX> ex;
  ex.m = m;
  // the only temperature of EXP_ONE: tau, or 1 where only the label counts
  ex.ct = kLog2e / (EX == EXP_ONE && p.mix == 0.f ? 1.f : p.tau);
  ex.sq = p.tau == 2.f ? 1 : p.tau == 4.f ? 2 : 3;
  return ex;
}

// One block a row; NC > 0: the row in registers, NC chunks a thread; NC = 0:
// the row is read twice.  GRAD: dz is written.
template <typename T, int NT, int NC, int EX, bool GRAD>
__global__ __launch_bounds__(NT) void distill_row_kernel(DistillParams p) {
  constexpr int VEC = Elem<T>::VEC;
  __shared__ Listed L;
  __shared__ float red[5][16];
  const int64_t t = blockIdx.x;
  const T* z = reinterpret_cast<const T*>(p.z) + t * p.ldz;
  T* dz = GRAD ? reinterpret_cast<T*>(p.dz) + t * p.lddz : nullptr;
  const int n = p.vocab, head = head_of(z);
  const bool vec = GRAD && head_of(dz) == head;
  const float wt = p.weights ? p.weights[t] : 1.f / (float)p.rows;
  if (wt == 0.f) {  // an ignored row: its logits are not read
    if (threadIdx.x == 0) {
      p.rows_loss[t] = 0.f;
      if (p.stats) p.stats[3 * t] = p.stats[3 * t + 1] = p.stats[3 * t + 2] = 0.f;
    }
    if (GRAD) {
      const float zero[VEC] = {};
      const int hd = head_of(dz);
      for (int c = threadIdx.x; c * VEC - hd < n; c += NT) store_chunk<T>(dz, c * VEC - hd, n, true, zero);
    }
    return;
  }
  u32x4_t v[NC > 0 ? NC : 1];
  float mx[2];
  mx[0] = kNegInf;
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c) v[c] = load_chunk<T>(z, (c * NT + (int)threadIdx.x) * VEC - head, n);
  }
  load_listed<T, NT>(L, p, t, z, mx[1]);
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) mx[0] = fmaxf(mx[0], Elem<T>::get(v[c], j));
  } else {
    for (int c = threadIdx.x; c * VEC - head < n; c += NT) {
      const u32x4_t u = load_chunk<T>(z, c * VEC - head, n);
#pragma unroll
      for (int j = 0; j < VEC; ++j) mx[0] = fmaxf(mx[0], Elem<T>::get(u, j));
    }
  }
  block_max<NT>(mx, red);
  const float m = mx[0] == kNegInf ? 0.f : mx[0];  // -inf - m stays -inf
  const float am = mx[1] == kNegInf ? 0.f : mx[1];
  const Expo<EX> ex = make_expo<EX>(p, m);
  float sum[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
  const float rt = 1.f / p.tau;
  for (int i = threadIdx.x; i < p.top; i += NT) {
    const float a = L.e[i] - am;
    const float e = __builtin_amdgcn_exp2f(a * kLog2e);
    L.e[i] = e;
    sum[0] += e;
    if (e != 0.f) {  // nothing (not NaN) where the teacher gives no weight
      sum[1] += e * a;
      sum[2] += e * (L.z[i] - m) * rt;
    }
  }
  if constexpr (NC > 0) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float et, e1;
        ex(Elem<T>::get(v[c], j), et, e1);
        sum[3] += et;
        if (EX != EXP_ONE) sum[4] += e1;
      }
  } else {
    for (int c = threadIdx.x; c * VEC - head < n; c += NT) {
      const u32x4_t u = load_chunk<T>(z, c * VEC - head, n);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float et, e1;
        ex(Elem<T>::get(u, j), et, e1);
        sum[3] += et;
        if (EX != EXP_ONE) sum[4] += e1;
      }
    }
  }
  if (EX == EXP_ONE) sum[4] = sum[3];
  block_sum<NT>(sum, red);
  const RowOut r = finish_row(p, L, m, sum);
  if (threadIdx.x == 0) {
    p.rows_loss[t] = r.loss;
    if (p.stats) {
      p.stats[3 * t] = r.m;
      p.stats[3 * t + 1] = r.inv_t;
      p.stats[3 * t + 2] = r.inv_1;
    }
  }
  if constexpr (GRAD) {
    const float w = wt * (p.upstream ? *p.upstream : 1.f);
    const Scales s = grad_scales<EX>(p, w, r.inv_t, r.inv_1, r.a_inv, L.id[p.top] >= 0);
    auto emit = [&](const u32x4_t& u, int e0) {
      float x[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float et, e1;
        ex(Elem<T>::get(u, j), et, e1);
        x[j] = s.gt * et + (EX == EXP_ONE ? 0.f : s.g1 * e1);
      }
      store_chunk<T>(dz, e0, n, vec, x);
    };
    if constexpr (NC > 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e0 = (c * NT + (int)threadIdx.x) * VEC - head;
        if (e0 < n) emit(v[c], e0);
      }
    } else {
      for (int c = threadIdx.x; c * VEC - head < n; c += NT)
        emit(load_chunk<T>(z, c * VEC - head, n), c * VEC - head);
    }
    __syncthreads();
    fix_listed<T, NT, EX>(L, p, dz, ex, s.gt, s.g1, s.gp, s.gc, 0, n);
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

// Gradient from the saved statistics: blockIdx.x cuts the row into gridDim.x
// slabs of whole chunks, blockIdx.y (and a stride) walks the rows.
template <typename T, int EX>
__global__ __launch_bounds__(256) void distill_grad_kernel(DistillParams p) {
  constexpr int VEC = Elem<T>::VEC, NT = 256;
  __shared__ Listed L;
  __shared__ float red[1][16];
  const int n = p.vocab;
  for (int64_t t = blockIdx.y; t < p.rows; t += gridDim.y) {
    const T* z = reinterpret_cast<const T*>(p.z) + t * p.ldz;
    T* dz = reinterpret_cast<T*>(p.dz) + t * p.lddz;
    const int head = head_of(z);
    const bool vec = head_of(dz) == head;
    const int chunks = (n + head + VEC - 1) / VEC;
    const int per = (chunks + (int)gridDim.x - 1) / (int)gridDim.x;
    const int c0 = (int)blockIdx.x * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    const float wt = p.weights ? p.weights[t] : 1.f / (float)p.rows;
    const float m = p.stats[3 * t], inv_t = p.stats[3 * t + 1], inv_1 = p.stats[3 * t + 2];
    if (wt == 0.f) {
      const float zero[VEC] = {};
      for (int c = c0 + threadIdx.x; c < c1; c += NT) store_chunk<T>(dz, c * VEC - head, n, vec, zero);
      continue;
    }
    // in place (dz = z) a later block may have overwritten a listed logit, so
    // the corrected columns are handled where their own slab is written: the
    // value at hand is the slab's own
    float am[1];
    load_listed<T, NT>(L, p, t, z, am[0]);
    block_max<NT>(am, red);
    const float amx = am[0] == kNegInf ? 0.f : am[0];
    float sum[1] = {0.f};
    for (int i = threadIdx.x; i < p.top; i += NT) {
      const float e = __builtin_amdgcn_exp2f((L.e[i] - amx) * kLog2e);
      L.e[i] = e;
      sum[0] += e;
    }
    block_sum<NT>(sum, red);
    const float a_inv = sum[0] != 0.f ? 1.f / sum[0] : 0.f;
    const float w = wt * (p.upstream ? *p.upstream : 1.f);
    const Expo<EX> ex = make_expo<EX>(p, m);
    const Scales s = grad_scales<EX>(p, w, inv_t, inv_1, a_inv, L.id[p.top] >= 0);
    for (int c = c0 + threadIdx.x; c < c1; c += NT) {
      const u32x4_t u = load_chunk<T>(z, c * VEC - head, n);
      float x[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float et, e1;
        ex(Elem<T>::get(u, j), et, e1);
        x[j] = s.gt * et + (EX == EXP_ONE ? 0.f : s.g1 * e1);
      }
      store_chunk<T>(dz, c * VEC - head, n, vec, x);
    }
    __syncthreads();
    fix_listed<T, NT, EX>(L, p, dz, ex, s.gt, s.g1, s.gp, s.gc, c0 * VEC - head, c1 * VEC - head);
    __syncthreads();
  }
}

template <typename T, int EX, bool GRAD>
hipError_t launch_rows(const DistillParams& p, hipStream_t s) {
  constexpr int VEC = Elem<T>::VEC;
  const dim3 grid((unsigned)p.rows);
  // the smallest block whose registers hold the row (VEC more for its head)
  const int64_t need = (int64_t)p.vocab + VEC;
#define PMX_ROWS(NT, NC)                                                                        \
  if (need <= (int64_t)NT * NC * VEC) {                                                         \
    hipLaunchKernelGGL((distill_row_kernel<T, NT, NC, EX, GRAD>), grid, dim3(NT), 0, s, p);     \
    return hipGetLastError();                                                                   \
  }
  PMX_ROWS(256, 2)
  PMX_ROWS(256, 4)
  PMX_ROWS(256, 8)
  PMX_ROWS(256, 16)
  PMX_ROWS(512, 16)
  PMX_ROWS(1024, 16)
#undef PMX_ROWS
  hipLaunchKernelGGL((distill_row_kernel<T, 1024, 0, EX, GRAD>), grid, dim3(1024), 0, s, p);
  return hipGetLastError();
}

int exps_of(const DistillParams& p) {
  if (p.mix == 0.f || p.mix == 1.f || p.tau == 1.f) return EXP_ONE;
  if (p.tau == 2.f || p.tau == 4.f || p.tau == 8.f) return EXP_SQ;
  return EXP_TWO;
}

template <typename T, bool GRAD>
hipError_t launch_loss_t(const DistillParams& p, hipStream_t s) {
  switch (exps_of(p)) {
    case EXP_ONE: return launch_rows<T, EXP_ONE, GRAD>(p, s);
    case EXP_TWO: return launch_rows<T, EXP_TWO, GRAD>(p, s);
    default: return launch_rows<T, EXP_SQ, GRAD>(p, s);
  }
}

template <typename T>
hipError_t launch_grad_t(const DistillParams& p, hipStream_t s) {
  // four chunks a thread and more, and blocks enough to fill the card
  const int chunks = (p.vocab + Elem<T>::VEC - 1) / Elem<T>::VEC + 1;
  int slabs = chunks / 1024;
  if (slabs < 1) slabs = 1;
  if (p.z == p.dz) slabs = 1;  // in place: one block owns the row
  const dim3 grid((unsigned)slabs, (unsigned)(p.rows < 65535 ? p.rows : 65535));
  switch (exps_of(p)) {
    case EXP_ONE: hipLaunchKernelGGL((distill_grad_kernel<T, EXP_ONE>), grid, dim3(256), 0, s, p); break;
    case EXP_TWO: hipLaunchKernelGGL((distill_grad_kernel<T, EXP_TWO>), grid, dim3(256), 0, s, p); break;
    default: hipLaunchKernelGGL((distill_grad_kernel<T, EXP_SQ>), grid, dim3(256), 0, s, p); break;
  }
  return hipGetLastError();
}

}  // namespace

int64_t distill_part_floats(int64_t, int, int) { return 0; }

hipError_t launch_distill_loss(const DistillParams& p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.rows == 0) ;  // total = 0
  else if (p.dtype == PMX_F32) e = p.dz ? launch_loss_t<float, true>(p, s) : launch_loss_t<float, false>(p, s);
  else e = p.dz ? launch_loss_t<uint16_t, true>(p, s) : launch_loss_t<uint16_t, false>(p, s);
  if (e != hipSuccess || !p.total) return e;
  hipLaunchKernelGGL(distill_total_kernel, dim3(1), dim3(1024), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_distill_grad(const DistillParams& p, hipStream_t s) {
  return p.dtype == PMX_F32 ? launch_grad_t<float>(p, s) : launch_grad_t<uint16_t>(p, s);
}

}  // namespace pmx
