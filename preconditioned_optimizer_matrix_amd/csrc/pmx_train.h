// Parameter blocks and launchers of the training-step operators: products
// grouped by expert (pmx_grouped.hip), the token embedding and its gradient
// (pmx_embed.hip), the distillation loss (pmx_distill.hip).
#pragma once

#include "pmx_internal.h"

namespace pmx {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Index arrays are int32 or int64 (pmx_itype).
__device__ __forceinline__ int64_t load_index(const void* p, int64_t i, int is64) {
  return is64 ? reinterpret_cast<const int64_t*>(p)[i]
              : (int64_t) reinterpret_cast<const int32_t*>(p)[i];
}

// Two floats to packed bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// ---------------------------------------------------------------------------
// Distillation loss.  Per row t, over the listed teacher entries i whose id is
// inside the vocabulary:
//   p = softmax(teacher / tau), q = softmax(z / tau), s = softmax(z)
//   L = mix tau^2 sum_i p_i (log p_i - log q_{id_i}) - (1 - mix) log s_label
//   dz_j = up w [mix tau (q_j - sum_{i: id_i = j} p_i) + (1 - mix)(s_j - [j = label])]
struct DistillParams {
  const void* z;
  int64_t ldz;
  void* dz;
  int64_t lddz;
  const void* ids;
  int64_t ld_ids;
  const void* teacher;
  int64_t ld_teacher;
  const void* labels;
  const float* weights;  // null: 1 / rows each
  const float* upstream; // null: 1
  float* rows_loss;
  float* total;
  float* stats;          // [rows][3]: max, 1 / sum exp((z - max) / tau), 1 / sum exp(z - max)
  float* part;           // rows cut over blocks: [rows][splits][3], then [rows][top + 1]
  int splits;
  uint32_t* next_row;    // rows taken by blocks as they go (same memory as part)
  int64_t rows;
  int vocab, top;
  int dtype, teacher_dtype;
  int ids64, labels64;
  float tau, mix;
  int num_cu;
};

// Floats of workspace: partial sums of rows cut over blocks, or the counter of
// claimed rows.
int64_t distill_part_floats(int64_t rows, int vocab, int top, int dtype);
hipError_t launch_distill_loss(DistillParams p, hipStream_t s);
hipError_t launch_distill_grad(const DistillParams& p, hipStream_t s);

// ---------------------------------------------------------------------------
// Embedding.
struct EmbedParams {
  const void* table;   // lookup: vocab x dim
  int64_t ld_table;
  const void* ids;
  int ids64;
  int64_t tokens;
  int vocab, dim;
  float scale;
  int dtype, out_dtype;
  void* out;           // lookup: tokens x dim; gradient: vocab x dim
  int64_t ld_out;
  // gradient
  const void* dy;      // tokens x dim
  int64_t ld_dy;
  int64_t padding_idx;
  int accumulate;
  void* ws;
};
size_t embed_grad_workspace(int64_t tokens, int vocab, int dim);
hipError_t launch_embed_lookup(const EmbedParams& p, hipStream_t s);
hipError_t launch_embed_grad(const EmbedParams& p, hipStream_t s);

// ---------------------------------------------------------------------------
// Products grouped by expert.
struct GroupedParams {
  const void* a;       // product: rows x k; outer: rows x m
  int64_t lda;
  const void* b;       // product: per group k x n (trans_b: n x k); outer: rows x n
  int64_t ldb, stride_b;
  void* c;             // product: rows x n; outer: per group m x n
  int64_t ldc, stride_c;
  const void* offsets; // groups + 1 row offsets (device)
  int off64;
  int groups;
  int64_t rows;
  int m, n, k;         // product: k, n (m unused); outer: m, n (k unused)
  int trans_b;
  int accumulate;      // outer: add to C
  int dtype, out_dtype;
  float* part;         // split contraction: partial results
  int splits;
  int num_cu;
  int round;           // quarters: blocks of the large tiles' launch
};
// Splits of the contraction (1: none) and the floats of workspace they need.
int grouped_product_splits(int64_t rows, int k, int n, int groups, int dtype);
int grouped_outer_splits(int64_t rows, int m, int n, int groups, int dtype);
hipError_t launch_grouped_product(const GroupedParams& p, hipStream_t s);
hipError_t launch_grouped_outer(const GroupedParams& p, hipStream_t s);

}  // namespace pmx
