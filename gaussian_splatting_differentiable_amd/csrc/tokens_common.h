// Internal types and device helpers shared by the token operators (norm and
// rotation of queries and keys, attention, dropout). gfx950 only, wave64.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gs.h"

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

template <class E, int N>
using vec = E __attribute__((ext_vector_type(N)));

typedef vec<float, 4> f32x4;
typedef vec<float, 16> f32x16;
typedef vec<int, 4> i32x4;
typedef vec<short, 4> i16x4;

// A [batch][token][head][dim] tensor as the kernels see it: element strides,
// dim contiguous.
struct TokK {
  void *data;
  int64_t bs, ts, hs;
};

template <class E>
__device__ __forceinline__ E *tok_row(const TokK &t, int64_t b, int64_t token, int64_t head) {
  return (E *)t.data + b * t.bs + token * t.ts + head * t.hs;
}

// Four consecutive elements to and from float registers (8 or 16 bytes).
template <class E>
__device__ __forceinline__ f32x4 load4(const E *p) {
  const vec<E, 4> v = *(const vec<E, 4> *)p;
  f32x4 r;
#pragma unroll
  for (int i = 0; i < 4; i++) r[i] = (float)v[i];
  return r;
}

template <class E>
__device__ __forceinline__ void store4(E *p, f32x4 x) {
  vec<E, 4> v;
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = (E)x[i];  // to nearest even
  *(vec<E, 4> *)p = v;
}

// Sum over aligned groups of n lanes (n a power of two up to 64), in every lane.
__device__ __forceinline__ float group_sum(float x, int n) {
  for (int m = 1; m < n; m <<= 1) x += __shfl_xor(x, m);
  return x;
}

// ------------------------------------------------------------------ kernel arguments

struct QkK {
  int batch, tokens, q_heads, k_heads, dim, rot, neighbours, n_positions;
  int lanes;  // lanes per row: the power of two from dim / 8 up
  float eps;
  int64_t pos_stride;
  const float *qw, *kw, *cos_sin;
  const int32_t *positions;
  TokK q, k;    // forward: inputs; backward: the forward's inputs
  TokK qg, kg;  // backward: gradients of the outputs
  TokK qo, ko;  // forward: outputs; backward: gradients of the inputs
  float *partial;  // backward: [2][blocks][dim] sums of the weight gradients
  float *dqw, *dkw;
  int blocks;
};

struct DropK {
  int64_t rows, cols;
  const void *x, *res;
  void *y;
  int64_t x_stride, res_stride, y_stride;
  uint64_t seed, offset;
  uint32_t drop_below;  // drop where the random word is below this
  float scale;
  int per_row;
};

struct AttnK {
  int batch, q_heads, kv_heads, share, q_len, kv_len, dim, causal;
  float scale, scale_log2;  // scale and scale * log2(e)
  const int2 *spans;
  int64_t span_stride;
  TokK q, k, v, o;
  float *lse;
  int passes;  // 2: blocks of rows are launched twice (attention_common.h: apart)
  // the split form
  int splits, split_keys;
  float *part_o, *part_ml;
  // backward
  TokK d_o, dq, dk, dv;
  int q_pad;  // queries, rounded up to whole tiles of 64
  float *row_lse, *row_delta;  // [batch][q_heads][q_pad]: -lse / scale (fp16: less 15 bits), -D_i
  int2 *row_spans;             // [batch][q_pad]: spans as the masks leave them
  int4 *tile_spans;
  int q_parts, kv_parts;
  float *part_q, *part_k, *part_v;
};
