// The norm of queries and keys for each head with the position rotation in the
// same pass, and its gradient.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps), z = x r w, y = R z: R turns the pairs of
//   the first `rot` elements by the angles of the row's position and leaves the
//   rest.
//   Backward: g = R^T dy, dw = sum over rows of g x r, h = g w,
//   dx = r (h - x r mean_d(h x r)).
//
// A row (batch, token, head) is held by dim / 8 lanes, four pairs in each, so a
// turn needs no exchange between lanes: a lane of the rotated part takes
// elements 4j.. and rot/2 + 4j.. (pairs of halves), any other lane the elements
// 8j.. (neighbours, and the part that is not rotated). Groups of lanes take four
// heads of one token at a time and read its angles and the weights once for
// them: the angles in 32 bits are twice a 16-bit row's bytes.
//
// Bound: HBM (each input read once, each output written once). 2 x 32768 tokens, 16 + 4
// heads of 128, bf16: 149 us for 671 MB in calls one after the other, 4.5 TB/s (a copy
// reaches 4.7). 3 x 5461 tokens, 12 + 12 heads of 64: forward 24 us (101 MB), backward 33
// (151 MB) and the weights' partial sums 4.
#include "tokens_common.h"

namespace {

constexpr int HC = 4;  // heads of one token that a group of lanes takes together

// Where a lane's two chunks of four elements are, and whether they hold pairs
// of halves (a[i], b[i]) or neighbours.
struct Lane {
  int j, e0, e1;
  bool on, split, turns;
};

__device__ __forceinline__ Lane lane_of(const QkK &p, int lane) {
  Lane l;
  l.j = lane & (p.lanes - 1);
  l.on = 8 * l.j < p.dim;
  l.turns = 8 * l.j < p.rot;
  l.split = l.turns && !p.neighbours;
  l.e0 = l.split ? 4 * l.j : 8 * l.j;
  l.e1 = l.split ? p.rot / 2 + 4 * l.j : 8 * l.j + 4;
  return l;
}

struct Angles {
  f32x4 c, s;
};

// The cosines and sines of a lane's pairs. A position outside the table gives
// NaN (a read is never made there), so that the mistake shows in the result.
__device__ __forceinline__ Angles angles_of(const QkK &p, const Lane &l, int64_t b, int token) {
  Angles a;
  a.c = 1.0f;
  a.s = 0.0f;
  if (l.turns) {
    const int at = p.positions ? p.positions[b * p.pos_stride + token] : token;
    if (at >= 0 && at < p.n_positions) {
      const float *row = p.cos_sin + (int64_t)at * p.rot + 4 * l.j;
      a.c = *(const f32x4 *)row;
      a.s = *(const f32x4 *)(row + p.rot / 2);
    } else {
      a.c = a.s = __builtin_nanf("");
    }
  }
  return a;
}

// The lane's four pairs turned by +angle (forward) or -angle (backward).
template <bool BACK>
__device__ __forceinline__ void turn(const Lane &l, const Angles &t, f32x4 &a, f32x4 &b) {
  f32x4 lo, hi;
  lo[0] = a[0];
  hi[3] = b[3];
  lo[1] = l.split ? a[1] : a[2];
  lo[2] = l.split ? a[2] : b[0];
  lo[3] = l.split ? a[3] : b[2];
  hi[0] = l.split ? b[0] : a[1];
  hi[1] = l.split ? b[1] : a[3];
  hi[2] = l.split ? b[2] : b[1];
  f32x4 x, y;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float s = BACK ? -t.s[i] : t.s[i];
    x[i] = lo[i] * t.c[i] - hi[i] * s;
    y[i] = lo[i] * s + hi[i] * t.c[i];
  }
  a[0] = x[0];
  b[3] = y[3];
  a[1] = l.split ? x[1] : y[0];
  a[2] = l.split ? x[2] : x[1];
  a[3] = l.split ? x[3] : y[1];
  b[0] = l.split ? y[0] : x[2];
  b[1] = l.split ? y[1] : y[2];
  b[2] = l.split ? y[2] : x[3];
}

__device__ __forceinline__ float sum8(f32x4 a, f32x4 b) {
  return ((a[0] + a[1]) + (a[2] + a[3])) + ((b[0] + b[1]) + (b[2] + b[3]));
}

template <class E>
__global__ __launch_bounds__(256) void k_qk_fwd(QkK p, unsigned items) {
  const Lane l = lane_of(p, threadIdx.x);
  const unsigned item = (blockIdx.x * 256u + threadIdx.x) / (unsigned)p.lanes;
  if (item >= items) return;  // whole groups of lanes leave together
  const int qc = (p.q_heads + HC - 1) / HC, kc = (p.k_heads + HC - 1) / HC;
  const unsigned bt = item / (unsigned)(qc + kc);
  const int chunk = (int)(item - bt * (qc + kc));
  const int64_t b = bt / (unsigned)p.tokens;
  const int token = (int)(bt - (unsigned)b * p.tokens);
  const bool key = chunk >= qc;
  const int h0 = (key ? chunk - qc : chunk) * HC, heads = key ? p.k_heads : p.q_heads;
  const TokK in = key ? p.k : p.q, out = key ? p.ko : p.qo;
  const float *w = key ? p.kw : p.qw;
  f32x4 a[HC], c[HC];
#pragma unroll
  for (int h = 0; h < HC; h++) {
    a[h] = c[h] = 0.0f;
    if (l.on && h0 + h < heads) {
      const E *x = tok_row<E>(in, b, token, h0 + h);
      a[h] = load4(x + l.e0);
      c[h] = load4(x + l.e1);
    }
  }
  f32x4 w0 = 1.0f, w1 = 1.0f;
  if (w && l.on) {
    w0 = *(const f32x4 *)(w + l.e0);
    w1 = *(const f32x4 *)(w + l.e1);
  }
  const Angles t = angles_of(p, l, b, token);
#pragma unroll
  for (int h = 0; h < HC; h++) {
    const float ms = group_sum(sum8(a[h] * a[h], c[h] * c[h]), p.lanes) / (float)p.dim;
    const float r = 1.0f / sqrtf(ms + p.eps);
    f32x4 x = a[h] * r * w0, y = c[h] * r * w1;
    turn<false>(l, t, x, y);
    if (l.on && h0 + h < heads) {
      E *o = tok_row<E>(out, b, token, h0 + h);
      store4(o + l.e0, x);
      store4(o + l.e1, y);
    }
  }
}

// blockIdx.y: 0 the queries, 1 the keys. A block strides over its side's items
// and keeps the weight gradient's sums of its lanes, which it adds in a fixed
// order at its end (no atomics: results do not depend on timing).
template <class E>
__global__ __launch_bounds__(256) void k_qk_bwd(QkK p) {
  __shared__ float sums[256 * 9];
  const Lane l = lane_of(p, threadIdx.x);
  const bool key = blockIdx.y != 0;
  const int heads = key ? p.k_heads : p.q_heads, chunks = (heads + HC - 1) / HC;
  const TokK in = key ? p.k : p.q, dy = key ? p.kg : p.qg, dx = key ? p.ko : p.qo;
  const float *w = key ? p.kw : p.qw;
  const int64_t items = (int64_t)p.batch * p.tokens * chunks;
  const int groups = 256 / p.lanes;
  f32x4 w0 = 1.0f, w1 = 1.0f, s0 = 0.0f, s1 = 0.0f;
  if (w && l.on) {
    w0 = *(const f32x4 *)(w + l.e0);
    w1 = *(const f32x4 *)(w + l.e1);
  }
  for (int64_t item = (int64_t)blockIdx.x * groups + threadIdx.x / p.lanes; item < items;
       item += (int64_t)gridDim.x * groups) {
    const unsigned bt = (unsigned)item / (unsigned)chunks;  // (items are below 2^32)
    const int h0 = (int)((unsigned)item - bt * chunks) * HC;
    const int64_t b = bt / (unsigned)p.tokens;
    const int token = (int)(bt - (unsigned)b * p.tokens);
    f32x4 a[HC], c[HC], g0[HC], g1[HC];
#pragma unroll
    for (int h = 0; h < HC; h++) {
      a[h] = c[h] = g0[h] = g1[h] = 0.0f;
      if (l.on && h0 + h < heads) {
        const E *x = tok_row<E>(in, b, token, h0 + h), *g = tok_row<E>(dy, b, token, h0 + h);
        a[h] = load4(x + l.e0);
        c[h] = load4(x + l.e1);
        g0[h] = load4(g + l.e0);
        g1[h] = load4(g + l.e1);
      }
    }
    const Angles t = angles_of(p, l, b, token);
#pragma unroll
    for (int h = 0; h < HC; h++) {
      if (h0 + h >= heads) continue;  // the same for the whole group of lanes
      const float ms = group_sum(sum8(a[h] * a[h], c[h] * c[h]), p.lanes) / (float)p.dim;
      const float r = 1.0f / sqrtf(ms + p.eps);
      f32x4 u = g0[h], v = g1[h];
      turn<true>(l, t, u, v);
      const f32x4 xa = a[h] * r, xb = c[h] * r;
      s0 += u * xa;
      s1 += v * xb;
      u *= w0;
      v *= w1;
      const float m = group_sum(sum8(u * xa, v * xb), p.lanes) / (float)p.dim;
      if (l.on) {
        E *o = tok_row<E>(dx, b, token, h0 + h);
        store4(o + l.e0, r * (u - xa * m));
        store4(o + l.e1, r * (v - xb * m));
      }
    }
  }
  if (!(key ? p.dkw : p.dqw)) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    sums[threadIdx.x * 9 + i] = s0[i];
    sums[threadIdx.x * 9 + 4 + i] = s1[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * p.lanes; i += 256) {
    const int j = i >> 3, e = i & 7;
    const Lane m = lane_of(p, j);
    if (!m.on) continue;
    float s = 0.0f;
    for (int g = 0; g < groups; g++) s += sums[(g * p.lanes + j) * 9 + e];
    const int at = e < 4 ? m.e0 + e : m.e1 + e - 4;
    p.partial[((int64_t)blockIdx.y * p.blocks + blockIdx.x) * p.dim + at] = s;
  }
}

// The weight gradients: 16 columns a block, their partial sums added by 64 threads
// each in a fixed order.
__global__ __launch_bounds__(1024) void k_qk_weights(QkK p) {
  __shared__ float sums[64][17];
  const int c = threadIdx.x & 15, col = blockIdx.x * 16 + c, part = threadIdx.x >> 4;
  float *out = blockIdx.y ? p.dkw : p.dqw;
  if (!out) return;
  const float *in = p.partial + (int64_t)blockIdx.y * p.blocks * p.dim;
  float s = 0.0f;
  if (col < p.dim)
#pragma unroll 4
    for (int i = part; i < p.blocks; i += 64) s += in[(int64_t)i * p.dim + col];
  sums[part][c] = s;
  __syncthreads();
  if (part < 8) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) s += sums[part * 8 + i][c];
    sums[part * 8][c] = s;  // read by this thread alone until here
  }
  __syncthreads();
  if (part == 0 && col < p.dim) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) s += sums[i * 8][c];
    out[col] = s;
  }
}

template <class E>
void launch_fwd(const QkK &p, hipStream_t st) {
  const int chunks = (p.q_heads + HC - 1) / HC + (p.k_heads + HC - 1) / HC;
  const int64_t items = (int64_t)p.batch * p.tokens * chunks;
  const int64_t blocks = (items * p.lanes + 255) / 256;
  k_qk_fwd<E><<<(unsigned)blocks, 256, 0, st>>>(p, (unsigned)items);
}

}  // namespace

// Blocks of the backward, each with its row of partial sums: enough to fill 256
// compute units, and no more than there are items.
int gs_qk_bwd_blocks(int64_t batch, int64_t tokens, int q_heads, int k_heads, int lanes) {
  const int heads = q_heads > k_heads ? q_heads : k_heads;
  const int64_t groups = batch * tokens * ((heads + HC - 1) / HC);
  const int64_t blocks = (groups * lanes + 255) / 256;
  return (int)(blocks < 512 ? blocks : 512);
}

hipError_t gs_launch_qk_fwd(const QkK &p, int dtype, hipStream_t st) {
  if (dtype == GS_F32) launch_fwd<float>(p, st);
  else if (dtype == GS_BF16) launch_fwd<bf16_t>(p, st);
  else launch_fwd<f16_t>(p, st);
  return hipGetLastError();
}

hipError_t gs_launch_qk_bwd(const QkK &p, int dtype, hipStream_t st) {
  const dim3 grid(p.blocks, p.k_heads || p.dkw ? 2 : 1);
  if (p.blocks) {  // without tokens only the weight gradients are written, as 0
    if (dtype == GS_F32) k_qk_bwd<float><<<grid, 256, 0, st>>>(p);
    else if (dtype == GS_BF16) k_qk_bwd<bf16_t><<<grid, 256, 0, st>>>(p);
    else k_qk_bwd<f16_t><<<grid, 256, 0, st>>>(p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !(p.dqw || p.dkw)) return e;
  k_qk_weights<<<dim3((p.dim + 15) / 16, 2), 1024, 0, st>>>(p);
  return hipGetLastError();
}
