// The gradient of attention, with the probabilities computed again from the
// row sums that the forward left: p_ij = exp(s_ij - lse_i),
//   D_i = do_i . o_i, dv_j = sum_i p_ij do_i, ds_ij = p_ij (do_i . v_j - D_i),
//   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i,
// the sums over i also over the heads that share key j.
//
// Three launches: D (and what the others need to skip tiles), then dK and dV by
// blocks that own keys and stream queries, then dQ by blocks that own queries and
// stream keys. The scores are computed in both (7 products of the size of
// q . k^T instead of 5): in exchange no sum is made by atomics, so results do not
// depend on timing, and nothing of size q_len x kv_len is ever stored.
//
// p and ds are rounded to the inputs' 16-bit type for the products. Probabilities
// of long rows fall below the normal range of fp16 (2^-14), so for fp16 the
// kernels work on p 2^15 and on ds 2^e with e from a bound on |ds|
// (|do_i| |v_j| + |D_i|), powers of two that are taken out of the 32-bit sums.
#include "attention_common.h"

namespace {

constexpr int WALK = 4096;  // streamed query tiles whose masks a block holds at a time

template <class E>
constexpr bool is_half = false;
template <>
constexpr bool is_half<f16_t> = true;

// 2^e with |ds| 2^e < 2^14 for |ds| <= bound.
__device__ __forceinline__ int headroom(float bound) {
  if (!(bound > 0.0f) || bound > 3e38f) return 0;
  return max(-100, min(100, 13 - ilogbf(bound)));
}

// ------------------------------------------------------------ rows done again
// As in the forward: a gradient row that holds a NaN is computed again from its
// own (query, key) pairs alone, since 0 x NaN from masked pairs may have spoilt it.

template <class E>
__device__ void redo_query(const AttnK &p, int b, int head, int t, int lane) {
  const int2 span = row_span(p, b, t);
  const int kvh = head / p.share;
  const int64_t at = ((int64_t)b * p.q_heads + head) * p.q_len + t;
  const E *q = tok_row<E>(p.q, b, t, head), *g = tok_row<E>(p.d_o, b, t, head);
  const float lse = p.lse[at] * ATTN_LOG2E, delta = p.delta[at];
  float a0 = 0.0f, a1 = 0.0f;
  for (int j0 = span.x; j0 < span.y; j0 += 64) {
    const int n = min(64, span.y - j0);
    float ds = 0.0f;
    if (lane < n) {
      const float s = dot_row(q, tok_row<E>(p.k, b, j0 + lane, kvh), p.dim) * p.scale_log2;
      ds = __builtin_amdgcn_exp2f(s - lse) *
           (dot_row(g, tok_row<E>(p.v, b, j0 + lane, kvh), p.dim) - delta);
    }
    for (int j = 0; j < n; j++) {
      const E *k = tok_row<E>(p.k, b, j0 + j, kvh);
      const float w = __shfl(ds, j);
      if (lane < p.dim) a0 = fmaf(w, (float)k[lane], a0);
      if (lane + 64 < p.dim) a1 = fmaf(w, (float)k[lane + 64], a1);
    }
  }
  E *o = tok_row<E>(p.dq, b, t, head);
  if (lane < p.dim) o[lane] = (E)(a0 * p.scale);
  if (lane + 64 < p.dim) o[lane + 64] = (E)(a1 * p.scale);
}

template <class E>
__device__ void redo_key(const AttnK &p, int b, int kvh, int key, int lane) {
  const E *k = tok_row<E>(p.k, b, key, kvh), *v = tok_row<E>(p.v, b, key, kvh);
  float k0 = 0.0f, k1 = 0.0f, v0 = 0.0f, v1 = 0.0f;
  for (int head = kvh * p.share; head < (kvh + 1) * p.share; head++)
    for (int t0 = 0; t0 < p.q_len; t0 += 64) {
      const int t = t0 + lane;
      const int2 span = t < p.q_len ? row_span(p, b, t) : make_int2(0, 0);
      const bool in = key >= span.x && key < span.y;
      uint64_t todo = __builtin_amdgcn_ballot_w64(in);
      if (!todo) continue;
      float w = 0.0f, ds = 0.0f;
      if (in) {
        const int64_t at = ((int64_t)b * p.q_heads + head) * p.q_len + t;
        const float s = dot_row(tok_row<E>(p.q, b, t, head), k, p.dim) * p.scale_log2;
        w = __builtin_amdgcn_exp2f(s - p.lse[at] * ATTN_LOG2E);
        ds = w * (dot_row(tok_row<E>(p.d_o, b, t, head), v, p.dim) - p.delta[at]);
      }
      while (todo) {
        const int j = __builtin_ctzll(todo);
        todo &= todo - 1;
        const E *q = tok_row<E>(p.q, b, t0 + j, head), *g = tok_row<E>(p.d_o, b, t0 + j, head);
        const float wj = __shfl(w, j), sj = __shfl(ds, j);
        if (lane < p.dim) {
          k0 = fmaf(sj, (float)q[lane], k0);
          v0 = fmaf(wj, (float)g[lane], v0);
        }
        if (lane + 64 < p.dim) {
          k1 = fmaf(sj, (float)q[lane + 64], k1);
          v1 = fmaf(wj, (float)g[lane + 64], v1);
        }
      }
    }
  E *dk = tok_row<E>(p.dk, b, key, kvh), *dv = tok_row<E>(p.dv, b, key, kvh);
  if (lane < p.dim) {
    dk[lane] = (E)(k0 * p.scale);
    dv[lane] = (E)v0;
  }
  if (lane + 64 < p.dim) {
    dk[lane + 64] = (E)(k1 * p.scale);
    dv[lane + 64] = (E)v1;
  }
}

// ------------------------------------------------------------ preparation
// D_i; for each 64 queries the keys that some row sees and that all see (lo, hi,
// in_lo, in_hi); for fp16 the largest |do_i| and |D_i| of each 64 queries and the
// largest |v_j| of each 64 keys. 16 lanes a row.
template <class E>
__global__ __launch_bounds__(256) void k_attn_prep(AttnK p, int q_tiles, int kv_tiles) {
  __shared__ float top[4][2];
  const int tid = threadIdx.x, lane = tid & 63, j = tid & 15;
  const int q_blocks = p.batch * p.q_heads * q_tiles;
  float m0 = 0.0f, m1 = 0.0f;
  if ((int)blockIdx.x < q_blocks) {
    const int bh = blockIdx.x / q_tiles, qt = blockIdx.x - bh * q_tiles;
    const int b = bh / p.q_heads, head = bh - b * p.q_heads;
    if (p.tile_spans && head == 0 && tid < 64) {
      const int t = qt * KT + lane;
      const int2 s = t < p.q_len ? row_span(p, b, t) : make_int2(0, 0);
      const bool on = t < p.q_len, some = s.x < s.y;
      const int4 r = {wave_min(some ? s.x : INT32_MAX), wave_max(s.y), wave_max(on ? s.x : 0),
                      wave_min(on ? s.y : INT32_MAX)};
      if (lane == 0) p.tile_spans[(int64_t)b * q_tiles + qt] = r;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int t = qt * KT + 16 * i + (tid >> 4);
      float d = 0.0f, n = 0.0f;
      if (t < p.q_len && 8 * j < p.dim) {
        const E *g = tok_row<E>(p.d_o, b, t, head) + 8 * j;
        const E *o = tok_row<E>(p.o, b, t, head) + 8 * j;
        const f32x4 g0 = load4(g), g1 = load4(g + 4), o0 = load4(o), o1 = load4(o + 4);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          d = fmaf(g0[e], o0[e], fmaf(g1[e], o1[e], d));
          n = fmaf(g0[e], g0[e], fmaf(g1[e], g1[e], n));
        }
      }
      d = group_sum(d, 16);
      if (t < p.q_len && j == 0) p.delta[((int64_t)b * p.q_heads + head) * p.q_len + t] = d;
      if (is_half<E>) {
        m0 = fmaxf(m0, sqrtf(group_sum(n, 16)));
        m1 = fmaxf(m1, fabsf(d));
      }
    }
  } else {
    const int at = blockIdx.x - q_blocks, bh = at / kv_tiles, jt = at - bh * kv_tiles;
    const int b = bh / p.kv_heads, head = bh - b * p.kv_heads;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int t = jt * KT + 16 * i + (tid >> 4);
      float n = 0.0f;
      if (t < p.kv_len && 8 * j < p.dim) {
        const E *v = tok_row<E>(p.v, b, t, head) + 8 * j;
        const f32x4 v0 = load4(v), v1 = load4(v + 4);
#pragma unroll
        for (int e = 0; e < 4; e++) n = fmaf(v0[e], v0[e], fmaf(v1[e], v1[e], n));
      }
      m0 = fmaxf(m0, sqrtf(group_sum(n, 16)));
    }
  }
  if (!is_half<E>) return;
  m0 = wave_fmax(m0);
  m1 = wave_fmax(m1);
  if (lane == 0) {
    top[tid >> 6][0] = m0;
    top[tid >> 6][1] = m1;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < 4; w++) {
      m0 = fmaxf(m0, top[w][0]);
      m1 = fmaxf(m1, top[w][1]);
    }
    if ((int)blockIdx.x < q_blocks) {
      p.q_bound[2 * (int64_t)blockIdx.x] = m0;
      p.q_bound[2 * (int64_t)blockIdx.x + 1] = m1;
    } else {
      p.v_bound[blockIdx.x - q_blocks] = m0;
    }
  }
}

// Largest of n floats at x, `stride` apart, by a block of 256 threads.
__device__ __forceinline__ float block_top(const float *x, int64_t n, int stride, float *lds) {
  float m = 0.0f;
  for (int64_t i = threadIdx.x; i < n; i += 256) m = fmaxf(m, x[i * stride]);
  m = wave_fmax(m);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
}

// Stores a transposed accumulator (lane: a row, registers: its elements) and
// returns the rows (bits 0..31) that hold a NaN and were not stored.
template <class E, int D>
__device__ __forceinline__ uint32_t store_rows(const f32x16 (&acc)[D / 32], float by, E *row,
                                               bool on, int dim, int lane, uint32_t skip) {
  bool nan = false;
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) nan |= acc[d][i] != acc[d][i];
  const uint64_t bits = __builtin_amdgcn_ballot_w64(on && nan);
  skip |= (uint32_t)bits | (uint32_t)(bits >> 32);
  if (on && !(skip >> (lane & 31) & 1)) {
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = 32 * d + acc_row(i, lane);
        const f32x16 x = acc[d];
        if (e < dim) store4(row + e, (f32x4){x[i] * by, x[i + 1] * by, x[i + 2] * by, x[i + 3] * by});
      }
  }
  return skip;
}

// ------------------------------------------------------------ dK and dV
// A block of four waves owns 128 keys of one key head (32 a wave, K and V in
// registers) and streams the queries that see them, head after head of those that
// share the key head, in tiles of 64.
template <class E, int D>
__global__ __launch_bounds__(256, D == 64 ? 2 : 1) void k_attn_bwd_kv(AttnK p, int tiles,
                                                                       int q_tiles) {
  __shared__ __attribute__((aligned(16))) E lds[2][2][KT * D];
  __shared__ __attribute__((aligned(16))) float stat[2][2][KT];
  __shared__ __attribute__((aligned(16))) int2 spans[2][KT];
  __shared__ uint64_t active[WALK / 64], partial[WALK / 64];
  __shared__ float tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int item = die_order(blockIdx.x, gridDim.x);
  const int bh = item / tiles, b = bh / p.kv_heads, kvh = bh - b * p.kv_heads;
  const int key0 = (item - bh * tiles) * 128, mine0 = key0 + 32 * wave;
  const int key = mine0 + (lane & 31);
  const bool on = key < p.kv_len;

  frag<E> kf[D / 16], vf[D / 16];
  {
    const E *kr = tok_row<E>(p.k, b, on ? key : 0, kvh), *vr = tok_row<E>(p.v, b, on ? key : 0, kvh);
#pragma unroll
    for (int k = 0; k < D / 16; k++) {
      const int chunk = 2 * k + (lane >> 5);
      kf[k] = row_operand<E>(kr, chunk, on && 8 * chunk < p.dim);
      vf[k] = row_operand<E>(vr, chunk, on && 8 * chunk < p.dim);
    }
  }
  int e = 0;
  if (is_half<E>) {
    const float *qb = p.q_bound + 2 * ((int64_t)b * p.q_heads + kvh * p.share) * q_tiles;
    const float g = block_top(qb, (int64_t)p.share * q_tiles, 2, tops);
    const float d = block_top(qb + 1, (int64_t)p.share * q_tiles, 2, tops);
    float n = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 16; k++)
#pragma unroll
      for (int i = 0; i < 8; i++) n = fmaf((float)vf[k][i], (float)vf[k][i], n);
    e = headroom(g * sqrtf(other_half(n, false)) + d);
  }
  const float ds_by = is_half<E> ? ldexpf(1.0f, e - 15) : 1.0f;

  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; d++) dk[d] = dv[d] = 0.0f;

  for (int walk0 = 0; walk0 < q_tiles; walk0 += WALK) {
    // Which of the next WALK query tiles see a key of this block, and which of
    // them not all of its keys with all of their rows.
    __syncthreads();
    for (int i = tid; i < WALK; i += 256) {
      const int qt = walk0 + i;
      bool act = qt < q_tiles, part = false;
      if (act && p.tile_spans) {
        const int4 r = p.tile_spans[(int64_t)b * q_tiles + qt];
        act = r.x < key0 + 128 && r.y > key0;
        part = r.z > key0 || r.w < min(key0 + 128, p.kv_len);
      }
      const uint64_t a = __builtin_amdgcn_ballot_w64(act), c = __builtin_amdgcn_ballot_w64(part);
      if (lane == 0) {
        active[i >> 6] = a;
        partial[i >> 6] = c;
      }
    }
    __syncthreads();
    auto next = [&](int from) {  // the first active tile from `from` on, or -1
      for (int w = from >> 6; w < WALK / 64; w++) {
        uint64_t m = active[w];
        if (w == from >> 6) m &= ~0ull << (from & 63);
        if (m) return __builtin_amdgcn_readfirstlane((w << 6) + __builtin_ctzll(m));
      }
      return -1;
    };
    const int first = next(0);
    if (first < 0) continue;

    Staged<E, D, 256, KT> sq, sg;
    float lse = 0.0f, delta = 0.0f;
    int2 span = make_int2(0, 0);
    auto load = [&](int head, int qt) {
      const int t0 = (walk0 + qt) * KT;
      sq.load({tok_row<E>(p.q, b, 0, head), p.q.ts, p.q_len, p.dim}, t0, tid);
      sg.load({tok_row<E>(p.d_o, b, 0, head), p.d_o.ts, p.q_len, p.dim}, t0, tid);
      if (tid < KT) {
        const int t = t0 + tid;
        lse = -INFINITY;
        delta = 0.0f;
        span = make_int2(0, 0);
        if (t < p.q_len) {
          const int64_t at = ((int64_t)b * p.q_heads + head) * p.q_len + t;
          lse = p.lse[at];
          delta = p.delta[at];
          if (p.tile_spans) span = row_span(p, b, t);
        }
      }
    };
    auto put = [&](int at) {
      sq.store(lds[at][0], tid);
      sg.store(lds[at][1], tid);
      if (tid < KT) {
        // a row that sees nothing, or is past the end: p = 2^-inf = 0
        stat[at][0][tid] = lse == -INFINITY ? INFINITY
                                            : lse * ATTN_LOG2E - (is_half<E> ? 15.0f : 0.0f);
        stat[at][1][tid] = delta;
        spans[at][tid] = span;
      }
    };
    int head = kvh * p.share, qt = first, at = 0;
    const int heads = head + p.share;
    load(head, qt);
    put(0);
    __syncthreads();
    while (head < heads) {
      int nqt = next(qt + 1), nhead = head;
      if (nqt < 0) {
        nqt = first;
        nhead++;
      }
      if (nhead < heads) load(nhead, nqt);
      const bool part = partial[qt >> 6] >> (qt & 63) & 1;
      const E *qs = lds[at][0], *gs = lds[at][1];
#pragma unroll
      for (int s = 0; s < KT / 32; s++) {
        f32x16 w = 0.0f, ds = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
          w = mfma(lds_rows<E, D>(qs, 32 * s, k, lane), kf[k], w);
          ds = mfma(lds_rows<E, D>(gs, 32 * s, k, lane), vf[k], ds);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int r = 32 * s + acc_row(i, lane);
          const f32x4 l4 = *(const f32x4 *)&stat[at][0][r], d4 = *(const f32x4 *)&stat[at][1][r];
#pragma unroll
          for (int c = 0; c < 4; c++) {
            w[i + c] = __builtin_amdgcn_exp2f(fmaf(w[i + c], p.scale_log2, -l4[c]));
            ds[i + c] = w[i + c] * (ds[i + c] - d4[c]);
            if (is_half<E>) ds[i + c] *= ds_by;
          }
        }
        if (part) {
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const int2 r = spans[at][32 * s + acc_row(i, lane)];
            if ((unsigned)(key - r.x) >= (unsigned)(r.y - r.x)) w[i] = ds[i] = 0.0f;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const frag<E> pw = pack8<E>(w, k), pd = pack8<E>(ds, k);
#pragma unroll
          for (int d = 0; d < D / 32; d++) {
            dv[d] = mfma(lds_cols<E, D>(gs, 32 * s + 16 * k, d, lane), pw, dv[d]);
            dk[d] = mfma(lds_cols<E, D>(qs, 32 * s + 16 * k, d, lane), pd, dk[d]);
          }
        }
      }
      if (nhead < heads) put(at ^ 1);
      __syncthreads();
      head = nhead;
      qt = nqt;
      at ^= 1;
    }
  }

  uint32_t again = store_rows<E, D>(dk, is_half<E> ? ldexpf(p.scale, -e) : p.scale,
                                    tok_row<E>(p.dk, b, key, kvh), on, p.dim, lane, 0);
  again |= store_rows<E, D>(dv, is_half<E> ? 0x1p-15f : 1.0f, tok_row<E>(p.dv, b, key, kvh), on,
                            p.dim, lane, again);
  if (again) __builtin_amdgcn_s_waitcnt(0x0f70);  // the stores above come first
  while (again) {
    const int r = __builtin_ctz(again);
    again &= again - 1;
    redo_key<E>(p, b, kvh, mine0 + r, lane);
  }
}

// ------------------------------------------------------------ dQ
// The forward's walk with a second score product and without a running maximum.
template <class E, int D, int NQ>
__global__ __launch_bounds__(256, D * NQ <= 128 ? 2 : 1) void k_attn_bwd_q(AttnK p, int tiles,
                                                                            int kv_tiles) {
  __shared__ __attribute__((aligned(16))) E lds[2][2][KT * D];
  __shared__ int2 range[4];
  __shared__ float tops[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int item = die_order(blockIdx.x, gridDim.x);
  const int bh = item / tiles, b = bh / p.q_heads, head = bh - b * p.q_heads;
  const int tile = p.causal ? tiles - 1 - (item - bh * tiles) : item - bh * tiles;
  const int kvh = head / p.share, row0 = tile * 128 * NQ + wave * 32 * NQ + (lane & 31);

  float v_top = 0.0f;
  if (is_half<E>)
    v_top = block_top(p.v_bound + ((int64_t)b * p.kv_heads + kvh) * kv_tiles, kv_tiles, 1, tops);
  frag<E> q[NQ][D / 16], g[NQ][D / 16];
  int2 span[NQ];
  float lse[NQ], delta[NQ];
  int e[NQ];
  int lo = INT32_MAX, hi = 0, in_lo = 0, in_hi = INT32_MAX;
#pragma unroll
  for (int n = 0; n < NQ; n++) {
    const int t = row0 + 32 * n;
    const bool on = t < p.q_len;
    span[n] = on ? row_span(p, b, t) : make_int2(0, 0);
    lse[n] = -INFINITY;
    delta[n] = 0.0f;
    if (on) {
      in_lo = max(in_lo, span[n].x);
      in_hi = min(in_hi, span[n].y);
      if (span[n].x < span[n].y) {
        lo = min(lo, span[n].x);
        hi = max(hi, span[n].y);
      }
      const int64_t at = ((int64_t)b * p.q_heads + head) * p.q_len + t;
      lse[n] = p.lse[at];
      delta[n] = p.delta[at];
    }
    const E *qr = tok_row<E>(p.q, b, on ? t : 0, head), *gr = tok_row<E>(p.d_o, b, on ? t : 0, head);
    float norm = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 16; k++) {
      const int chunk = 2 * k + (lane >> 5);
      q[n][k] = row_operand<E>(qr, chunk, on && 8 * chunk < p.dim);
      g[n][k] = row_operand<E>(gr, chunk, on && 8 * chunk < p.dim);
      if (is_half<E>)
#pragma unroll
        for (int i = 0; i < 8; i++) norm = fmaf((float)g[n][k][i], (float)g[n][k][i], norm);
    }
    e[n] = is_half<E> ? headroom(sqrtf(other_half(norm, false)) * v_top + fabsf(delta[n])) : 0;
    lse[n] = lse[n] == -INFINITY ? INFINITY : lse[n] * ATTN_LOG2E - (float)e[n];
  }
  lo = __builtin_amdgcn_readfirstlane(wave_min(lo));
  hi = __builtin_amdgcn_readfirstlane(wave_max(hi));
  in_lo = __builtin_amdgcn_readfirstlane(wave_max(in_lo));
  in_hi = __builtin_amdgcn_readfirstlane(wave_min(in_hi));
  if (lane == 0) range[wave] = make_int2(lo, hi);
  __syncthreads();
  int first = INT32_MAX, end = 0;
#pragma unroll
  for (int w = 0; w < 4; w++) {
    first = min(first, range[w].x);
    end = max(end, range[w].y);
  }
  first = __builtin_amdgcn_readfirstlane(first < end ? first / KT : 0);
  end = __builtin_amdgcn_readfirstlane((end + KT - 1) / KT);

  const Stream<E> ks = {tok_row<E>(p.k, b, 0, kvh), p.k.ts, p.kv_len, p.dim};
  const Stream<E> vs = {tok_row<E>(p.v, b, 0, kvh), p.v.ts, p.kv_len, p.dim};
  f32x16 dq[NQ][D / 32];
#pragma unroll
  for (int n = 0; n < NQ; n++)
#pragma unroll
    for (int d = 0; d < D / 32; d++) dq[n][d] = 0.0f;
  Staged<E, D, 256, KT> sk, sv;
  if (first < end) {
    sk.load(ks, first * KT, tid);
    sv.load(vs, first * KT, tid);
    sk.store(lds[0][0], tid);
    sv.store(lds[0][1], tid);
  }
  __syncthreads();
  for (int j = first; j < end; j++) {
    const int at = (j - first) & 1;
    if (j + 1 < end) {
      sk.load(ks, (j + 1) * KT, tid);
      sv.load(vs, (j + 1) * KT, tid);
    }
    const int key0 = j * KT;
    if (key0 < hi && key0 + KT > lo) {
      const bool full = key0 >= in_lo && key0 + KT <= in_hi;
      const E *kt = lds[at][0], *vt = lds[at][1];
#pragma unroll
      for (int s = 0; s < KT / 32; s++) {
        f32x16 w[NQ], ds[NQ];
#pragma unroll
        for (int n = 0; n < NQ; n++) w[n] = ds[n] = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
          const frag<E> a = lds_rows<E, D>(kt, 32 * s, k, lane), c = lds_rows<E, D>(vt, 32 * s, k, lane);
#pragma unroll
          for (int n = 0; n < NQ; n++) {
            w[n] = mfma(a, q[n][k], w[n]);
            ds[n] = mfma(c, g[n][k], ds[n]);
          }
        }
#pragma unroll
        for (int n = 0; n < NQ; n++) {
#pragma unroll
          for (int i = 0; i < 16; i++)
            ds[n][i] = __builtin_amdgcn_exp2f(fmaf(w[n][i], p.scale_log2, -lse[n])) *
                       (ds[n][i] - delta[n]);
          if (!full) {
#pragma unroll
            for (int i = 0; i < 16; i++) {
              const int key = key0 + 32 * s + acc_row(i, lane);
              if ((unsigned)(key - span[n].x) >= (unsigned)(span[n].y - span[n].x)) ds[n][i] = 0.0f;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 2; k++) {
          frag<E> pd[NQ];
#pragma unroll
          for (int n = 0; n < NQ; n++) pd[n] = pack8<E>(ds[n], k);
#pragma unroll
          for (int d = 0; d < D / 32; d++) {
            const frag<E> a = lds_cols<E, D>(kt, 32 * s + 16 * k, d, lane);
#pragma unroll
            for (int n = 0; n < NQ; n++) dq[n][d] = mfma(a, pd[n], dq[n][d]);
          }
        }
      }
    }
    if (j + 1 < end) {
      sk.store(lds[at ^ 1][0], tid);
      sv.store(lds[at ^ 1][1], tid);
    }
    __syncthreads();
  }
#pragma unroll
  for (int n = 0; n < NQ; n++) {
    const int t = row0 + 32 * n;
    const bool on = t < p.q_len;
    uint32_t again = store_rows<E, D>(dq[n], is_half<E> ? ldexpf(p.scale, -e[n]) : p.scale,
                                      tok_row<E>(p.dq, b, on ? t : 0, head), on, p.dim, lane, 0);
    while (again) {
      const int r = __builtin_ctz(again);
      again &= again - 1;
      redo_query<E>(p, b, head, tile * 128 * NQ + wave * 32 * NQ + 32 * n + r, lane);
    }
  }
}

template <class E, int D>
hipError_t launch(const AttnK &p, hipStream_t st) {
  const int q_tiles = (p.q_len + KT - 1) / KT, kv_tiles = (p.kv_len + KT - 1) / KT;
  const int prep = p.batch * (p.q_heads * q_tiles + (is_half<E> ? p.kv_heads * kv_tiles : 0));
  if (prep) k_attn_prep<E><<<prep, 256, 0, st>>>(p, q_tiles, kv_tiles);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int k_tiles = (p.kv_len + 127) / 128, tiles = (p.q_len + 127) / 128;
  if (k_tiles) k_attn_bwd_kv<E, D><<<p.batch * p.kv_heads * k_tiles, 256, 0, st>>>(p, k_tiles, q_tiles);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (tiles) k_attn_bwd_q<E, D, 1><<<p.batch * p.q_heads * tiles, 256, 0, st>>>(p, tiles, kv_tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t gs_launch_attn_bwd(const AttnK &p, int dtype, hipStream_t st) {
  if (dtype == GS_BF16) return p.dim <= 64 ? launch<bf16_t, 64>(p, st) : launch<bf16_t, 128>(p, st);
  return p.dim <= 64 ? launch<f16_t, 64>(p, st) : launch<f16_t, 128>(p, st);
}
