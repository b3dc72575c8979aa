// Attention: o_i = sum_j p_ij v_j, p_ij = exp(s_ij - lse_i), s_ij = scale q_i . k_j
// over the keys j of query i's span, lse_i = log sum_j exp s_ij. A query that
// sees no key gets o = 0, lse = -inf.
//
// One pass over the keys with a running reference m_i and sum l_i (32 bits, in
// powers of two): p = 2^(s - m), o and l scaled by 2^(m - m') when the reference
// moves. It moves only when some score of the wave passes it by 8 (p <= 256
// stays exact enough in 16 bits: rounding is relative), so most tiles skip the
// 16 D / 32 multiplications per row block.
// p is rounded to the inputs' 16-bit type for the second product, as matrix
// instructions take it; l sums the unrounded p.
#include "attention_common.h"

namespace {

// ------------------------------------------------------------ rows done again
// 0 x NaN and 0 x infinity are NaN: in a matrix product, a masked key whose value
// row is not finite spoils rows that do not see it. A row whose result holds a
// NaN is therefore computed again from its own keys alone, by one wave: a lane
// takes a key's score, then two elements of the output.
template <class E>
__device__ void redo_row(const AttnK &p, int b, int head, int t, int lane) {
  const int2 span = row_span(p, b, t);
  const int kvh = head / p.share;
  const E *q = tok_row<E>(p.q, b, t, head);
  float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
  for (int j0 = span.x; j0 < span.y; j0 += 64) {
    const int n = min(64, span.y - j0);
    float s = -INFINITY;
    if (lane < n) s = dot_row(q, tok_row<E>(p.k, b, j0 + lane, kvh), p.dim) * p.scale_log2;
    const float top = fmaxf(m, wave_fmax(s)), ref = top == -INFINITY ? 0.0f : top;
    const float w = lane < n ? __builtin_amdgcn_exp2f(s - ref) : 0.0f;
    const float shrink = __builtin_amdgcn_exp2f((m == -INFINITY ? ref : m) - ref);
    l = l * shrink + group_sum(w, 64);
    o0 *= shrink;
    o1 *= shrink;
    m = top;
    for (int j = 0; j < n; j++) {
      const E *v = tok_row<E>(p.v, b, j0 + j, kvh);
      const float wj = __shfl(w, j);
      if (lane < p.dim) o0 = fmaf(wj, (float)v[lane], o0);
      if (lane + 64 < p.dim) o1 = fmaf(wj, (float)v[lane + 64], o1);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  E *o = tok_row<E>(p.o, b, t, head);
  if (lane < p.dim) o[lane] = (E)(o0 * inv);
  if (lane + 64 < p.dim) o[lane + 64] = (E)(o1 * inv);
  if (lane == 0)
    p.lse[((int64_t)b * p.q_heads + head) * p.q_len + t] =
        l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + __builtin_amdgcn_logf(l)) * ATTN_LN2;
}

// A wave's running softmax over NQ blocks of 32 rows and its share of o.
template <class E, int D, int NQ>
struct Softmax {
  f32x16 o[NQ][D / 32];
  float m[NQ], l[NQ];

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int n = 0; n < NQ; n++) {
      m[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 32; d++) o[n][d] = 0.0f;
    }
  }

  // One tile of 32 NS keys from row `key0` of the streams (row 0 of the tiles).
  // full: every row of the wave sees all of them.
  template <int NS>
  __device__ __forceinline__ void tile(const E *kt, const E *vt, const frag<E> (&q)[NQ][D / 16],
                                       const int2 (&span)[NQ], bool full, int key0,
                                       float scale_log2, int lane) {
    f32x16 s[NQ][NS];
    frag<E> a[NS][D / 16];
#pragma unroll
    for (int k = 0; k < D / 16; k++)
#pragma unroll
      for (int b = 0; b < NS; b++) a[b][k] = lds_rows<E, D>(kt, 32 * b, k, lane);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < D / 16; k++)
#pragma unroll
      for (int n = 0; n < NQ; n++)
#pragma unroll
        for (int b = 0; b < NS; b++) {
          if (k == 0) s[n][b] = 0.0f;
          s[n][b] = mfma(a[b][k], q[n][k], s[n][b]);
        }
    if (!full) {
#pragma unroll
      for (int n = 0; n < NQ; n++)
#pragma unroll
        for (int b = 0; b < NS; b++)
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const int j = key0 + 32 * b + acc_row(i, lane);
            if ((unsigned)(j - span[n].x) >= (unsigned)(span[n].y - span[n].x))
              s[n][b][i] = -INFINITY;
          }
    }
    // the first half's values, on their way while the softmax is computed
    frag<E> v0[2][D / 32];
#pragma unroll
    for (int k = 0; k < 2; k++)
#pragma unroll
      for (int d = 0; d < D / 32; d++) v0[k][d] = lds_cols<E, D>(vt, 16 * k, d, lane);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NQ; n++) {
      float top = s[n][0][0];
#pragma unroll
      for (int b = 0; b < NS; b++)
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, s[n][b][i]);
      top = other_half(top, true) * scale_log2;
      if (__builtin_amdgcn_ballot_w64(top > m[n] + 8.0f)) {
        const float to = fmaxf(m[n], top), ref = to == -INFINITY ? 0.0f : to;
        const float shrink = __builtin_amdgcn_exp2f((m[n] == -INFINITY ? ref : m[n]) - ref);
        m[n] = to;
        l[n] *= shrink;
#pragma unroll
        for (int d = 0; d < D / 32; d++) o[n][d] *= shrink;
      }
      const float ref = m[n] == -INFINITY ? 0.0f : m[n];
      float sum = 0.0f;
#pragma unroll
      for (int b = 0; b < NS; b++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
          s[n][b][i] = __builtin_amdgcn_exp2f(fmaf(s[n][b][i], scale_log2, -ref));
          sum += s[n][b][i];
        }
      l[n] += sum;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NS; b++) {
      frag<E> c[2][D / 32];
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int d = 0; d < D / 32; d++) c[k][d] = b ? lds_cols<E, D>(vt, 32 * b + 16 * k, d, lane) : v0[k][d];
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int n = 0; n < NQ; n++) {
          const frag<E> w = pack8<E>(s[n][b], k);
#pragma unroll
          for (int d = 0; d < D / 32; d++) o[n][d] = mfma(c[k][d], w, o[n][d]);
        }
    }
  }
};

// ------------------------------------------------------------ many rows
// A block of four waves takes 128 NQ queries of one head and streams the keys
// and values of their spans through LDS in tiles of 64, the next one on its way
// while this one is computed.
template <class E, int D, int NQ>
__global__ __launch_bounds__(256, D * NQ <= 128 ? 2 : 1) void k_attn_fwd(AttnK p, int tiles) {
  // Objects of their own, and turns of the loop that name theirs: the compiler then
  // sees that reads of one do not wait for copies into the other.
  using Buf = E[2][KT * D];
  __shared__ __attribute__((aligned(16))) Buf b0, b1;
  __shared__ int2 range[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int item = die_order(blockIdx.x, gridDim.x);
  const int2 bt = block_item(p, item, p.batch * p.q_heads, tiles);
  const int bh = bt.x, tile = bt.y, b = bh / p.q_heads, head = bh - b * p.q_heads;
  const int kvh = head / p.share, row0 = tile * 128 * NQ + wave * 32 * NQ + (lane & 31);

  frag<E> q[NQ][D / 16];
  int2 span[NQ];
  int lo = INT32_MAX, hi = 0, in_lo = 0, in_hi = INT32_MAX;
#pragma unroll
  for (int n = 0; n < NQ; n++) {
    const int t = row0 + 32 * n;
    const bool on = t < p.q_len;
    span[n] = on ? row_span(p, b, t) : make_int2(0, 0);
    if (on) {
      in_lo = max(in_lo, span[n].x);
      in_hi = min(in_hi, span[n].y);
      if (span[n].x < span[n].y) {
        lo = min(lo, span[n].x);
        hi = max(hi, span[n].y);
      }
    }
    const E *row = tok_row<E>(p.q, b, on ? t : 0, head);
#pragma unroll
    for (int k = 0; k < D / 16; k++) {
      const int chunk = 2 * k + (lane >> 5);
      q[n][k] = row_operand<E>(row, chunk, on && 8 * chunk < p.dim);
    }
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
  Softmax<E, D, NQ> sm;
  sm.init();
  using Tile = Copy<E, D, 256, KT>;
  if (first < end) {
    Tile::issue(ks, first * KT, b0[0], tid);
    Tile::issue(vs, first * KT, b0[1], tid);
  }
  auto turn = [&](int j, Buf &here, Buf &there) {
    block_copied();  // tile j is there, and nobody reads the other one any more
    if (j + 1 < end) {
      Tile::issue(ks, (j + 1) * KT, there[0], tid);
      Tile::issue(vs, (j + 1) * KT, there[1], tid);
    }
    const int key0 = j * KT;
    if (key0 < hi && key0 + KT > lo)
      sm.template tile<KT / 32>(here[0], here[1], q, span, key0 >= in_lo && key0 + KT <= in_hi,
                                key0, p.scale_log2, lane);
  };
  for (int j = first; j < end; j += 2) {
    turn(j, b0, b1);
    if (j + 1 < end) turn(j + 1, b1, b0);
  }

#pragma unroll
  for (int n = 0; n < NQ; n++) {
    const int t = row0 + 32 * n;
    const bool on = t < p.q_len;
    const float l = other_half(sm.l[n], false), inv = l == 0.0f ? 0.0f : 1.0f / l;
    bool nan = false;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int i = 0; i < 16; i++) {
        sm.o[n][d][i] *= inv;
        nan |= sm.o[n][d][i] != sm.o[n][d][i];
      }
    uint64_t again = __builtin_amdgcn_ballot_w64(on && nan);
    again = (again | again >> 32) & 0xffffffffu;
    const bool keep = on && !(again >> (lane & 31) & 1);
    if (keep) {
      E *o = tok_row<E>(p.o, b, t, head);
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int e = 32 * d + acc_row(i, lane);
          const f32x16 x = sm.o[n][d];
          if (e < p.dim) store4(o + e, (f32x4){x[i], x[i + 1], x[i + 2], x[i + 3]});
        }
      if (lane < 32)
        p.lse[((int64_t)b * p.q_heads + head) * p.q_len + t] =
            l == 0.0f ? -INFINITY
                      : ((sm.m[n] == -INFINITY ? 0.0f : sm.m[n]) + __builtin_amdgcn_logf(l)) *
                            ATTN_LN2;
    }
    while (again) {
      const int r = __builtin_ctzll(again);
      again &= again - 1;
      redo_row<E>(p, b, head, tile * 128 * NQ + wave * 32 * NQ + 32 * n + r, lane);
    }
  }
}

// ------------------------------------------------------------ few rows
// Single tokens and short queries over long caches: the share x q_len rows that
// read one key head are packed into blocks of 32 (row r is token r / share of
// head r % share), the keys are cut into `splits` parts for as many workgroups,
// and the four waves of a block take every fourth tile of 32 keys of its part,
// each in LDS of its own, without barriers. The block joins its waves; the
// parts' m, l and o go to the workspace in 32 bits and are joined by
// k_attn_join.
constexpr int FT = 32;

template <class E, int D>
__global__ __launch_bounds__(256, 1) void k_attn_few(AttnK p, int row_tiles) {
  // per wave two tiles of keys and values; afterwards m, l and o of the waves
  using Buf = E[4][2][FT * D];
  __shared__ __attribute__((aligned(16))) Buf b0, b1;
  __shared__ float ml[4][2][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int item = die_order(blockIdx.x, gridDim.x);
  const int part = item % p.splits, rest = item / p.splits;
  const int rt = rest % row_tiles, bh = rest / row_tiles;
  const int b = bh / p.kv_heads, kvh = bh - b * p.kv_heads;
  const int64_t rows = (int64_t)p.q_len * p.share, r = (int64_t)rt * 32 + (lane & 31);
  const bool on = r < rows;
  const int t = on ? (int)(r / p.share) : 0, head = kvh * p.share + (on ? (int)(r % p.share) : 0);

  frag<E> q[1][D / 16];
  const E *row = tok_row<E>(p.q, b, t, head);
#pragma unroll
  for (int k = 0; k < D / 16; k++) {
    const int chunk = 2 * k + (lane >> 5);
    q[0][k] = row_operand<E>(row, chunk, on && 8 * chunk < p.dim);
  }
  int2 span[1] = {on ? row_span(p, b, t) : make_int2(0, 0)};
  const int p0 = part * p.split_keys, p1 = min(p0 + p.split_keys, p.kv_len);
  const int lo = max(wave_min(span[0].x < span[0].y ? span[0].x : INT32_MAX), p0);
  const int hi = min(wave_max(span[0].y), p1);
  const int in_lo = wave_max(on ? span[0].x : 0), in_hi = wave_min(on ? span[0].y : INT32_MAX);
  span[0].x = max(span[0].x, p0);
  span[0].y = min(span[0].y, p1);
  if (span[0].x >= span[0].y) span[0] = make_int2(0, 0);

  const Stream<E> ks = {tok_row<E>(p.k, b, 0, kvh), p.k.ts, p.kv_len, p.dim};
  const Stream<E> vs = {tok_row<E>(p.v, b, 0, kvh), p.v.ts, p.kv_len, p.dim};
  Softmax<E, D, 1> sm;
  sm.init();
  using Tile = Copy<E, D, 64, FT>;
  const int first = __builtin_amdgcn_readfirstlane(lo < hi ? lo / FT + wave : 0);
  const int end = __builtin_amdgcn_readfirstlane(lo < hi ? (hi + FT - 1) / FT : 0);
  if (first < end) {
    Tile::issue(ks, first * FT, b0[wave][0], lane);
    Tile::issue(vs, first * FT, b0[wave][1], lane);
  }
  auto turn = [&](int j, Buf &here, Buf &there) {
    if (j + 4 < end) {
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the buffer's last reads are done
      Tile::issue(ks, (j + 4) * FT, there[wave][0], lane);
      Tile::issue(vs, (j + 4) * FT, there[wave][1], lane);
      copied<2 * Tile::N>();
    } else {
      copied<0>();
    }
    wave_order();
    const int key0 = j * FT;
    const bool full = key0 >= in_lo && key0 + FT <= in_hi && key0 >= p0 && key0 + FT <= p1;
    sm.template tile<1>(here[wave][0], here[wave][1], q, span, full, key0, p.scale_log2, lane);
  };
  for (int j = first; j < end; j += 8) {
    turn(j, b0, b1);
    if (j + 4 < end) turn(j + 4, b1, b0);
  }

  // Join the waves: a common reference, then sums in LDS in wave order.
  sm.l[0] = other_half(sm.l[0], false);
  if (lane < 32) {
    ml[wave][0][lane] = sm.m[0];
    ml[wave][1][lane] = sm.l[0];
  }
  __syncthreads();
  float m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; w++) m = fmaxf(m, ml[w][0][lane & 31]);
  const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
  for (int w = 0; w < 4; w++)
    l += ml[w][1][lane & 31] * __builtin_amdgcn_exp2f(ml[w][0][lane & 31] - ref);
  const float mine = __builtin_amdgcn_exp2f(sm.m[0] - ref);
  float *sum = (float *)&b0[0][0][0];  // [32][D + 4]
  for (int w = 0; w < 4; w++) {
    if (w == wave) {
      float *to = sum + (lane & 31) * (D + 4);
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x16 o = sm.o[0][d];
          f32x4 x = {o[i], o[i + 1], o[i + 2], o[i + 3]};
          f32x4 *at4 = (f32x4 *)(to + 32 * d + acc_row(i, lane));
          x *= mine;
          *at4 = w ? *at4 + x : x;
        }
    }
    __syncthreads();
  }
  if (wave == 0 && lane < 32) {
    ml[0][0][lane] = m;
    ml[0][1][lane] = l;
  }
  __syncthreads();
  // Eight threads a row.
  const int rr = tid >> 3;
  const int64_t r2 = min((int64_t)rt * 32 + rr, rows - 1);
  const bool live = (int64_t)rt * 32 + rr < rows;
  const int t2 = (int)(r2 / p.share), head2 = kvh * p.share + (int)(r2 % p.share);
  m = ml[0][0][rr];
  l = ml[0][1][rr];
  const int64_t at_row = ((int64_t)b * p.q_heads + head2) * p.q_len + t2;
  if (p.splits > 1) {
    if (!live) return;
    const int64_t all = (int64_t)p.batch * p.q_heads * p.q_len, slot = part * all + at_row;
    for (int e = 4 * (tid & 7); e < p.dim; e += 32)
      *(f32x4 *)(p.part_o + slot * p.dim + e) = *(const f32x4 *)(sum + rr * (D + 4) + e);
    if ((tid & 7) == 0) {
      p.part_ml[2 * slot] = m;
      p.part_ml[2 * slot + 1] = l;
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  bool nan = false;
  E *o = tok_row<E>(p.o, b, t2, head2);
  for (int e = 4 * (tid & 7); live && e < p.dim; e += 32) {
    const f32x4 x = *(const f32x4 *)(sum + rr * (D + 4) + e) * inv;
    nan |= x[0] != x[0] || x[1] != x[1] || x[2] != x[2] || x[3] != x[3];
    store4(o + e, x);
  }
  if (live && (tid & 7) == 0)
    p.lse[at_row] = l == 0.0f ? -INFINITY
                              : ((m == -INFINITY ? 0.0f : m) + __builtin_amdgcn_logf(l)) * ATTN_LN2;
  // Rows of this wave whose result holds a NaN, after its stores.
  uint64_t again = __builtin_amdgcn_ballot_w64(nan);
  if (again) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  for (int k = 0; k < 8 && again; k++) {
    if (!(again >> (8 * k) & 0xff)) continue;
    const int64_t r3 = (int64_t)rt * 32 + wave * 8 + k;
    redo_row<E>(p, b, kvh * p.share + (int)(r3 % p.share), (int)(r3 / p.share), lane);
  }
}

// Joins the parts of one row: a block a row, 32 lanes with four elements each for
// every eighth part.
template <class E>
__global__ __launch_bounds__(256) void k_attn_join(AttnK p) {
  __shared__ float tops[4];
  __shared__ __attribute__((aligned(16))) float sums[8][132];
  const int tid = threadIdx.x, lane = tid & 63, e = 4 * (tid & 31);
  const int64_t all = (int64_t)p.batch * p.q_heads * p.q_len, row = blockIdx.x;
  float top = -INFINITY;
  for (int s = tid; s < p.splits; s += 256) top = fmaxf(top, p.part_ml[2 * (s * all + row)]);
  top = wave_fmax(top);
  if (lane == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float ref = top == -INFINITY ? 0.0f : top;
  float l = 0.0f;
  f32x4 o = 0.0f;
#pragma unroll 4
  for (int s = tid >> 5; s < p.splits; s += 8) {
    const int64_t slot = s * all + row;
    const float w = __builtin_amdgcn_exp2f(p.part_ml[2 * slot] - ref);
    l = fmaf(p.part_ml[2 * slot + 1], w, l);
    if (e < p.dim) o += *(const f32x4 *)(p.part_o + slot * p.dim + e) * w;
  }
  *(f32x4 *)&sums[tid >> 5][e] = o;
  if ((tid & 31) == 0) sums[tid >> 5][128] = l;
  __syncthreads();
  if (tid >= 64) return;
  l = 0.0f;
  float o0 = 0.0f, o1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    l += sums[i][128];
    o0 += sums[i][lane];
    o1 += sums[i][lane + 64];
  }
  const int64_t bh = row / p.q_len;
  const int t = (int)(row - bh * p.q_len), b = (int)(bh / p.q_heads);
  const int head = (int)(bh - (int64_t)b * p.q_heads);
  if (__builtin_amdgcn_ballot_w64(o0 != o0 || o1 != o1)) {
    redo_row<E>(p, b, head, t, lane);
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  E *to = tok_row<E>(p.o, b, t, head);
  if (lane < p.dim) to[lane] = (E)(o0 * inv);
  if (lane + 64 < p.dim) to[lane + 64] = (E)(o1 * inv);
  if (lane == 0)
    p.lse[row] = l == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(l)) * ATTN_LN2;
}

template <class E, int D>
hipError_t launch(const AttnK &p, hipStream_t st) {
  if (p.splits) {
    const int row_tiles = (int)(((int64_t)p.q_len * p.share + 31) / 32);
    k_attn_few<E, D><<<p.batch * p.kv_heads * row_tiles * p.splits, 256, 0, st>>>(p, row_tiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t rows = (int64_t)p.batch * p.q_heads * p.q_len;
    k_attn_join<E><<<(unsigned)rows, 256, 0, st>>>(p);
    return hipGetLastError();
  }
  const int tiles = (p.q_len + 127) / 128;
  k_attn_fwd<E, D, 1><<<p.batch * p.q_heads * tiles, 256, 0, st>>>(p, tiles);
  return hipGetLastError();
}

}  // namespace

// The split of the keys that a call takes, 0: the form for many rows.
//   few rows: no more than 32 rows read a key head (one block of rows), or the
//   form for many rows would leave most of 256 compute units without work.
void gs_attn_plan(AttnK *p) {
  const int64_t rows = (int64_t)p->q_len * p->share, row_tiles = (rows + 31) / 32;
  const int64_t many = (int64_t)p->batch * p->q_heads * ((p->q_len + 127) / 128);
  p->splits = 0;
  p->split_keys = 0;
  if (!p->batch || !p->q_len || (rows > 32 && many >= 256)) return;
  const int64_t blocks = (int64_t)p->batch * p->kv_heads * row_tiles;
  // about 512 workgroups, none with fewer than 256 keys
  int64_t splits = (512 + blocks - 1) / blocks;
  const int64_t most = (p->kv_len + 255) / 256;
  splits = splits < most ? splits : most;
  if (splits < 1) splits = 1;
  const int64_t keys = ((p->kv_len + splits - 1) / splits + FT - 1) / FT * FT;
  p->split_keys = (int)(keys ? keys : FT);
  p->splits = (int)(p->kv_len ? (p->kv_len + p->split_keys - 1) / p->split_keys : 1);
}

hipError_t gs_launch_attn_fwd(const AttnK &p, int dtype, hipStream_t st) {
  if (dtype == GS_BF16) return p.dim <= 64 ? launch<bf16_t, 64>(p, st) : launch<bf16_t, 128>(p, st);
  return p.dim <= 64 ? launch<f16_t, 64>(p, st) : launch<f16_t, 128>(p, st);
}
