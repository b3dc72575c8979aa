// Attention: o_i = sum_j p_ij v_j, p_ij = exp(s_ij - lse_i), s_ij = scale q_i . k_j
// over the keys j of query i's span, lse_i = log sum_j exp s_ij. A query that
// sees no key gets o = 0, lse = -inf.
//
// One pass over the keys with a running reference m_i and sum l_i (32 bits, in
// powers of two): p = 2^(s - m), o and l scaled by 2^(m - m') when the reference
// moves. It moves only when some score of the wave passes it by 8 (rounding is
// relative, so p above 1 are as exact as those below). In fp16 p below 2^-14 lose bits and
// below 2^-25 count as 0, which many keys add up: there the reference is taken 5 below the
// largest score and moves when one passes it by 10, so that p is off by 2^-30 of the row's
// largest at most.
// With many rows a wave looks for its largest scores in the first tile only. Later
// tiles compute p with the reference that is there; if a lane's sum of them passes 2^13
// (fp16: 2^15; or is NaN), the wave computes the tile's scores again and looks. Both measured
// in turn: 2 x 8192 tokens, 16 heads of 64: 5% less than looking at every tile; with few rows
// (2331 tokens, 8 heads of 64) 27 us and 24, there every tile is looked at.
// p is rounded to the inputs' 16-bit type for the second product, as matrix
// instructions take it; l sums the unrounded p.
#include "attention_common.h"

namespace {

// ------------------------------------------------------------ rows done again
// One row's o (its lse is right: masked scores are replaced): a lane takes a key's score.
template <class E, int N>
__device__ __forceinline__ void redo_row(const AttnK &p, int b, int head, int t, int lane) {
  const int2 span = row_span(p, b, t);
  const int kvh = head / p.share;
  const E *q = tok_row<E>(p.q, b, t, head);
  float m = -INFINITY, l = 0.0f;
  RowSum<N> o;
  bool open = true;
#pragma unroll 1
  for (int j0 = span.x; open && j0 < span.y; j0 += 64) {
    const int n = min(64, span.y - j0);
    float s = -INFINITY;
    if (lane < n) s = dot_row<4>(q, tok_row<E>(p.k, b, j0 + lane, kvh), p.dim) * p.scale_log2;
    const float top = fmaxf(m, wave_fmax(s)), ref = top == -INFINITY ? 0.0f : top;
    const float w = lane < n ? __builtin_amdgcn_exp2f(s - ref) : 0.0f;
    const float shrink = __builtin_amdgcn_exp2f((m == -INFINITY ? ref : m) - ref);
    l = l * shrink + group_sum(w, 64);
    o.shrink(shrink);
    m = top;
    open = o.template add<E>(w, first_bits(n), p.v, b, kvh, j0, span.y - 1, p.dim, lane);
  }
  o.store(tok_row<E>(p.o, b, t, head), l == 0.0f ? 0.0f : 1.0f / l, p.dim, lane);
}

// How far the reference is below the largest score when it moves, and how far a score may
// pass it, in powers of two; and the largest sum of a lane's p of a tile that needs no look:
// that of its 32 p as large as a look leaves them, each of which fits the type.
template <class E>
struct Room {
  static constexpr float BELOW = 0.0f, PASS = 8.0f, SUM = 0x1p13f;
};
template <>
struct Room<f16_t> {
  static constexpr float BELOW = 5.0f, PASS = 10.0f, SUM = 0x1p15f;
};

// A wave's running softmax over its 32 rows and its share of o.
template <class E, int D>
struct Softmax {
  f32x16 o[D / 32];
  float m, l;

  // sees: whether the lane's row sees any key (one that does not has no reference to
  // wait for).
  __device__ __forceinline__ void init(bool sees) {
    m = sees ? -INFINITY : 0.0f;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 32; d++) o[d] = 0.0f;
  }

  // A tile of 32 NS keys, the first of them `key0`. full: every row of the wave sees all
  // of them.
  template <int NS>
  __device__ __forceinline__ void tile(const E *kt, const E *vt, const frag<E> (&q)[D / 16],
                                       int2 span, bool full, int key0, float scale_log2, int lane) {
    // The keys' operands of step k, AHEAD steps before they are used: a wave waits for
    // LDS once, not at every step, and the registers hold them beside o (168 of the form
    // of 96, else 256; that one also reads no values early).
    constexpr int STEPS = D / 16, AHEAD = D == 96 ? 2 : 4;
    f32x16 s[NS];
    frag<E> v0[2][D / 32];
    float sum;
    bool look = NS == 1 || __builtin_amdgcn_ballot_w64(m == -INFINITY);
    for (;;) {
      frag<E> a[NS][STEPS];
      auto read = [&](int k) {
#pragma unroll
        for (int b = 0; b < NS; b++) a[b][k] = lds_rows<E, D>(kt, 32 * b, k, lane);
      };
#pragma unroll
      for (int k = 0; k < AHEAD; k++) read(k);
#pragma unroll
      for (int k = 0; k < STEPS; k++) {
        __builtin_amdgcn_sched_barrier(0);
        if (k + AHEAD < STEPS) read(k + AHEAD);
#pragma unroll
        for (int b = 0; b < NS; b++) {
          if (k == 0) s[b] = 0.0f;
          s[b] = mfma(a[b][k], q[k], s[b]);
        }
      }
      if (!full) {
#pragma unroll
        for (int b = 0; b < NS; b++)
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const int j = key0 + 32 * b + acc_row(i, lane);
            if ((unsigned)(j - span.x) >= (unsigned)(span.y - span.x)) s[b][i] = -INFINITY;
          }
      }
      // the first 32 keys' values, on their way while the softmax is computed
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int d = 0; d < D / 32; d++)
          if (D != 96) v0[k][d] = lds_cols<E, D>(vt, 16 * k, d, lane);
      __builtin_amdgcn_sched_barrier(0);
      if (look) {
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < NS; b++)
#pragma unroll
          for (int i = 0; i < 16; i++) top = fmaxf(top, s[b][i]);
        top = other_half(top, true) * scale_log2;
        if (__builtin_amdgcn_ballot_w64(top > m + Room<E>::PASS)) {
          const float to = fmaxf(m, top - Room<E>::BELOW), ref = to == -INFINITY ? 0.0f : to;
          const float shrink = __builtin_amdgcn_exp2f((m == -INFINITY ? ref : m) - ref);
          m = to;
          l *= shrink;
#pragma unroll
          for (int d = 0; d < D / 32; d++) o[d] *= shrink;
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      sum = 0.0f;
#pragma unroll
      for (int b = 0; b < NS; b++)
#pragma unroll
        for (int i = 0; i < 16; i++) {
          s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], scale_log2, -ref));
          sum += s[b][i];
        }
      if (look || !__builtin_amdgcn_ballot_w64(!(sum <= Room<E>::SUM))) break;
      look = true;
    }
    l += sum;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NS; b++) {
      frag<E> c[2][D / 32];
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int d = 0; d < D / 32; d++)
          c[k][d] = b || D == 96 ? lds_cols<E, D>(vt, 32 * b + 16 * k, d, lane) : v0[k][d];
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const frag<E> w = pack8<E>(s[b], k);
#pragma unroll
        for (int d = 0; d < D / 32; d++) o[d] = mfma(c[k][d], w, o[d]);
      }
    }
  }
};

// ------------------------------------------------------------ many rows
// A block takes 128 queries of one head, 32 a wave, and streams the keys and values
// of their spans through LDS in tiles of 64, the next one on its way while this one is
// computed.
// Bound by the matrix units, and in short calls by how evenly blocks fall on the
// compute units: 16384 tokens, 8 heads of 128, bf16: 985 us, 1116 TFLOP/s. Heads of 65
// to 96 have a form of 96, of which three blocks fit a compute unit: 6037 tokens in four
// sequences, 12 heads of 80: 55 us, in the form of 128 67; 2 x 2048 tokens, 12 heads of
// 80: 59 and 70. 64 rows a wave instead of 32 took 17% longer (2 x 8192 tokens, 16 heads of
// 64, in turn: there the exponentials take as long as the products; 580 to 680 us now, by
// the clock that the power limit leaves).
template <class E, int D>
__global__ __launch_bounds__(256, D == 96 ? 3 : 2) void k_attn_fwd(AttnK p, int tiles) {
  // Objects of their own, and turns of the loop that name theirs: the compiler then
  // sees that reads of one do not wait for copies into the other.
  using Buf = E[2][KT * D];
  __shared__ __attribute__((aligned(16))) Buf b0, b1;
  __shared__ int2 range[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int once = gridDim.x / p.passes, pass = blockIdx.x / once;
  const Item it = die_item(blockIdx.x % once, p.batch * p.q_heads, tiles, 1, p.causal || p.spans);
  if (it.head < 0) return;
  const int bh = it.head, tile0 = it.tile * 128, b = bh / p.q_heads, head = bh - b * p.q_heads;
  const int kvh = head / p.share, t = tile0 + wave * 32 + (lane & 31);
  bool on = t < p.q_len;
  int2 span = on ? row_span(p, b, t) : make_int2(0, 0);
  if (p.passes == 2) {
    const bool other = apart(span, range, wave, lane);  // every thread: it has a barrier
    on = on && other == (pass == 1);
    if (!on) span = make_int2(0, 0);
    if (__syncthreads_count(on) == 0) return;
  }

  frag<E> q[D / 16];
  {
    const E *row = tok_row<E>(p.q, b, on ? t : 0, head);
#pragma unroll
    for (int k = 0; k < D / 16; k++) {
      const int chunk = 2 * k + (lane >> 5);
      q[k] = row_operand<E>(row, chunk, on && 8 * chunk < p.dim);
    }
  }
  const bool some = span.x < span.y;
  const int lo = __builtin_amdgcn_readfirstlane(wave_min(some ? span.x : INT32_MAX));
  const int hi = __builtin_amdgcn_readfirstlane(wave_max(span.y));
  const int in_lo = __builtin_amdgcn_readfirstlane(wave_max(on ? span.x : 0));
  const int in_hi = __builtin_amdgcn_readfirstlane(wave_min(on ? span.y : INT32_MAX));
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
  Softmax<E, D> sm;
  sm.init(span.x < span.y);
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
  sm.l = other_half(sm.l, false);

  const float l = sm.l, inv = l == 0.0f ? 0.0f : 1.0f / l;
  bool nan = false;
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) {
      sm.o[d][i] *= inv;
      nan |= sm.o[d][i] != sm.o[d][i];
    }
  if (on) {
    E *o = tok_row<E>(p.o, b, t, head);
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = 32 * d + acc_row(i, lane);
        const f32x16 x = sm.o[d];
        if (e < p.dim) store4(o + e, (f32x4){x[i], x[i + 1], x[i + 2], x[i + 3]});
      }
    if (lane < 32)
      p.lse[((int64_t)b * p.q_heads + head) * p.q_len + t] =
          l == 0.0f ? -INFINITY
                    : ((sm.m == -INFINITY ? 0.0f : sm.m) + __builtin_amdgcn_logf(l)) * ATTN_LN2;
  }
  // (with a sum that is NaN all of o is)
  uint64_t again = __builtin_amdgcn_ballot_w64(on && nan && l == l);
  again = (again | again >> 32) & 0xffffffffu;
  if (!again) return;
  const AttnK &c = args_again();
  const int4 see = {lo, hi, in_lo, in_hi};
  if (!keys_spoil<E, KT, is_half<E>>(c, c.v, b, kvh, see, lane)) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the stores above come first
  while (again) {
    const int r = __builtin_ctzll(again);
    again &= again - 1;
    redo_row<E, 8>(c, b, head, tile0 + wave * 32 + r, lane);
  }
}

// ------------------------------------------------------------ few rows
// Single tokens and short queries over long caches: the share x q_len rows that
// read one key head are packed into blocks of 32 (row r is token r / share of
// head r % share), the keys are cut into `splits` parts for as many workgroups,
// and the four waves of a block take every fourth tile of 32 keys of its part,
// each in LDS of its own, without barriers. The block joins its waves; the
// parts' m, l and o go to the workspace in 32 bits and are joined by
// k_attn_join. Bound by the cache's bytes: 4 tokens over 16384 keys each, 16 heads on 2 of
// 128, bf16: 17 us for 67 MB, 3.9 TB/s, and the join 3.9 us.
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
  // (below 2^29: 32-bit divisions)
  const unsigned share = p.share, rows = p.q_len * share, r = rt * 32u + (lane & 31);
  const bool on = r < rows;
  const int t = on ? (int)(r / share) : 0, head = kvh * p.share + (on ? (int)(r % share) : 0);

  frag<E> q[D / 16];
  const E *row = tok_row<E>(p.q, b, t, head);
#pragma unroll
  for (int k = 0; k < D / 16; k++) {
    const int chunk = 2 * k + (lane >> 5);
    q[k] = row_operand<E>(row, chunk, on && 8 * chunk < p.dim);
  }
  int2 span = on ? row_span(p, b, t) : make_int2(0, 0);
  const int p0 = part * p.split_keys, p1 = min(p0 + p.split_keys, p.kv_len);
  const int lo = max(wave_min(span.x < span.y ? span.x : INT32_MAX), p0);
  const int hi = min(wave_max(span.y), p1);
  const int in_lo = wave_max(on ? span.x : 0), in_hi = wave_min(on ? span.y : INT32_MAX);
  span.x = max(span.x, p0);
  span.y = min(span.y, p1);
  if (span.x >= span.y) span = make_int2(0, 0);

  const Stream<E> ks = {tok_row<E>(p.k, b, 0, kvh), p.k.ts, p.kv_len, p.dim};
  const Stream<E> vs = {tok_row<E>(p.v, b, 0, kvh), p.v.ts, p.kv_len, p.dim};
  Softmax<E, D> sm;
  sm.init(span.x < span.y);
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
  sm.l = other_half(sm.l, false);
  if (sm.l == 0.0f) sm.m = -INFINITY;  // a row that sees nothing here has no reference
  if (lane < 32) {
    ml[wave][0][lane] = sm.m;
    ml[wave][1][lane] = sm.l;
  }
  __syncthreads();
  float m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; w++) m = fmaxf(m, ml[w][0][lane & 31]);
  const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
  for (int w = 0; w < 4; w++)
    l += ml[w][1][lane & 31] *
         (ml[w][0][lane & 31] == -INFINITY ? 1.0f
                                           : __builtin_amdgcn_exp2f(ml[w][0][lane & 31] - ref));
  // (a wave without keys has zeros, one with NaN scores alone NaN: both as they are)
  const float mine = sm.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sm.m - ref);
  float *sum = (float *)&b0[0][0][0];  // [32][D + 4]
  for (int w = 0; w < 4; w++) {
    if (w == wave) {
      float *to = sum + (lane & 31) * (D + 4);
#pragma unroll
      for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const f32x16 o = sm.o[d];
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
  const unsigned r2 = min(rt * 32u + rr, rows - 1);
  const bool live = rt * 32u + rr < rows;
  const int t2 = (int)(r2 / share), head2 = kvh * p.share + (int)(r2 % share);
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
  // Rows of this wave, as above.
  uint64_t again = __builtin_amdgcn_ballot_w64(nan && l == l);
  if (!again) return;
  const AttnK &c = args_again();
  const int4 see = {lo, hi, in_lo, in_hi};
  if (!keys_spoil<E, FT, is_half<E>>(c, c.v, b, kvh, see, lane)) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  for (int k = 0; k < 8 && again; k++) {
    if (!(again >> (8 * k) & 0xff)) continue;
    const unsigned r3 = rt * 32u + wave * 8 + k;
    redo_row<E, 8>(c, b, kvh * c.share + (int)(r3 % share), (int)(r3 / share), lane);
  }
}

// Joins the parts of one row: a block a row, 32 lanes with four elements each for
// every eighth part, in one pass (what bounds it is latency: the loads of four parts
// are under way together, and nothing is read first to start them).
template <class E>
__global__ __launch_bounds__(256) void k_attn_join(AttnK p) {
  __shared__ __attribute__((aligned(16))) float sums[8][132];
  const int tid = threadIdx.x, lane = tid & 63, e = 4 * (tid & 31);
  const int64_t all = (int64_t)p.batch * p.q_heads * p.q_len, row = blockIdx.x;
  float m = -INFINITY, l = 0.0f;
  f32x4 o = 0.0f;
  for (int s0 = tid >> 5; s0 < p.splits; s0 += 32) {
    float2 ml[4];
    f32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const bool in = s0 + 8 * i < p.splits;
      const int64_t slot = (in ? s0 + 8 * i : 0) * all + row;
      ml[i] = *(const float2 *)(p.part_ml + 2 * slot);
      x[i] = *(const f32x4 *)(p.part_o + slot * p.dim + (e < p.dim ? e : 0));
      if (!in) ml[i].x = -INFINITY;
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < 4; i++) top = fmaxf(top, ml[i].x);
    const float shrink = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
    l *= shrink;
    o *= shrink;
    m = top;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (s0 + 8 * i >= p.splits) continue;
      // a part without keys holds zeros, one of NaN scores alone NaN: both as they are
      const float w = ml[i].x == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ml[i].x - top);
      l = fmaf(ml[i].y, w, l);
      o += x[i] * w;
    }
  }
  *(f32x4 *)&sums[tid >> 5][e] = o;
  if ((tid & 31) == 0) {
    sums[tid >> 5][128] = l;
    sums[tid >> 5][129] = m;
  }
  __syncthreads();
  if (tid >= 64) return;
  float ref = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; i++) ref = fmaxf(ref, sums[i][129]);
  ref = ref == -INFINITY ? 0.0f : ref;
  l = 0.0f;
  float o0 = 0.0f, o1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float w = sums[i][129] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(sums[i][129] - ref);
    l = fmaf(sums[i][128], w, l);
    o0 = fmaf(sums[i][lane], w, o0);
    o1 = fmaf(sums[i][lane + 64], w, o1);
  }
  const unsigned bh = (unsigned)row / (unsigned)p.q_len;  // (row is below 2^29)
  const int t = (int)((unsigned)row - bh * p.q_len), b = (int)(bh / (unsigned)p.q_heads);
  const int head = (int)(bh - (unsigned)b * p.q_heads);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  E *to = tok_row<E>(p.o, b, t, head);
  if (lane < p.dim) to[lane] = (E)(o0 * inv);
  if (lane + 64 < p.dim) to[lane + 64] = (E)(o1 * inv);
  if (lane == 0)
    p.lse[row] = l == 0.0f ? -INFINITY : (ref + __builtin_amdgcn_logf(l)) * ATTN_LN2;
  if (l != l || !__builtin_amdgcn_ballot_w64(o0 != o0 || o1 != o1)) return;
  // the tokens of this row's block of 32
  const AttnK &c = args_again();
  const int share = c.share, kvh = head / share, r0 = (t * share + head - kvh * share) / 32 * 32;
  const int t0 = r0 / share, n = min((r0 + 31) / share, c.q_len - 1) - t0 + 1;
  if (!keys_spoil<E, FT, is_half<E>>(c, c.v, b, kvh, rows_see(c, b, t0, n, lane), lane)) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
  redo_row<E, 4>(c, b, head, t, lane);
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
  const int blocks = die_blocks(p.batch * p.q_heads, tiles, 1) * p.passes;
  if (D == 128 && p.dim <= 96) k_attn_fwd<E, 96><<<blocks, 256, 0, st>>>(p, tiles);
  else k_attn_fwd<E, D><<<blocks, 256, 0, st>>>(p, tiles);
  return hipGetLastError();
}

}  // namespace

// The split of the keys that a call takes, 0: the form for many rows.
//   few rows: no more than 32 rows read a key head (one block of rows), or the blocks
//   of 32 rows are no more than run at once (by their LDS, one on each of 256 compute
//   units for heads above 64, else two), or twice that where a mask makes them uneven.
// Measured, few and many, 8 heads: 2048 tokens, heads of 64 (512 blocks) 24 and 34 us,
// 3000 tokens (752) 51 and 48, 3000 causal 37 and 46; 1024 tokens, heads of 128 (256) 17
// and 26, 1536 (384) 38 and 36, 2048 causal (512) 38 and 44, 3000 causal (752) 66 and 61.
void gs_attn_plan(AttnK *p) {
  const int64_t rows = (int64_t)p->q_len * p->share, row_tiles = (rows + 31) / 32;
  const int64_t blocks = (int64_t)p->batch * p->kv_heads * row_tiles;
  const int64_t room = p->dim <= 64 ? 512 : 256;
  p->splits = 0;
  p->split_keys = 0;
  if (!blocks || (rows > 32 && blocks > (p->causal || p->spans ? 2 : 1) * room)) return;
  // Parts: one round of workgroups, none with fewer than 256 keys, and where they cost
  // less than they save. Joining them takes as long as a workgroup's 600 keys, and a
  // row's part as long as 1/16 key (about 5.5 ns a key with heads of 64, 7.6 with 128).
  // Measured, 8 heads of 64: 1 token, 512 keys 8.3 us whole and 9.3 in two parts, 1024
  // keys 11.1 whole and 9.4 in four, 2048 keys 9.6 in eight; 64 tokens, 1024 keys 11.2
  // and 9.8 in four; 512 tokens, 1024 keys 11.6 and 15.2 in four.
  const int64_t all = (int64_t)p->batch * p->q_heads * p->q_len;
  int64_t splits = blocks < room ? room / blocks : 1;
  const int64_t most = p->kv_len / 256, even = (int64_t)sqrt(16.0 * p->kv_len / all);
  splits = splits < most ? splits : most;
  splits = splits < even ? splits : even;
  if (splits < 2 || p->kv_len / splits + 600 + all * splits / 16 >= p->kv_len) splits = 1;
  const int64_t keys = ((p->kv_len + splits - 1) / splits + FT - 1) / FT * FT;
  p->split_keys = (int)(keys ? keys : FT);
  p->splits = (int)(p->kv_len ? (p->kv_len + p->split_keys - 1) / p->split_keys : 1);
}

// Whether blocks of 128 rows are launched twice: with spans, unless there are so many
// of them that one with two sequences' keys is hidden among the others. Measured, 6037
// tokens in four sequences, 12 heads of 80 (576 blocks): 71 us with one pass, 55 with
// two; where no block has rows of two, 51 and 52.
int gs_attn_passes(const AttnK &p) {
  return p.spans && (int64_t)p.batch * p.q_heads * ((p.q_len + 127) / 128) < 4096 ? 2 : 1;
}

hipError_t gs_launch_attn_fwd(AttnK p, int dtype, hipStream_t st) {
  p.passes = gs_attn_passes(p);
  if (dtype == GS_BF16) return p.dim <= 64 ? launch<bf16_t, 64>(p, st) : launch<bf16_t, 128>(p, st);
  return p.dim <= 64 ? launch<f16_t, 64>(p, st) : launch<f16_t, 128>(p, st);
}
