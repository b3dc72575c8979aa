// The gradient of attention, with the probabilities computed again from the
// row sums that the forward left: p_ij = exp(s_ij - lse_i),
//   D_i = do_i . o_i, dv_j = sum_i p_ij do_i, ds_ij = p_ij (do_i . v_j - D_i),
//   dq_i = scale sum_j ds_ij k_j, dk_j = scale sum_i ds_ij q_i,
// the sums over i also over the heads that share key j.
//
// The launches: D (and what the others need to skip tiles), then dK and dV by
// blocks that own keys and stream queries, then dQ by blocks that own queries and
// stream keys, then the sums of what was computed in parts. The scores are computed
// in both (7 products of the size of q . k^T instead of 5): in exchange no sum is made
// by atomics, so results do not depend on timing, and nothing of size q_len x kv_len
// is ever stored.
//
// p and ds are rounded to the inputs' 16-bit type for the products: against 64 bits dv's
// error is 1.3 to 1.43 times that of rounding the results alone, dq's and dk's 1.4 to 1.55,
// and up to 1.67 where rows see a few dozen keys (D, below). Probabilities
// of long rows fall below the normal range of fp16 (2^-14), so for fp16 the
// kernels work on p 2^15 and on ds 2^e, powers of two that are taken out of the 32-bit
// sums. e is each key's own in dK and each query's in dQ, and falls as the largest |ds| of
// the pairs that are seen does not fit: what masked pairs hold, and the gradients of other
// sequences in a row, do not matter. (8192 tokens, fp16, forward and backward, against e from
// a bound of all |do| |v| + |D|: 8 heads of 64 745 us for 721, of 128 on 2 1217 for 1205.)
#include "attention_common.h"

namespace {

constexpr int WALK = 4096;  // streamed query tiles whose masks a block holds at a time

// The powers of two that ds 2^e starts with: more than any result of fp16 shows, and far
// from 2^128 where ds is largest (|do . v| and |D| are below 2^40).
constexpr int DS_POWERS = 60;

// The powers of two that ds 2^e of a lane's own row has too many where its largest
// magnitude is `top` (both halves' lanes of the row together): then 2^10 is left, which
// keeps 2^24 below it in fp16's normal numbers, and later ones may be 32 times as large.
__device__ __forceinline__ int too_many(float top) {
  top = other_half(top, true);
  return top >= 32768.0f && top <= 3e38f ? ilogbf(top) - 10 : 0;
}

// ------------------------------------------------------------ rows done again

template <class E, int N>
__device__ __forceinline__ void redo_query(const AttnK &p, int b, int head, int t, int lane) {
  const int2 span = row_span(p, b, t);
  const int kvh = head / p.share;
  const int64_t bh = (int64_t)b * p.q_heads + head;
  const E *q = tok_row<E>(p.q, b, t, head), *g = tok_row<E>(p.d_o, b, t, head);
  const float lse = p.lse[bh * p.q_len + t] * ATTN_LOG2E, delta = -p.row_delta[bh * p.q_pad + t];
  RowSum<N> dq;
  bool open = true;
#pragma unroll 1
  for (int j0 = span.x; open && j0 < span.y; j0 += 64) {
    const int n = min(64, span.y - j0);
    float ds = 0.0f;
    if (lane < n) {
      const float s = dot_row<4>(q, tok_row<E>(p.k, b, j0 + lane, kvh), p.dim) * p.scale_log2;
      ds = __builtin_amdgcn_exp2f(s - lse) *
           (dot_row<4>(g, tok_row<E>(p.v, b, j0 + lane, kvh), p.dim) - delta);
    }
    open = dq.template add<E>(ds, first_bits(n), p.k, b, kvh, j0, span.y - 1, p.dim, lane);
  }
  dq.store(tok_row<E>(p.dq, b, t, head), p.scale, p.dim, lane);
}

// One key's row of dV, or of dK.
template <class E, int N>
__device__ __forceinline__ void redo_key(const AttnK &p, int b, int kvh, int key, bool of_v, int lane) {
  const E *k = tok_row<E>(p.k, b, key, kvh), *v = tok_row<E>(p.v, b, key, kvh);
  const TokK x = of_v ? p.d_o : p.q;
  RowSum<N> sum;
  bool open = true;
#pragma unroll 1
  for (int head = kvh * p.share; head < (kvh + 1) * p.share; head++)
#pragma unroll 1
    for (int t0 = 0; open && t0 < p.q_len; t0 += 64) {
      const int t = t0 + lane;
      const int2 span = t < p.q_len ? row_span(p, b, t) : make_int2(0, 0);
      const bool in = key >= span.x && key < span.y;
      const uint64_t seen = __builtin_amdgcn_ballot_w64(in);
      if (!seen) continue;
      float w = 0.0f;
      if (in) {
        const int64_t bh = (int64_t)b * p.q_heads + head;
        const float s = dot_row<4>(tok_row<E>(p.q, b, t, head), k, p.dim) * p.scale_log2;
        w = __builtin_amdgcn_exp2f(s - p.lse[bh * p.q_len + t] * ATTN_LOG2E);
        if (!of_v)
          w *= dot_row<4>(tok_row<E>(p.d_o, b, t, head), v, p.dim) + p.row_delta[bh * p.q_pad + t];
      }
      open = sum.template add<E>(w, seen, x, b, head, t0, p.q_len - 1, p.dim, lane);
    }
  sum.store(tok_row<E>(of_v ? p.dv : p.dk, b, key, kvh), of_v ? 1.0f : p.scale, p.dim, lane);
}

// Whether the output gradients (for dV; else the queries) hold a row that spoils among those
// of the tiles that the block of 128 keys from `block` on was multiplied with and that do not
// see all of the n keys from `key` on; for dV in fp16 also among those that do.
template <class E>
__device__ __forceinline__ bool queries_spoil(const AttnK &p, int b, int kvh, int block, int key,
                                              int n, bool of_v, int lane) {
  const bool all = is_half<E> && of_v;
  const TokK x = of_v ? p.d_o : p.q;
  if (!p.tile_spans && !all) return false;
  const int q_tiles = p.q_pad / KT, key_end = min(key + n, p.kv_len);
#pragma unroll 1
  for (int i0 = 0; i0 < q_tiles; i0 += 64) {
    bool at = i0 + lane < q_tiles;
    if (at && p.tile_spans) {
      const int4 r = p.tile_spans[(int64_t)b * q_tiles + i0 + lane];
      at = r.x < block + 128 && r.y > block && (all || r.z > key || r.w < key_end);
    }
    for (uint64_t todo = __builtin_amdgcn_ballot_w64(at); todo; todo &= todo - 1) {
      const int t = (i0 + __builtin_ctzll(todo)) * KT + lane;
      const bool on = t < p.q_len;
      const int2 s = on ? row_span(p, b, t) : make_int2(0, 0);
      const bool seen = s.x <= key && s.y >= key_end;
#pragma unroll 1
      for (int head = kvh * p.share; head < (kvh + 1) * p.share; head++) {
        const bool bad = on && (all || !seen) && row_spoils(tok_row<E>(x, b, t, head), p.dim, seen);
        if (__builtin_amdgcn_ballot_w64(bad)) return true;
      }
    }
  }
  return false;
}

// ------------------------------------------------------------ preparation
// The rows' values as dK and dV start from them, in whole tiles (rows past the end
// and rows that see nothing: -inf, which gives p = 0); with masks the rows' spans, and
// for each 64 queries the keys that some row sees and that all see (lo, hi, in_lo,
// in_hi). 16 lanes a row, 8 of up to 64 elements. Bound by its bytes: 2 x 4096 queries, 16
// heads of 128, bf16, 67 MB: 13 us, and 4 for the rows of few keys below.
//
// o was rounded to 16 bits, and D_i of it is off by as much. Beside gradients of many
// keys that is little, but rows of a few have the largest ones: their D_i are summed
// from their pairs, sum_j p_ij (do_i . v_j). Relative error of dq, causal, bf16, 64
// queries: 0.0030 with o alone, 0.0025 so (0.0023 with exact D_i: ds in 16 bits). Of 16
// keys it is 0.0024 and costs twice as much: 8 us instead of 4 of 4096 causal queries'
// 720, a chain of loads that the few blocks with such rows wait for.
constexpr int D_PAIRS = 8;

template <class E, int LANES>
__device__ __forceinline__ float pairs_d(const AttnK &p, int b, int head, int t, int2 see,
                                         int j) {
  const int kvh = head / p.share;
  const float lse = p.lse[((int64_t)b * p.q_heads + head) * p.q_len + t] * ATTN_LOG2E;
  const bool in = 8 * j < p.dim;
  const int at = in ? 8 * j : 0;
  const E *q = tok_row<E>(p.q, b, t, head) + at, *g = tok_row<E>(p.d_o, b, t, head) + at;
  const frag<E> fq = *(const frag<E> *)q, fg = *(const frag<E> *)g;
  float d = 0.0f;
  for (int key = see.x; key < see.y; key++) {
    const frag<E> k = *(const frag<E> *)(tok_row<E>(p.k, b, key, kvh) + at);
    const frag<E> v = *(const frag<E> *)(tok_row<E>(p.v, b, key, kvh) + at);
    float s = 0.0f, dp = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      s = fmaf((float)fq[e], (float)k[e], s);
      dp = fmaf((float)fg[e], (float)v[e], dp);
    }
    s = group_sum(in ? s : 0.0f, LANES) * p.scale_log2 - lse;
    d = fmaf(__builtin_amdgcn_exp2f(s), group_sum(in ? dp : 0.0f, LANES), d);
  }
  return d;
}

template <class E, int LANES>
__global__ __launch_bounds__(256) void k_attn_prep(AttnK p, int q_tiles) {
  const int tid = threadIdx.x, lane = tid & 63, j = tid & (LANES - 1);
  constexpr int AT_ONCE = 256 / LANES;  // rows
  const int bh = blockIdx.x / q_tiles, qt = blockIdx.x - bh * q_tiles;
  const int b = bh / p.q_heads, head = bh - b * p.q_heads;
  if (p.tile_spans && head == 0 && tid < 64) {
    const int t = qt * KT + lane;
    const int2 s = t < p.q_len ? row_span(p, b, t) : make_int2(0, 0);
    const bool on = t < p.q_len, some = s.x < s.y;
    const int4 r = {wave_min(some ? s.x : INT32_MAX), wave_max(s.y), wave_max(on ? s.x : 0),
                    wave_min(on ? s.y : INT32_MAX)};
    if (lane == 0) p.tile_spans[(int64_t)b * q_tiles + qt] = r;
    p.row_spans[(int64_t)b * p.q_pad + t] = s;
  }
  int few = 0;
#pragma unroll
  for (int i = 0; i < KT / AT_ONCE; i++) {
    const int t = qt * KT + AT_ONCE * i + tid / LANES;
    float d = 0.0f;
    if (t < p.q_len && 8 * j < p.dim) {
      const E *g = tok_row<E>(p.d_o, b, t, head) + 8 * j;
      const E *o = tok_row<E>(p.o, b, t, head) + 8 * j;
      const f32x4 g0 = load4(g), g1 = load4(g + 4), o0 = load4(o), o1 = load4(o + 4);
#pragma unroll
      for (int e = 0; e < 4; e++) d = fmaf(g0[e], o0[e], fmaf(g1[e], o1[e], d));
    }
    d = group_sum(d, LANES);
    const float lse = t < p.q_len ? p.lse[(int64_t)bh * p.q_len + t] : -INFINITY;
    const int2 see = t < p.q_len ? row_span(p, b, t) : make_int2(0, 0);
    const bool pairs = see.x < see.y && see.y - see.x <= D_PAIRS;
    few |= (int)pairs << i;
    if (j == 0) {
      const int64_t at = (int64_t)bh * p.q_pad + t;
      if (!pairs) p.row_delta[at] = -d;
      p.row_lse[at] = lse == -INFINITY
                          ? -INFINITY
                          : ((is_half<E> ? 15.0f * ATTN_LN2 : 0.0f) - lse) / p.scale;
    }
  }
  // a loop of its own, not unrolled: registers for one row's pairs, not for four
#pragma unroll 1
  for (int i = 0; i < KT / AT_ONCE; i++) {
    if (!(few >> i & 1)) continue;
    const int t = qt * KT + AT_ONCE * i + tid / LANES;
    const float d = pairs_d<E, LANES>(p, b, head, t, row_span(p, b, t), j);
    if (j == 0) p.row_delta[(int64_t)bh * p.q_pad + t] = -d;
  }
}

// Stores a transposed accumulator (lane: a row, registers: its elements) and
// returns the rows (bits 0..31) that hold a NaN.
template <class E, int D>
__device__ __forceinline__ uint32_t store_rows(const f32x16 (&acc)[D / 32], float by, E *row,
                                               bool on, int dim, int lane) {
  bool nan = false;
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) nan |= acc[d][i] != acc[d][i];
  const uint64_t bits = __builtin_amdgcn_ballot_w64(on && nan);
  if (on) {
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = 32 * d + acc_row(i, lane);
        const f32x16 x = acc[d];
        if (e < dim) store4(row + e, (f32x4){x[i] * by, x[i + 1] * by, x[i + 2] * by, x[i + 3] * by});
      }
  }
  return (uint32_t)bits | (uint32_t)(bits >> 32);
}

// The same into one part's 32-bit sums, which k_attn_sum adds and looks over.
template <int D>
__device__ __forceinline__ void store_part(const f32x16 (&acc)[D / 32], float by, float *row,
                                           bool on, int dim, int lane) {
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int e = 32 * d + acc_row(i, lane);
      const f32x16 x = acc[d];
      if (on && e < dim) *(f32x4 *)(row + e) = (f32x4){x[i], x[i + 1], x[i + 2], x[i + 3]} * by;
    }
}

// ------------------------------------------------------------ dK and dV
// A block of eight waves owns 128 keys of one key head and streams the queries that
// see them in tiles of 64, head after head of those that share the key head: wave w
// takes keys 32 (w % 4) .. + 31 and rows 32 (w / 4) .. + 31 of every tile, so that
// each SIMD has two waves whose matrix and vector work overlap. K and V stay in LDS
// (beside dK and dV a wave's 256 registers have no room for them). Where there are too
// few such blocks, or masks make them uneven, a block takes one of kv_parts equal runs
// of those tiles, and k_attn_sum adds the parts' 32-bit sums. -lse / scale and -D_i are
// the accumulators' starting values. Bound by the matrix units: 16384 tokens, 8 heads of
// 128 on 2, bf16: 1930 us, 1140 TFLOP/s of its four products (four waves a block, 32
// keys each and all rows, took 18% longer).
template <class E, int D>
__global__ __launch_bounds__(512, 2) void k_attn_bwd_kv(AttnK p, int tiles, int q_tiles) {
  // Objects of their own, and turns of the loop that name theirs: the compiler then
  // sees that reads of one do not wait for copies into another.
  using Buf = E[2][KT * D];
  __shared__ __attribute__((aligned(16))) Buf b0, b1;
  __shared__ __attribute__((aligned(16))) E own[2][128 * D];  // keys, values; then sums
  __shared__ __attribute__((aligned(16))) float stat[2][2][KT];
  __shared__ __attribute__((aligned(16))) int2 spans[2][KT];
  __shared__ uint64_t active[WALK / 64], partly[WALK / 64];
  __shared__ uint16_t list[WALK];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = wave >> 2;
  const bool uneven = p.causal || p.spans;
  const Item it = die_item(blockIdx.x, p.batch * p.kv_heads, tiles, p.kv_parts, uneven);
  if (it.head < 0) return;
  const int piece = it.part, bh = it.head, b = bh / p.kv_heads, kvh = bh - b * p.kv_heads;
  // (causal: the first keys are seen by the most queries)
  const int key0 = (uneven ? tiles - 1 - it.tile : it.tile) * 128, mine0 = key0 + 32 * (wave & 3);
  const int key = mine0 + (lane & 31);
  const bool on = key < p.kv_len;

  {
    const Stream<E> ks = {tok_row<E>(p.k, b, 0, kvh), p.k.ts, p.kv_len, p.dim};
    const Stream<E> vs = {tok_row<E>(p.v, b, 0, kvh), p.v.ts, p.kv_len, p.dim};
#pragma unroll
    for (int i = 0; i < 128; i += 64) {
      Copy<E, D, 512, 64>::issue(ks, key0 + i, own[0] + i * D, tid);
      Copy<E, D, 512, 64>::issue(vs, key0 + i, own[1] + i * D, tid);
    }
  }
  // The masks of the first tiles are on their way with them; nothing waits before the
  // first tile is sent for too.
  int4 early = {0, 0, 0, 0};
  if (p.tile_spans && tid < q_tiles) early = p.tile_spans[(int64_t)b * q_tiles + tid];
  int e = is_half<E> ? DS_POWERS : 0;  // of ds of the lane's key, whose p has 15 already
  float ds_by = ldexpf(1.0f, e - 15);

  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; d++) dk[d] = dv[d] = 0.0f;

  for (int walk0 = 0; walk0 < q_tiles; walk0 += WALK) {
    // The list of those of the next WALK tiles that see a key of this block; bit 15:
    // not all of its keys with all of their rows.
    const int n = min(q_tiles - walk0, WALK), words = (n + 63) >> 6;
    __syncthreads();
    for (int i = tid; i < words * 64; i += 512) {
      bool act = i < n, part = false;
      if (act && p.tile_spans) {
        const int4 r = walk0 + i == tid ? early : p.tile_spans[(int64_t)b * q_tiles + walk0 + i];
        act = r.x < key0 + 128 && r.y > key0;
        part = r.z > key0 || r.w < min(key0 + 128, p.kv_len);
      }
      const uint64_t a = __builtin_amdgcn_ballot_w64(act), c = __builtin_amdgcn_ballot_w64(part);
      if (lane == 0) {
        active[i >> 6] = a;
        partly[i >> 6] = c;
      }
    }
    __syncthreads();
    int count = 0;
    for (int w = 0; w < words; w++) {
      const uint64_t a = active[w];
      if ((w & 7) == wave && a >> lane & 1)
        list[count + __builtin_popcountll(a & ((1ull << lane) - 1))] =
            (uint16_t)(64 * w + lane + (partly[w] >> lane & 1 ? 0x8000 : 0));
      count += __builtin_popcountll(a);
    }
    count = __builtin_amdgcn_readfirstlane(count);
    __syncthreads();
    // This block's run of the (head, tile) pairs: `left` of them from list[at] of
    // head `head` on.
    const int64_t pairs = (int64_t)count * p.share;
    const int64_t from = pairs * piece / p.kv_parts;
    int left = (int)(pairs * (piece + 1) / p.kv_parts - from);
    if (left == 0) continue;
    int head = kvh * p.share + (int)(from / count), at = (int)(from % count);
    auto tile_at = [&](int i) { return (int)__builtin_amdgcn_readfirstlane(list[i]); };

    // Queries, output gradients and row values of tile `t` of head `head`.
    using Tile = Copy<E, D, 512, KT, true>;
    auto load = [&](int t, Buf &to, int in) {
      const int t0 = (walk0 + (t & 0x7fff)) * KT;
      Tile::issue({tok_row<E>(p.q, b, 0, head), p.q.ts, p.q_len, p.dim}, t0, to[0], tid);
      Tile::issue({tok_row<E>(p.d_o, b, 0, head), p.d_o.ts, p.q_len, p.dim}, t0, to[1], tid);
      const int64_t at = ((int64_t)b * p.q_heads + head) * p.q_pad + t0;
      // (constant places: of one that depends on the wave the compiler would not see
      // that it is none of the tiles')
      if (wave == 0) copy_words(p.row_lse + at, stat[in][0], lane);
      if (wave == 1) copy_words(p.row_delta + at, stat[in][1], lane);
      if (wave < 4 || !p.tile_spans) return;
      const int *spans_at = (const int *)(p.row_spans + (int64_t)b * p.q_pad + t0);
      if (wave == 4) copy_words(spans_at, (int *)spans[in], lane);
      if (wave == 5) copy_words(spans_at + 64, (int *)spans[in] + 64, lane);
    };
    // Steps to the tile after `next`, which is read from the list a turn before it is
    // needed.
    auto step = [&]() {
      if (++at == count) {
        at = 0;
        head++;
      }
    };
    int now = tile_at(at);
    load(now, b0, 0);
    step();
    int next = tile_at(at);
    // One tile, in buffer `here`; the next one is sent for into `there`.
    auto turn = [&](Buf &here, Buf &there, int in) {
      block_copied();  // this tile is there, and nobody reads the other one any more
      const bool part = now & 0x8000;
      const E *q = here[0], *g = here[1];
      const int z = opaque_zero() + 32 * (wave & 3) * D;
      // The operands of step k of both products, AHEAD steps before they are used.
      constexpr int STEPS = D / 16, AHEAD = D == 64 ? 2 : 1;
      frag<E> x[4][STEPS];
      auto read = [&](int k) {
        x[0][k] = lds_rows<E, D>(q, 32 * half, k, lane);
        x[1][k] = lds_rows<E, D>(own[0] + z, 0, k, lane);
        x[2][k] = lds_rows<E, D>(g, 32 * half, k, lane);
        x[3][k] = lds_rows<E, D>(own[1] + z, 0, k, lane);
      };
      f32x16 w, ds;
#pragma unroll
      for (int k = 0; k < AHEAD; k++) read(k);
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int r = 32 * half + acc_row(i, lane);
        const f32x4 l4 = *(const f32x4 *)&stat[in][0][r];
        const f32x4 d4 = *(const f32x4 *)&stat[in][1][r];
#pragma unroll
        for (int c = 0; c < 4; c++) {
          w[i + c] = l4[c];
          ds[i + c] = d4[c];
        }
      }
      left--;
      now = next;
      if (left > 0) {
        load(now, there, in ^ 1);
        step();
        next = tile_at(at);
      }
#pragma unroll
      for (int k = 0; k < STEPS; k++) {
        __builtin_amdgcn_sched_barrier(0);
        if (k + AHEAD < STEPS) read(k + AHEAD);
        w = mfma(x[0][k], x[1][k], w);
        ds = mfma(x[2][k], x[3][k], ds);
      }
      frag<E> cols[2][D / 32];  // of dO, on their way while the vector unit works
#pragma unroll
      for (int d = 0; d < D / 32; d++) cols[0][d] = lds_cols<E, D, KT>(g, 32 * half, d, lane);
      __builtin_amdgcn_sched_barrier(0);
      if (part) {
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const int2 r = spans[in][32 * half + acc_row(i, lane)];
          if ((unsigned)(key - r.x) >= (unsigned)(r.y - r.x)) {
            w[i] = -INFINITY;
            ds[i] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 16; i++) {
        w[i] = __builtin_amdgcn_exp2f(w[i] * p.scale_log2);
        ds[i] *= w[i];
        if (is_half<E>) ds[i] *= ds_by;
      }
      if (is_half<E>) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(ds[i]));
        if (__builtin_amdgcn_ballot_w64(top >= 32768.0f)) {
          const int down = too_many(top);
          const float by = ldexpf(1.0f, -down);
          e -= down;
          ds_by *= by;
          ds *= by;
#pragma unroll
          for (int d = 0; d < D / 32; d++) dk[d] *= by;
        }
      }
      frag<E> pw[2], pd[2];
#pragma unroll
      for (int k = 0; k < 2; k++) {
        pw[k] = pack8<E>(w, k);
        pd[k] = pack8<E>(ds, k);
      }
      __builtin_amdgcn_sched_barrier(0);
      // Groups of D / 32 transposed operands: dO and Q for the first 16 rows, then for
      // the others, each read while the one before it is used.
#pragma unroll
      for (int c = 0; c < 4; c++) {
        if (c < 3)
#pragma unroll
          for (int d = 0; d < D / 32; d++)
            cols[(c + 1) & 1][d] =
                lds_cols<E, D, KT>(c & 1 ? g : q, 32 * half + (c ? 16 : 0), d, lane);
#pragma unroll
        for (int d = 0; d < D / 32; d++) {
          if (c & 1) dk[d] = mfma(cols[1][d], pd[c >> 1], dk[d]);
          else dv[d] = mfma(cols[0][d], pw[c >> 1], dv[d]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    while (left > 0) {
      turn(b0, b1, 0);
      if (left > 0) turn(b1, b0, 1);
    }
  }
  copied<0>();
  if (is_half<E>) {  // the halves have powers of their own
    const float by = ldexpf(1.0f, -e);
#pragma unroll
    for (int d = 0; d < D / 32; d++) dk[d] *= by;
  }

  // The two halves' sums, W columns at a time through LDS: the upper waves' dK goes to
  // the lower ones, whose dV goes to the upper ones. Chunk c of row r is at c ^ r.
  constexpr int W = D / 2;
  const int last = lane + opaque_zero();  // places that take no registers before here
  const int row = 32 * (wave & 3) + (last & 31);
  float *sums = (float *)own[0] + row * W;  // [2][128][W]
  static_assert(2 * 128 * W * sizeof(float) <= sizeof(own), "the sums fit");
  auto place = [&](int d, int i) { return ((8 * d + acc_row(i, last) / 4) ^ (row & (W / 4 - 1))) * 4; };
  auto put = [&](const f32x16 (&from)[D / 32], int h, float *to) {
#pragma unroll
    for (int d = 0; d < D / 64; d++)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x16 x = from[h * (D / 64) + d];
        *(f32x4 *)(to + place(d, i)) = (f32x4){x[i], x[i + 1], x[i + 2], x[i + 3]};
      }
  };
  auto add = [&](f32x16 (&to)[D / 32], int h, const float *from) {
#pragma unroll
    for (int d = 0; d < D / 64; d++)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 y = *(const f32x4 *)(from + place(d, i));
#pragma unroll
        for (int c = 0; c < 4; c++) to[h * (D / 64) + d][i + c] += y[c];
      }
  };
#pragma unroll
  for (int h = 0; h < 2; h++) {
    __syncthreads();
    if (half) put(dk, h, sums);
    else put(dv, h, sums + 128 * W);
    __syncthreads();
    if (half) add(dv, h, sums + 128 * W);
    else add(dk, h, sums);
  }

  const int64_t rows = (int64_t)p.batch * p.kv_heads * p.kv_len;
  const int64_t at = (piece * rows + (int64_t)bh * p.kv_len + key) * p.dim;
  uint32_t again;
  if (half) {
    const float by = is_half<E> ? 0x1p-15f : 1.0f;
    if (p.kv_parts > 1) return store_part<D>(dv, by, p.part_v + at, on, p.dim, lane);
    again = store_rows<E, D>(dv, by, tok_row<E>(p.dv, b, on ? key : 0, kvh), on, p.dim, lane);
  } else {
    if (p.kv_parts > 1) return store_part<D>(dk, p.scale, p.part_k + at, on, p.dim, lane);
    again = store_rows<E, D>(dk, p.scale, tok_row<E>(p.dk, b, on ? key : 0, kvh), on, p.dim, lane);
  }
  if (!again) return;
  const AttnK &c = args_again();
  if (!queries_spoil<E>(c, b, kvh, key0, mine0, 32, half, lane)) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the stores above come first
  while (again) {
    const int r = __builtin_ctz(again);
    again &= again - 1;
    redo_key<E, 8>(c, b, kvh, mine0 + r, half, lane);
  }
}

// ------------------------------------------------------------ dQ
// The forward's walk with a second score product and without a running maximum; a
// block takes one of q_parts runs of its key tiles, as above. Bound by the matrix
// units' rate at the clock that their power leaves: 16384 tokens, 8 heads of 128, bf16:
// 1350 us, 1220 TFLOP/s of its three products. Heads of 65 to 96 have a form of 96 (2 x 2048 queries,
// 12 heads of 80, bf16: 74 us, in the form of 128 90).
template <class E, int D>
__global__ __launch_bounds__(256, 2) void k_attn_bwd_q(AttnK p, int tiles) {
  using Buf = E[2][KT * D];
  __shared__ __attribute__((aligned(16))) Buf b0, b1;
  __shared__ int2 range[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int once = gridDim.x / p.passes, pass = blockIdx.x / once;
  const Item it = die_item(blockIdx.x % once, p.batch * p.q_heads, tiles, p.q_parts,
                           p.causal || p.spans);
  if (it.head < 0) return;
  const int piece = it.part;
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

  const float row_lse = on ? p.lse[(int64_t)bh * p.q_len + t] : -INFINITY;
  const float delta = on ? -p.row_delta[(int64_t)bh * p.q_pad + t] : 0.0f;
  frag<E> q[D / 16], g[D / 16];
  const E *qr = tok_row<E>(p.q, b, on ? t : 0, head), *gr = tok_row<E>(p.d_o, b, on ? t : 0, head);
#pragma unroll
  for (int k = 0; k < D / 16; k++) {
    const int chunk = 2 * k + (lane >> 5);
    q[k] = row_operand<E>(qr, chunk, on && 8 * chunk < p.dim);
    g[k] = row_operand<E>(gr, chunk, on && 8 * chunk < p.dim);
  }
  int e = is_half<E> ? DS_POWERS : 0;  // of ds of the lane's query
  float lse = row_lse == -INFINITY ? INFINITY : row_lse * ATTN_LOG2E - (float)e;
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
  if (p.q_parts > 1) {
    const int n = end > first ? end - first : 0;
    end = first + (int)((int64_t)n * (piece + 1) / p.q_parts);
    first += (int)((int64_t)n * piece / p.q_parts);
  }

  const Stream<E> ks = {tok_row<E>(p.k, b, 0, kvh), p.k.ts, p.kv_len, p.dim};
  const Stream<E> vs = {tok_row<E>(p.v, b, 0, kvh), p.v.ts, p.kv_len, p.dim};
  f32x16 dq[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; d++) dq[d] = 0.0f;
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
    if (key0 >= hi || key0 + KT <= lo) return;
    const bool full = key0 >= in_lo && key0 + KT <= in_hi;
    const E *kt = here[0], *vt = here[1];
#pragma unroll
    for (int s = 0; s < KT / 32; s++) {
      // The first product's operands are read together; the second one's arrive under
      // it. Reads of both a few steps ahead of each use measured the same with heads of
      // 64, and spill with heads of 128.
      constexpr int STEPS = D / 16;
      frag<E> a[STEPS];
#pragma unroll
      for (int k = 0; k < STEPS; k++) a[k] = lds_rows<E, D>(kt, 32 * s, k, lane);
      __builtin_amdgcn_sched_barrier(0);
      f32x16 w = 0.0f, ds = 0.0f;
#pragma unroll
      for (int k = 0; k < STEPS; k++) w = mfma(a[k], q[k], w);
#pragma unroll
      for (int k = 0; k < STEPS; k++) ds = mfma(lds_rows<E, D>(vt, 32 * s, k, lane), g[k], ds);
      frag<E> cols[2][D / 32];  // on their way while the vector unit works
#pragma unroll
      for (int k = 0; k < 2; k++)
#pragma unroll
        for (int d = 0; d < D / 32; d++) cols[k][d] = lds_cols<E, D>(kt, 32 * s + 16 * k, d, lane);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 16; i++)
        ds[i] = __builtin_amdgcn_exp2f(fmaf(w[i], p.scale_log2, -lse)) * (ds[i] - delta);
      if (!full) {
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const int key = key0 + 32 * s + acc_row(i, lane);
          if ((unsigned)(key - span.x) >= (unsigned)(span.y - span.x)) ds[i] = 0.0f;
        }
      }
      if (is_half<E>) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(ds[i]));
        if (__builtin_amdgcn_ballot_w64(top >= 32768.0f)) {
          const int down = too_many(top);
          const float by = ldexpf(1.0f, -down);
          e -= down;
          lse += (float)down;
          ds *= by;
#pragma unroll
          for (int d = 0; d < D / 32; d++) dq[d] *= by;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; k++) {
        const frag<E> pd = pack8<E>(ds, k);
#pragma unroll
        for (int d = 0; d < D / 32; d++) dq[d] = mfma(cols[k][d], pd, dq[d]);
      }
    }
  };
  for (int j = first; j < end; j += 2) {
    turn(j, b0, b1);
    if (j + 1 < end) turn(j + 1, b1, b0);
  }

  const float by = is_half<E> ? ldexpf(p.scale, -e) : p.scale;
  if (p.q_parts > 1) {
    const int64_t rows = (int64_t)p.batch * p.q_heads * p.q_len;
    store_part<D>(dq, by, p.part_q + (piece * rows + (int64_t)bh * p.q_len + t) * p.dim, on, p.dim,
                  lane);
    return;
  }
  uint32_t again =
      store_rows<E, D>(dq, by, tok_row<E>(p.dq, b, on ? t : 0, head), on, p.dim, lane);
  // (with a log sum or a D that is NaN all of dq is, of a query that sees any key)
  again &= ~(uint32_t)__builtin_amdgcn_ballot_w64(some && (lse != lse || delta != delta));
  if (!again) return;
  const AttnK &c = args_again();
  const int4 see = {lo, hi, in_lo, in_hi};
  if (!keys_spoil<E, KT, false>(c, c.k, b, kvh, see, lane)) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the stores above come first
  while (again) {
    const int r = __builtin_ctz(again);
    again &= again - 1;
    redo_query<E, 8>(c, b, head, tile0 + wave * 32 + r, lane);
  }
}

// ------------------------------------------------------------ the parts' sums
// 32 lanes a row (16 of up to 64 elements), in the order of the parts: rows of dQ (KEYS 0), or of dK and dV. Bound
// by its bytes: 2 x 4096 keys, 4 heads of 128, two parts, 84 MB: 14 us.
template <class E, bool KEYS, int LANES>
__device__ __forceinline__ void sum_rows(const AttnK &p, int block) {
  const int lane = threadIdx.x & 63, e = 4 * (lane & (LANES - 1));
  const int len = KEYS ? p.kv_len : p.q_len, heads = KEYS ? p.kv_heads : p.q_heads;
  const int parts = KEYS ? p.kv_parts : p.q_parts;
  const int64_t rows = (int64_t)p.batch * heads * len;
  const int64_t row = (int64_t)block * (256 / LANES) + threadIdx.x / LANES;
  const bool on = row < rows && e < p.dim;
  const unsigned r = on ? (unsigned)row : 0, bh = r / (unsigned)len;  // (below 2^29)
  const int t = (int)(r - bh * len), b = (int)(bh / (unsigned)heads), head = (int)(bh - b * heads);
  f32x4 x = 0.0f, y = 0.0f;
  if (on) {
    const float *px = (KEYS ? p.part_k : p.part_q) + row * p.dim + e;
    const float *py = p.part_v + row * p.dim + e;
    for (int i = 0; i < parts; i += 2) {  // two parts under way at a time
      const int64_t at = i * rows * p.dim, next = min(i + 1, parts - 1) * rows * p.dim;
      const f32x4 x0 = *(const f32x4 *)(px + at), x1 = *(const f32x4 *)(px + next);
      f32x4 y0 = 0.0f, y1 = 0.0f;
      if (KEYS) {
        y0 = *(const f32x4 *)(py + at);
        y1 = *(const f32x4 *)(py + next);
      }
      x += x0;
      y += y0;
      if (i + 1 < parts) {
        x += x1;
        y += y1;
      }
    }
    store4(tok_row<E>(KEYS ? p.dk : p.dq, b, t, head) + e, x);
    if (KEYS) store4(tok_row<E>(p.dv, b, t, head) + e, y);
  }
  bool x_nan = false, y_nan = false;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    x_nan |= x[i] != x[i];
    y_nan |= y[i] != y[i];
  }
  const uint64_t x_bits = __builtin_amdgcn_ballot_w64(x_nan), y_bits = __builtin_amdgcn_ballot_w64(y_nan);
  const uint64_t bits = x_bits | y_bits;
  if (!bits) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): the stores above come first
  const AttnK &c = args_again();
  const int most = KEYS ? 128 : 32;  // rows that a block's waves, or a wave, took together
  int until = 0;
  bool spoilt[2] = {false, false};  // of dK and dV, or of dQ
#pragma unroll 1
  for (int i = 0; i < 64; i += LANES) {
    if (!(bits >> i & ((1ull << LANES) - 1))) continue;
    const int hb = __builtin_amdgcn_readlane(b, i), hh = __builtin_amdgcn_readlane(head, i);
    const int ht = __builtin_amdgcn_readlane(t, i), first = ht / most * most;
    if (i >= until) {  // the rows of this wave from here on that were taken together
      const int n = min(min((64 - i) / LANES, first + most - ht), (KEYS ? c.kv_len : c.q_len) - ht);
      until = i + n * LANES;
      if (KEYS) {
        spoilt[0] = x_bits && queries_spoil<E>(c, hb, hh, first, ht, n, false, lane);
        spoilt[1] = y_bits && queries_spoil<E>(c, hb, hh, first, ht, n, true, lane);
      } else {
        const int4 s = rows_see(c, hb, first, min(most, c.q_len - first), lane);
        spoilt[0] = keys_spoil<E, KT, false>(c, c.k, hb, hh / c.share, s, lane);
      }
    }
    if (KEYS) {
      const uint64_t row = ((1ull << LANES) - 1) << i;
      if (spoilt[0] && x_bits & row) redo_key<E, 4>(c, hb, hh, ht, false, lane);
      if (spoilt[1] && y_bits & row) redo_key<E, 4>(c, hb, hh, ht, true, lane);
    } else if (spoilt[0]) {
      const int64_t bh = (int64_t)hb * c.q_heads + hh;
      const float lse = c.lse[bh * c.q_len + ht], delta = c.row_delta[bh * c.q_pad + ht];
      const int2 s = row_span(c, hb, ht);
      if (s.x >= s.y || (lse == lse && delta == delta)) redo_query<E, 4>(c, hb, hh, ht, lane);
    }
  }
}

// Both in one launch: the first `key_blocks` are keys'.
template <class E, int LANES>
__global__ __launch_bounds__(256) void k_attn_sum(AttnK p, int key_blocks) {
  if ((int)blockIdx.x < key_blocks) sum_rows<E, true, LANES>(p, blockIdx.x);
  else sum_rows<E, false, LANES>(p, blockIdx.x - key_blocks);
}

template <class E, int D>
hipError_t launch(const AttnK &p, hipStream_t st) {
  const int q_tiles = (p.q_len + KT - 1) / KT;
  if (q_tiles)
    k_attn_prep<E, D == 64 ? 8 : 16><<<p.batch * p.q_heads * q_tiles, 256, 0, st>>>(p, q_tiles);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int k_tiles = (p.kv_len + 127) / 128, tiles = (p.q_len + 127) / 128;
  if (k_tiles) {
    k_attn_bwd_kv<E, D><<<die_blocks(p.batch * p.kv_heads, k_tiles, p.kv_parts), 512, 0, st>>>(
        p, k_tiles, q_tiles);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (tiles) {
    const int blocks = die_blocks(p.batch * p.q_heads, tiles, p.q_parts) * p.passes;
    if (D == 128 && p.dim <= 96) k_attn_bwd_q<E, 96><<<blocks, 256, 0, st>>>(p, tiles);
    else k_attn_bwd_q<E, D><<<blocks, 256, 0, st>>>(p, tiles);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  constexpr int LANES = D == 64 ? 16 : 32;
  auto blocks_of = [](int64_t rows, int parts) {
    return parts > 1 ? (int)((rows * LANES + 255) / 256) : 0;
  };
  const int keys = blocks_of((int64_t)p.batch * p.kv_heads * p.kv_len, p.kv_parts);
  const int queries = blocks_of((int64_t)p.batch * p.q_heads * p.q_len, p.q_parts);
  if (keys + queries) k_attn_sum<E, LANES><<<keys + queries, 256, 0, st>>>(p, keys);
  return hipGetLastError();
}

}  // namespace

// Parts of a block's streamed tiles: enough to have a workgroup for each of 256
// compute units, every part with four tiles or more. With spans at least two where the
// blocks are no more than one for each; with causal rows, whose blocks are the most
// uneven, as many as make two for each, of six tiles or more. A part costs the write and
// the read of its 32-bit sums. No more than 16, which keeps the workspace to 16 results in 32
// bits; few queries over many keys would gain by more (16384 keys, 8 heads of 128, 1 query:
// 93 us, with up to 32 parts 87; 262144 keys, 2 heads, 64 queries: 660 and 497).
// Measured, q_len 2331, 8 heads of 64 with spans (152 blocks): dK and dV in one part 55
// us, in two 38 and their sum 7, in four 49 and 8; dQ in one part 35, in two 24 and their
// sum 5. Causal, whole backward, 4096 tokens, 16 heads of 128 on 4 (128 blocks of keys):
// in two parts 368 us, in four 300, in six 323; 2 x 4096 (256): dK and dV in one part
// 576, in two 330 and their sum 15.
void gs_attn_bwd_plan(AttnK *p, bool masked) {
  const bool causal = p->causal;
  auto parts = [masked, causal](int64_t blocks, int64_t tiles) {
    if (!blocks) return 1;
    auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    int64_t n = (256 + blocks - 1) / blocks;
    if (masked && !causal && blocks <= 256) n = n < 2 ? 2 : n;
    n = least(n, tiles / 4);
    const int64_t more = causal ? least((512 + blocks / 2) / blocks, tiles / 6) : 0;
    n = n < more ? more : n;
    return (int)(n < 1 ? 1 : n < 16 ? n : 16);
  };
  p->kv_parts = parts((int64_t)p->batch * p->kv_heads * ((p->kv_len + 127) / 128),
                      (int64_t)((p->q_len + 63) / 64) * p->share);
  p->q_parts = parts((int64_t)p->batch * p->q_heads * ((p->q_len + 127) / 128),
                     (p->kv_len + 63) / 64);
}

int gs_attn_passes(const AttnK &p);

hipError_t gs_launch_attn_bwd(AttnK p, int dtype, hipStream_t st) {
  p.passes = gs_attn_passes(p);
  if (dtype == GS_BF16) return p.dim <= 64 ? launch<bf16_t, 64>(p, st) : launch<bf16_t, 128>(p, st);
  return p.dim <= 64 ? launch<f16_t, 64>(p, st) : launch<f16_t, 128>(p, st);
}
