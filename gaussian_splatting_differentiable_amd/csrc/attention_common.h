// Shared parts of the attention kernels: tiles in LDS, matrix operands, masks.
//
// Every kernel computes with v_mfma_f32_32x32x16: operand A holds 32 rows and B
// 32 columns of 16 contraction slots, lane l the 8 slots 8 (l / 32) .. of row or
// column l % 32; the result holds column l % 32 and, in register i, row
// 8 (i / 4) + 4 (l / 32) + i % 4. The scores are computed with the streamed rows
// (keys in the forward and in dQ, queries in dK and dV) as rows and the wave's
// own rows as columns. A lane then holds scores of one own row only, so the
// softmax needs one exchange (lanes l and l + 32), and its registers 8 k .. + 7
// are already the B operand of the second product: contraction slots may be in
// any order that A shares. A for that product is the transpose of a streamed
// tile, read by ds_read_b64_tr_b16 in that order.
#pragma once
#include "tokens_common.h"

#define LDS_PTR(T, p) ((__attribute__((address_space(3))) T *)(p))

constexpr float ATTN_LN2 = 0.6931471805599453f;
constexpr float ATTN_LOG2E = 1.4426950408889634f;
constexpr int KT = 64;  // streamed rows per tile

template <class E>
using frag = vec<E, 8>;

__device__ __forceinline__ f32x16 mfma(frag<bf16_t> a, frag<bf16_t> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(frag<f16_t> a, frag<f16_t> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// x of lane l combined with x of lane l ^ 32.
__device__ __forceinline__ float other_half(float x, bool max) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float a = __uint_as_float(r[0]), b = __uint_as_float(r[1]);
  return max ? fmaxf(a, b) : a + b;
}

__device__ __forceinline__ int wave_min(int x) {
  for (int m = 32; m; m >>= 1) x = min(x, __shfl_xor(x, m));
  return x;
}
__device__ __forceinline__ int wave_max(int x) {
  for (int m = 32; m; m >>= 1) x = max(x, __shfl_xor(x, m));
  return x;
}
__device__ __forceinline__ float wave_fmax(float x) {
  for (int m = 32; m; m >>= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}

// Orders this wave's LDS stores before its later LDS loads (and the reverse), for
// LDS that only this wave uses.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The keys [x, y) that query `t` of batch entry b sees; (0, 0) if it sees none: the
// span as it is stored, and cut to the keys and the causal rule.
__device__ __forceinline__ int2 raw_span(const AttnK &p, int b, int t) {
  return p.spans ? p.spans[(int64_t)b * p.span_stride + t] : make_int2(0, p.kv_len);
}
__device__ __forceinline__ int2 cut_span(const AttnK &p, int t, int2 s) {
  const int lo = max(s.x, 0);
  int hi = min(s.y, p.kv_len);
  if (p.causal) hi = min((int64_t)hi, (int64_t)t + 1 + p.kv_len - p.q_len);
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}
__device__ __forceinline__ int2 row_span(const AttnK &p, int b, int t) {
  return cut_span(p, t, raw_span(p, b, t));
}

// Rows of a 128-row block whose spans have no key in common with that of its first row
// that sees any. A block whose rows belong to two sequences would walk over the keys
// of both, one after the other; with p.passes 2 every block is launched twice, once
// for the other rows and once for these (most of the second ones have none and end at
// once). `firsts`: LDS for four spans; every thread of the block calls it.
__device__ __forceinline__ bool apart(int2 span, int2 *firsts, int wave, int lane) {
  const uint64_t some = __builtin_amdgcn_ballot_w64(span.x < span.y);
  const int at = some ? __builtin_ctzll(some) : 0;
  const int2 first = make_int2(__shfl(span.x, at), __shfl(span.y, at));
  if (lane == 0) firsts[wave] = first;
  __syncthreads();
  int2 s = firsts[0];
#pragma unroll
  for (int w = 1; w < 4; w++)
    if (s.x >= s.y) s = firsts[w];
  return span.x < span.y && (span.x >= s.y || span.y <= s.x);
}

// Workgroups are dealt to the 8 dies in turn, each with an L2 of its own: give a
// die a run of consecutive items, which share their heads' streamed rows.
__device__ __forceinline__ int die_order(int block, int blocks) {
  const int per = blocks >> 3, rest = blocks & 7, die = block & 7;
  return die * per + min(die, rest) + (block >> 3);
}

// The dies that share a group of heads: one for each group where the heads divide
// evenly, else 2, 4 or 8 that take its items in turn.
inline __host__ __device__ int group_dies(int heads) {
  return heads & 1 ? 8 : heads & 2 ? 4 : heads & 4 ? 2 : 1;
}

// Workgroups for `parts` of every row tile of every head, a multiple of 8.
inline int die_blocks(int heads, int tiles, int parts) {
  const int64_t dies = group_dies(heads), group = heads * dies / 8 * tiles * parts;
  return (int)(8 * ((group + dies - 1) / dies));
}

struct Item {
  int head, tile, part;  // head < 0: none (the last ones of a group)
};

// What workgroup `block` works on. Its die's heads share their streamed rows in the
// die's L2: a head's tiles follow each other. Where a mask makes rows' keys uneven,
// the heads do, from the last tile (causal rows see more keys the later they are) to
// the first: long blocks come early, and those that a compute unit takes differ.
__device__ __forceinline__ Item die_item(int block, int heads, int tiles, int parts, bool uneven) {
  const int dies = group_dies(heads), n = (int)((int64_t)heads * dies >> 3), die = block & 7;
  const int at = (block >> 3) * dies + die % dies, whole = at / parts;
  Item x = {-1, 0, at - whole * parts};
  if (whole >= n * tiles) return x;
  if (uneven) {
    x.tile = tiles - 1 - whole / n;
    x.head = die / dies * n + whole % n;
  } else {
    x.tile = whole % tiles;
    x.head = die / dies * n + whole / tiles;
  }
  return x;
}

// ---- tiles in LDS: KT rows of D elements in 16-byte chunks. Chunk c of row r is
// stored as chunk c ^ swizzle(r) of that row, so that neither the 16-byte row
// reads of 16 consecutive rows nor the transposing reads of 4 consecutive rows
// meet in the 64 banks.
template <int D>
__device__ __forceinline__ int swizzle(int row) {
  if (D == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
  if (D == 96) return (row >> 2) & 3;  // a row is 3/4 of the banks: its 4 next ones differ
  return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);  // D == 64: two rows to the banks
}

template <int D>
__device__ __forceinline__ int lds_at(int row, int chunk) {  // in elements
  return row * D + ((chunk ^ swizzle<D>(row)) << 3);
}

// A streamed matrix of `rows` rows of `dim` elements, 16-byte chunks read with
// bounds checks: rows past its end and elements past `dim` read as 0.
template <class E>
struct Stream {
  const E *base;
  int64_t ts;
  int rows, dim;
};

// NT threads copy one tile of R rows from global memory straight into LDS (no
// registers in between): N copies of 16 bytes a thread. The copies of a wave land
// in consecutive chunks, so the swizzle is applied to where a lane reads: lanes of
// a row read all of its chunks, in another order. Bounds as for Stream. The data
// is there after copied<>() in the issuing wave.
// LEAN: a thread's copies, which must be of rows with the same swizzle, share one offset
// through a descriptor each, and their places in LDS are scalars: for a kernel without
// vector registers to spare (where there are, the scalar instructions cost more: 16384
// tokens, heads of 128, forward 1036 us so and 992 plain).
template <class E, int D, int NT, int R, bool LEAN = false>
struct Copy {
  static constexpr int C = D / 8, N = R * C / NT;
  static_assert(R * C % NT == 0, "whole copies");
  static_assert(!LEAN || NT % (16 * C) == 0, "rows of one swizzle");

  static __device__ __forceinline__ void issue(const Stream<E> &m, int row0, E *lds, int tid) {
    const int left = min(m.rows - row0, R);
    const int64_t bytes = left > 0 ? ((int64_t)(left - 1) * m.ts + m.dim) * 2 : 0;
    const char *base = (const char *)(m.base + (int64_t)row0 * m.ts);
    const int step = LEAN ? NT / C * (int)m.ts * 2 : 0;
    const int wave0 = LEAN ? __builtin_amdgcn_readfirstlane(tid) & ~63 : NT > 64 ? tid & ~63 : 0;
#pragma unroll
    for (int i = 0; i < N; i++) {
      auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)(base + (LEAN ? (int64_t)i * step : 0)),
                                                    0, max((int)bytes - i * step, 0), 0x00020000);
      const int at_once = LEAN ? tid : i * NT + tid;
      const int row = NT % C ? at_once / C : (LEAN ? 0 : i * (NT / C)) + tid / C;
      const int col = (NT % C ? at_once % C : tid % C) ^ swizzle<D>(row);
      // past `dim`: an offset out of every tile's bounds
      const unsigned at = 8 * col < m.dim ? (unsigned)(row * (int)m.ts + 8 * col) * 2u : 0x7fffff00u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, LDS_PTR(void, lds + (i * NT + wave0) * 8), 16, at, 0, 0, 0);
    }
  }
};

// 0, which the compiler does not know: what is read from LDS at an offset of it in a
// loop is read in every turn, not kept in registers across them.
__device__ __forceinline__ int opaque_zero() {
  int z;
  asm volatile("s_mov_b32 %0, 0" : "=s"(z));
  return z;
}

// One wave copies 64 words into LDS, as Copy does.
template <class T>
__device__ __forceinline__ void copy_words(const T *from, T *lds, int lane) {
  auto rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)from, 0, 256, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, LDS_PTR(void, lds), 4, lane * 4, 0, 0, 0);
}

// Waits until at most `left` of this wave's newest memory operations are under way
// (0: all are done), and for its LDS reads.
template <int left>
__device__ __forceinline__ void copied() {
  __builtin_amdgcn_s_waitcnt((left & 15) | (left >> 4 << 14) | 0x70);
}

// Tiles that the block copied are there for all its waves.
__device__ __forceinline__ void block_copied() {
  copied<0>();
  __syncthreads();
}

// Operand of 32 rows (as rows of A or columns of B) and 16 elements from a row on;
// zero where not `on`. The load is made either way, from the row's start then, so
// that the loads of a row are under way together and not each in a branch.
template <class E>
__device__ __forceinline__ frag<E> row_operand(const E *row, int chunk, bool on) {
  const frag<E> f = *(const frag<E> *)(row + (on ? 8 * chunk : 0));
  return on ? f : (frag<E>)(E)0.0f;
}

// row0: a multiple of 32, so that the swizzle depends on the lane alone.
template <class E, int D>
__device__ __forceinline__ frag<E> lds_rows(const E *tile, int row0, int k, int lane) {
  return *(const frag<E> *)(tile + row0 * D + lds_at<D>(lane & 31, 2 * k + (lane >> 5)));
}

// Operand A of the transpose: rows = elements 32 d .. + 31 of the tile's rows,
// contraction = tile rows row0 .. + 15 (row0 a multiple of 16) in the order of a
// score register run. The rows 8 further on have the swizzle of these ^ 2. ROWS: the
// tile's rows, where row0 is not known to the compiler; it must see that the reads
// stay in their buffer, or they wait for copies into the others.
template <class E, int D, int ROWS = 0>
__device__ __forceinline__ frag<E> lds_cols(const E *tile, int row0, int d, int lane) {
  const int r = 4 * (lane >> 5) + ((lane & 15) >> 2);
  const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), in = 4 * (lane & 1);
  int x = in + lds_at<D>(r, c), y = in + lds_at<D>(r, c ^ 2), more = row0 * D;
  if (ROWS) {
    x = (x + more) & (ROWS * D - 1);
    y = (y + more) & (ROWS * D - 1);
    more = 0;
  }
  // The constant last: it stays in the instruction, and the lane's part in registers
  // that all reads share.
  const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, tile + x + more));
  const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, tile + y + more + 8 * D));
  return __builtin_bit_cast(frag<E>, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Registers 8 k .. + 7 of a score block as operand B.
template <class E>
__device__ __forceinline__ frag<E> pack8(const f32x16 &s, int k) {
  frag<E> f;
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = (E)s[8 * k + i];  // to nearest even
  return f;
}

// Row of the streamed 32 that register i of a lane holds.
__device__ __forceinline__ int acc_row(int i, int lane) {
  return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
}

// ---- rows done again. 0 x NaN and 0 x infinity are NaN: in a matrix product, a row of a
// masked pair that is not finite spoils results that do not see it; and in fp16 a p that
// rounds to 0 those that see an infinity. A result with a NaN is therefore computed again
// from its own pairs in 32 bits, by one wave: but only where there is such a row (else the
// NaN is its own), and not on once all of it is NaN. 2048 tokens, 8 heads of 64, bf16, one
// value row with a NaN that is seen, forward and backward: 0.1 ms, as without it (every NaN
// computed again: 7.2 ms); where two sequences that share a block meet, 0.6 (they are
// latency: about 3.5 us for 64 pairs of a row).

template <class E>
inline constexpr bool is_half = false;
template <>
inline constexpr bool is_half<f16_t> = true;

// The kernel's arguments (its first), read again where this is called: code that hardly ever
// runs then keeps none of them in registers while the rest of the kernel does.
__device__ __forceinline__ const AttnK &args_again() {
  auto at = (const __attribute__((address_space(4))) AttnK *)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return *(const AttnK *)at;
}

// Whether a row can spoil results that it is multiplied into by 0: it is not finite, or,
// with `seen` (by all of them), infinite.
template <class E>
__device__ __forceinline__ bool row_spoils(const E *row, int dim, bool seen) {
  typedef vec<unsigned short, 8> bits;
  const bits inf = (unsigned short)(is_half<E> ? 0x7c00 : 0x7f80);
  bits most = 0, off = 0x7fff;  // largest magnitude; how near one comes to an infinity
#pragma unroll 1
  for (int d = 0; d < dim; d += 32) {  // the loads of 32 elements together
    bits x[4];
#pragma unroll
    for (int k = 0; k < 4; k++) x[k] = *(const bits *)(row + (d + 8 * k < dim ? d + 8 * k : 0));
#pragma unroll
    for (int k = 0; k < 4; k++) {
      x[k] &= (unsigned short)0x7fff;
      most = __builtin_elementwise_max(most, x[k]);
      off = __builtin_elementwise_min(off, x[k] ^ inf);
    }
  }
  int top = 0, near = 0x7fff;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    top = max(top, (int)most[i]);
    near = min(near, (int)off[i]);
  }
  return near == 0 || (!seen && top > inf[0]);
}

// What n <= 64 queries from t0 on see: the first key and the end of all their spans, then
// those of the keys that all of them see.
__device__ __forceinline__ int4 rows_see(const AttnK &p, int b, int t0, int n, int lane) {
  const bool on = lane < n;
  const int2 s = on ? row_span(p, b, t0 + lane) : make_int2(0, 0);
  return {wave_min(s.x < s.y ? s.x : INT32_MAX), wave_max(s.y), wave_max(on ? s.x : 0),
          wave_min(on ? s.y : INT32_MAX)};
}

// Whether x (keys or values) holds a row that spoils among those of the tiles of T rows
// that queries were multiplied with and that not all of them see (`see` of rows_see); with
// SEEN also among those that all see.
template <class E, int T, bool SEEN>
__device__ __forceinline__ bool keys_spoil(const AttnK &p, const TokK &x, int b, int kvh, int4 see,
                                           int lane) {
  if (see.x >= see.y) return false;
  const int end = min((see.y + T - 1) / T * T, p.kv_len);
#pragma unroll 1
  for (int j0 = see.x / T * T; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    const bool seen = j >= see.z && j < see.w;
    bool bad = false;
    if (j < end && (SEEN || !seen)) bad = row_spoils(tok_row<E>(x, b, j, kvh), p.dim, seen);
    if (__builtin_amdgcn_ballot_w64(bad)) return true;
  }
  return false;
}

// A sum of rows that a wave does again: 16 lanes a row, eight elements in each, four rows
// (j % 4 = lane / 16) at a time, the loads of 4 N rows together (N: as the kernel has
// registers).
template <int N>
struct RowSum {
  float a[8] = {};

  // += w_j x_j of the rows j0 + j with bit j of `some` (j < 64; w of lane j), none of them
  // past `last`. Returns whether anything is not NaN yet.
  template <class E>
  __device__ __forceinline__ bool add(float w, uint64_t some, const TokK &x, int b, int head,
                                      int j0, int last, int dim, int lane) {
    const int e = 8 * (lane & 15), group = lane >> 4;
    bool open = true;
#pragma unroll 1
    for (int j1 = 0; open && j1 < 64 && some >> j1; j1 += 4 * N) {
      frag<E> f[N];
#pragma unroll
      for (int i = 0; i < N; i++)
        f[i] = *(const frag<E> *)(tok_row<E>(x, b, min(j0 + j1 + 4 * i + group, last), head) +
                                  (e < dim ? e : 0));
#pragma unroll
      for (int i = 0; i < N; i++) {
        const int j = j1 + 4 * i + group;
        const float wj = __shfl(w, j);
        const bool on = some >> j & 1;
#pragma unroll
        for (int c = 0; c < 8; c++) a[c] = on ? fmaf(wj, (float)f[i][c], a[c]) : a[c];
      }
      float left = a[0];  // NaN where all are
#pragma unroll
      for (int c = 1; c < 8; c++) left = fmaxf(left, a[c]);
      open = __builtin_amdgcn_ballot_w64(e < dim && left == left);
    }
    return open;
  }

  __device__ __forceinline__ void shrink(float by) {
#pragma unroll
    for (int c = 0; c < 8; c++) a[c] *= by;
  }

  // The sum times `by`, stored.
  template <class E>
  __device__ __forceinline__ void store(E *row, float by, int dim, int lane) {
    frag<E> f;
#pragma unroll
    for (int c = 0; c < 8; c++) {
      a[c] += __shfl_xor(a[c], 16);
      a[c] += __shfl_xor(a[c], 32);
      f[c] = (E)(a[c] * by);
    }
    if (lane < 16 && 8 * lane < dim) *(frag<E> *)(row + 8 * lane) = f;
  }
};

__device__ __forceinline__ uint64_t first_bits(int n) { return n < 64 ? (1ull << n) - 1 : ~0ull; }

// (the loads of 8 N elements together)
template <int N, class E>
__device__ __forceinline__ float dot_row(const E *a, const E *b, int dim) {
  float s = 0.0f;
#pragma unroll 1
  for (int d = 0; d < dim; d += 8 * N) {
    frag<E> x[N], y[N];
#pragma unroll
    for (int k = 0; k < N; k++) {
      const int at = d + 8 * k < dim ? d + 8 * k : 0;
      x[k] = *(const frag<E> *)(a + at);
      y[k] = *(const frag<E> *)(b + at);
    }
#pragma unroll
    for (int k = 0; k < N; k++) {
      if (d + 8 * k >= dim) continue;
#pragma unroll
      for (int i = 0; i < 8; i++) s = fmaf((float)x[k][i], (float)y[k][i], s);
    }
  }
  return s;
}
