// Dropout whose mask comes from a counter-based generator and is never stored.
//
// keep(i) = word(i) >= drop_below; y = residual + keep(i) x scale, with scale =
// 1 / (1 - p). word(i) is word i % 4 of the Philox 4x32 block (10 rounds) at
// counter offset + i / 4 under key `seed`: J. Salmon et al., "Parallel random
// numbers: as easy as 1, 2, 3" (2011). The gradient with respect to x is the
// same map applied to dL/dy, so one kernel serves both directions. A dropped
// element is selected away, not multiplied by 0: its NaN or infinity is gone.
//
// Bound: HBM. The generator costs about 100 instructions per four elements (20
// of them 32-bit multiplies at a quarter of the rate). 32768 x 1024, bf16: 34 us with a
// residual (201 MB), 31 without (134 MB), partly from the last-level cache; 1535033 x 1,
// fp32: 4.2 us (12 MB), where the launch is what bounds it.
#include "tokens_common.h"

namespace {

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t ctr, uint64_t key) {
  uint32_t a = (uint32_t)ctr, b = (uint32_t)(ctr >> 32), c = 0, d = 0;
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; r++) {
    const uint32_t h0 = __umulhi(a, 0xD2511F53u), l0 = a * 0xD2511F53u;
    const uint32_t h1 = __umulhi(c, 0xCD9E8D57u), l1 = c * 0xCD9E8D57u;
    a = h1 ^ b ^ k0;
    b = l1;
    c = h0 ^ d ^ k1;
    d = l0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{a, b, c, d}};
}

// Contiguous arrays on 16-byte boundaries: a thread takes 8 elements, two
// generator blocks, and one thread the last count % 8; per_row: 8 elements of one
// row (cols a multiple of 8), one block.
template <class E, bool RES, bool ROW>
__global__ __launch_bounds__(256) void k_dropout_vec(DropK p, int64_t n8) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += step) {
    const f32x4 x0 = load4((const E *)p.x + 8 * i), x1 = load4((const E *)p.x + 8 * i + 4);
    f32x4 y0 = 0, y1 = 0;
    if (RES) {
      y0 = load4((const E *)p.res + 8 * i);
      y1 = load4((const E *)p.res + 8 * i + 4);
    }
    if (ROW) {
      const int64_t r = 8 * i / p.cols;
      const Words w = philox(p.offset + (uint64_t)(r >> 2), p.seed);
      const uint32_t m = r & 2 ? (r & 1 ? w.w[3] : w.w[2]) : (r & 1 ? w.w[1] : w.w[0]);
      if (m >= p.drop_below) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          y0[j] = x0[j] * p.scale + y0[j];
          y1[j] = x1[j] * p.scale + y1[j];
        }
      }
    } else {
      const Words a = philox(p.offset + 2 * (uint64_t)i, p.seed);
      const Words b = philox(p.offset + 2 * (uint64_t)i + 1, p.seed);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        y0[j] += a.w[j] >= p.drop_below ? x0[j] * p.scale : 0.0f;
        y1[j] += b.w[j] >= p.drop_below ? x1[j] * p.scale : 0.0f;
      }
    }
    store4((E *)p.y + 8 * i, y0);
    store4((E *)p.y + 8 * i + 4, y1);
  }
  if (ROW || blockIdx.x || threadIdx.x) return;
  const int64_t n = p.rows * p.cols;
  for (int64_t i = 8 * n8; i < n; i++) {
    const Words w = philox(p.offset + (uint64_t)(i >> 2), p.seed);
    const uint32_t m = i & 2 ? (i & 1 ? w.w[3] : w.w[2]) : (i & 1 ? w.w[1] : w.w[0]);
    float y = m >= p.drop_below ? (float)((const E *)p.x)[i] * p.scale : 0.0f;
    if (RES) y += (float)((const E *)p.res)[i];
    ((E *)p.y)[i] = (E)y;
  }
}

// Any strides, alignment and column count: a thread takes four consecutive
// elements of the [rows][cols] order, one generator block.
template <class E, bool RES>
__global__ __launch_bounds__(256) void k_dropout_any(DropK p, int64_t n4) {
  const int64_t step = (int64_t)gridDim.x * 256, n = p.rows * p.cols;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += step) {
    int64_t r = 4 * i / p.cols, c = 4 * i - r * p.cols;
    Words w = philox(p.offset + (uint64_t)(p.per_row ? r >> 2 : i), p.seed);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (4 * i + j < n) {
        const uint32_t m =
            !p.per_row ? w.w[j]
                       : (r & 2 ? (r & 1 ? w.w[3] : w.w[2]) : (r & 1 ? w.w[1] : w.w[0]));
        float y = m >= p.drop_below ? (float)((const E *)p.x)[r * p.x_stride + c] * p.scale : 0.0f;
        if (RES) y += (float)((const E *)p.res)[r * p.res_stride + c];
        ((E *)p.y)[r * p.y_stride + c] = (E)y;
        if (++c == p.cols) {
          c = 0;
          if ((++r & 3) == 0 && p.per_row) w = philox(p.offset + (uint64_t)(r >> 2), p.seed);
        }
      }
    }
  }
}

template <class E, bool RES>
void launch(const DropK &p, bool vector, hipStream_t st) {
  const int64_t n = p.rows * p.cols, items = vector ? n / 8 : (n + 3) / 4;
  const int blocks = (int)((items + 255) / 256 < 16384 ? (items + 255) / 256 : 16384);
  if (!vector)
    k_dropout_any<E, RES><<<blocks, 256, 0, st>>>(p, items);
  else if (p.per_row)
    k_dropout_vec<E, RES, true><<<blocks, 256, 0, st>>>(p, items);
  else
    k_dropout_vec<E, RES, false><<<blocks, 256, 0, st>>>(p, items);
}

template <class E>
void launch_type(const DropK &p, hipStream_t st) {
  const int64_t n = p.rows * p.cols;
  const bool flat = p.rows == 1 || (p.x_stride == p.cols && p.y_stride == p.cols &&
                                    (!p.res || p.res_stride == p.cols));
  const uintptr_t at = (uintptr_t)p.x | (uintptr_t)p.res | (uintptr_t)p.y;
  const bool vector = flat && at % 16 == 0 && n >= 8 && (!p.per_row || p.cols % 8 == 0);
  if (p.res) launch<E, true>(p, vector, st);
  else launch<E, false>(p, vector, st);
}

}  // namespace

hipError_t gs_launch_dropout(DropK p, int dtype, hipStream_t st) {
  if (p.per_row && p.cols == 1) {
    // one element a row: the same words, one to an element of a strided column
    p.per_row = 0;
  }
  if (dtype == GS_F32) launch_type<float>(p, st);
  else if (dtype == GS_BF16) launch_type<bf16_t>(p, st);
  else launch_type<f16_t>(p, st);
  return hipGetLastError();
}
