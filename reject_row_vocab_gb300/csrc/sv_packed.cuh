// A KV cache held in 4 bits: its layout, its numbers, and the host checks of
// the caller's description.
//
// 16 neighbouring columns of a head share a scale.  A value is scale * code:
// codes are e2m1 (a sign, and 0, 0.5, 1, 1.5, 2, 3, 4 or 6), scales are a half
// float's upper eight bits without the sign (five exponent bits, three of
// mantissa), at most 10240.  The product has six significant bits and lies
// below 2^16, so it is exact in a half float, in bf16 and in fp32: what reads
// the cache computes with exactly the values that it holds.  (Scales with
// seven exponent steps more than e4m3's need no second scale for a tensor:
// groups whose largest value is 4e-4 keep all three bits.)
//
// The entries of one page and head lie together, in a block: K's codes, V's
// codes ([page_size][head_dim / 2] bytes each, the even column in the lower
// half), K's scales, V's scales ([page_size][head_dim / 16]), up to a multiple
// of 16 bytes.  So a page's K and V of a head come with one bulk copy.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "sv_kv.cuh"

namespace sv {

constexpr uint32_t kMostScale = 0xe2u;  // 10240: the largest scale with 6 * scale below 2^16

struct PackedView {
  char* data;  // of layer 0, or of the call's layer
  int32_t layers, pages, page_size, heads, head_dim;
  int64_t layer_stride, page_stride, head_stride;  // bytes
  const int32_t* table;
  int32_t max_pages;
  int64_t ld_table;
  uint32_t div_mul, div_shift;  // as in KvView
  int32_t dtype;                // of the rows that go with the cache
};

// Where things lie in a block of `rows` entries.
__host__ __device__ __forceinline__ int packed_v_codes(int rows, int dim) { return rows * (dim / 2); }
__host__ __device__ __forceinline__ int packed_k_scales(int rows, int dim) { return rows * dim; }
__host__ __device__ __forceinline__ int packed_v_scales(int rows, int dim) { return rows * dim + rows * (dim / 16); }
inline int64_t packed_block_bytes(int64_t rows, int64_t dim) { return (rows * dim + rows * (dim / 8) + 15) / 16 * 16; }

inline bool packed_shape(int32_t page_size, int32_t head_dim) {
  return page_size >= 1 && page_size <= (1 << 20) && head_dim >= 32 && head_dim <= 256 && head_dim % 32 == 0;
}

inline sv_status_t check_packed_cache(const sv_packed_kv_cache_t* c, PackedView* v) {
  if (!c) return SV_ERR_NULL_ARG;
  if (!c->data || !c->page_table) return SV_ERR_NULL_ARG;
  if (c->dtype != SV_F32 && c->dtype != SV_BF16) return SV_ERR_BAD_DTYPE;
  if (c->layers < 1 || c->pages < 1 || !packed_shape(c->page_size, c->head_dim) || c->heads < 1 || c->heads > 65535 ||
      c->max_pages < 1 || c->ld_table < c->max_pages)
    return SV_ERR_BAD_SHAPE;
  if (c->layer_stride < 0 || c->page_stride < 0 || c->head_stride < 0) return SV_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX / 2 ||
      static_cast<int64_t>(c->pages) * c->page_size > INT32_MAX / 2)
    return SV_ERR_BAD_SHAPE;
  if (!aligned16(c->data) || c->layer_stride % 16 != 0 || c->page_stride % 16 != 0 || c->head_stride % 16 != 0)
    return SV_ERR_MISALIGNED;
  const Divider d = divider(static_cast<uint32_t>(c->page_size));
  *v = PackedView{static_cast<char*>(c->data), c->layers,      c->pages,       c->page_size,  c->heads,
                  c->head_dim,                 c->layer_stride, c->page_stride, c->head_stride, c->page_table,
                  c->max_pages,                c->ld_table,     d.mul,          d.shift,        static_cast<int32_t>(c->dtype)};
  return SV_OK;
}

// Whether the steps of `n` axes are nested, each at least what the axes with smaller ones span, over rows of `row` bytes; the
// whole span is left in *bytes.
struct StepAxis {
  int64_t step, n;
};
inline bool steps_nested(StepAxis* axes, int count, int64_t row, int64_t* bytes) {
  int used = 0;
  for (int i = 0; i < count; ++i) {  // sorted by their steps, those of one entry left out
    if (axes[i].n < 2) continue;
    const StepAxis a = axes[i];
    int j = used++;
    for (; j > 0 && axes[j - 1].step > a.step; --j) axes[j] = axes[j - 1];
    axes[j] = a;
  }
  int64_t span = row;
  for (int i = 0; i < used; ++i) {
    if (axes[i].step < span || axes[i].step > (INT64_MAX - span) / axes[i].n) return false;
    span += axes[i].step * (axes[i].n - 1);
  }
  *bytes = span;
  return true;
}

// Whether every block has memory of its own (a call that writes to the cache needs that).
inline bool blocks_apart(const PackedView& c) {
  StepAxis axes[3] = {{c.head_stride, c.heads}, {c.page_stride, c.pages}, {c.layer_stride, c.layers}};
  int64_t span;
  return steps_nested(axes, 3, packed_block_bytes(c.page_size, c.head_dim), &span);
}

// ---------------------------------------------------------------------------
// The numbers
// ---------------------------------------------------------------------------

// The values of eight codes (a word; the lowest nibble first) as four pairs of half floats.
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two scales as a pair of half floats, from bytes 0 and 2 of w (the others 0), times `one` / 128: a shift that may also silence
// them.  Bytes that no call writes, above the largest scale, count as it: every pattern stands for a number.
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, uint32_t one = 128u) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w * one), "r"(kMostScale << 7 | kMostScale << 23));
  return r;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t b = byte < kMostScale ? byte : kMostScale;
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7)));
}

// The scale's byte for a group whose largest magnitude is `top` (finite): the scale nearest to top / 6, half way to the even
// one.  Which of two neighbouring scales is nearer is decided on 6 * (their middle), which is exact: a quotient is not.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  top = fminf(top, 61440.0f);
  // the half float below top / 6, or the one beside it
  uint32_t b = __half_as_ushort(__float2half_rz(top * (1.0f / 6.0f))) >> 7;
  if (b >= kMostScale) b = kMostScale - 1;
  const float lo = scale_value(b), hi = scale_value(b + 1);
  const float mid = 3.0f * (lo + hi);  // six times the middle
  return top > mid || (top == mid && (b & 1u)) ? b + 1 : b;
}

// The codes of eight quotients: each the nearest code, half way to the even one, 6 at most.
__device__ __forceinline__ uint32_t pack_codes(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

}  // namespace sv
