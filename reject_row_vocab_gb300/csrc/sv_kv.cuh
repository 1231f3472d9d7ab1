// The paged KV cache as the kernels see it: host checks of the caller's
// description and the address of a position or slot.
#pragma once

#include <cstdint>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

// Strides in elements, as the caller gives them.
struct KvView {
  char* k;
  char* v;
  int32_t es;  // bytes an element
  int32_t layers, pages, page_size, heads, head_dim;
  int64_t layer_stride, page_stride, slot_stride, head_stride;
  const int32_t* table;
  int32_t max_pages;
  int64_t ld_table;
  uint32_t div_mul, div_shift;  // x / page_size = umulhi(x, div_mul) >> div_shift for x < 2^31
};

// Multiplier and shift of an exact division of 31-bit numbers by d >= 2: with 2^l >= d, m = ceil(2^(31 + l) / d) exceeds
// 2^(31 + l) / d by less than 1, so x m / 2^(31 + l) exceeds x / d by less than 2^-l <= 1 / d for x < 2^31, which cannot
// reach the next whole number; m < 2^32 as 2^(l - 1) < d.
struct Divider {
  uint32_t mul, shift;
};
inline Divider divider(uint32_t d) {
  if (d < 2) return Divider{0u, 0u};  // the quotient is x itself
  uint32_t l = 1;
  while ((1ull << l) < d) ++l;
  return Divider{static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ uint32_t divide(uint32_t x, uint32_t mul, uint32_t shift) {
  return mul ? __umulhi(x, mul) >> shift : x;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline sv_status_t check_cache(const sv_kv_cache_t* c, KvView* v) {
  if (!c) return SV_ERR_NULL_ARG;
  if (!c->k || !c->v || !c->page_table) return SV_ERR_NULL_ARG;
  if (c->dtype != SV_F32 && c->dtype != SV_BF16) return SV_ERR_BAD_DTYPE;
  if (c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->heads > 65535 || c->head_dim < 1 ||
      c->head_dim > 256 || c->max_pages < 1 || c->ld_table < c->max_pages)
    return SV_ERR_BAD_SHAPE;
  if (c->layer_stride < 0 || c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0) return SV_ERR_BAD_SHAPE;
  // positions and slots are 31-bit numbers inside the kernels
  if (static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX / 2 ||
      static_cast<int64_t>(c->pages) * c->page_size > INT32_MAX / 2)
    return SV_ERR_BAD_SHAPE;
  const int32_t es = c->dtype == SV_BF16 ? 2 : 4;
  if (!aligned16(c->k) || !aligned16(c->v) || (c->head_dim * es) % 16 != 0 || (c->layer_stride * es) % 16 != 0 ||
      (c->page_stride * es) % 16 != 0 || (c->slot_stride * es) % 16 != 0 || (c->head_stride * es) % 16 != 0)
    return SV_ERR_MISALIGNED;
  const Divider d = divider(static_cast<uint32_t>(c->page_size));
  *v = KvView{static_cast<char*>(c->k), static_cast<char*>(c->v), es,          c->layers,      c->pages,
              c->page_size,             c->heads,                 c->head_dim, c->layer_stride, c->page_stride,
              c->slot_stride,           c->head_stride,           c->page_table, c->max_pages, c->ld_table,
              d.mul,                    d.shift};
  return SV_OK;
}

// Whether every entry of K and V has memory of its own (a call that writes to the cache needs that).  The steps have to be
// nested: each at least what the axes with smaller ones span.  Then K and V meet if and only if some combination of steps
// comes within a row of the distance between them, and of each axis, from the largest step down, only the multiples about
// what is left can.
inline bool entries_apart(const KvView& c) {
  struct Axis {
    int64_t step, n;  // bytes, entries
  } axes[4] = {};
  int count = 0;
  auto add = [&](int64_t step, int64_t n) {
    if (n < 2) return;
    int i = count++;
    for (; i > 0 && axes[i - 1].step > step; --i) axes[i] = axes[i - 1];
    axes[i] = Axis{step, n};
  };
  add(c.head_stride * c.es, c.heads), add(c.slot_stride * c.es, c.page_size);
  add(c.page_stride * c.es, c.pages), add(c.layer_stride * c.es, c.layers);
  const int64_t row = c.head_dim * c.es;
  int64_t span = row;
  for (int i = 0; i < count; ++i) {
    if (axes[i].step < span || axes[i].step > (INT64_MAX - span) / axes[i].n) return false;
    span += axes[i].step * (axes[i].n - 1);
  }
  const int64_t apart = reinterpret_cast<intptr_t>(c.v) - reinterpret_cast<intptr_t>(c.k);
  if (apart >= span || apart <= -span) return true;
  auto meets = [&](auto&& self, int i, int64_t left) -> bool {
    if (i < 0) return -row < left && left < row;
    const int64_t most = axes[i].n - 1, d = left / axes[i].step;
    for (int64_t m = d - 1; m <= d + 1; ++m)
      if (-most <= m && m <= most && self(self, i - 1, left - m * axes[i].step)) return true;
    return false;
  };
  return !meets(meets, count - 1, apart);
}

// Element offset (within a layer and head 0) of a slot, or -1 outside the cache.
__device__ __forceinline__ int64_t kv_slot_offset(const KvView& c, int64_t slot) {
  if (slot < 0 || slot >= static_cast<int64_t>(c.pages) * c.page_size) return -1;
  const uint32_t s = static_cast<uint32_t>(slot), page = divide(s, c.div_mul, c.div_shift);
  return page * c.page_stride + static_cast<int64_t>(s - page * c.page_size) * c.slot_stride;
}

// Element offset of entry `off` of page `page` (a page table's word), or -1 outside the cache.
__device__ __forceinline__ int64_t kv_page_offset(const KvView& c, int32_t page, uint32_t off) {
  if (page < 0 || page >= c.pages) return -1;
  return page * c.page_stride + static_cast<int64_t>(off) * c.slot_stride;
}

}  // namespace sv
