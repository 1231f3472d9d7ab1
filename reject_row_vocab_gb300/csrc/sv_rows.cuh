// A call's new rows: which request a row belongs to, and where its entry lies
// in the cache (the layout of the attention calls).
#pragma once

#include <cstdint>

#include "sv_packed.cuh"

namespace sv {

struct RowsView {
  int32_t batch, max_len;
  int64_t total;
  const int32_t* cu;
  const int64_t* seq_lens;
  const int64_t* row_slots;
};

inline sv_status_t check_rows(const sv_rows_t* r, RowsView* v) {
  if (!r) return SV_ERR_NULL_ARG;
  if (r->batch < 0 || r->batch > 65535 || r->max_len < 1 || r->total_rows < 0 || r->total_rows > INT32_MAX)
    return SV_ERR_BAD_SHAPE;
  if (!r->cu_seqlens && r->total_rows < static_cast<int64_t>(r->batch) * r->max_len) return SV_ERR_BAD_SHAPE;
  *v = RowsView{r->batch, r->max_len, r->total_rows, r->cu_seqlens, r->seq_lens, r->row_slots};
  return SV_OK;
}

// Rows that can belong to a request.
__host__ __device__ __forceinline__ int64_t rows_count(const RowsView& v) {
  return v.cu ? v.total : static_cast<int64_t>(v.batch) * v.max_len;
}

__device__ __forceinline__ bool range_ok(const RowsView& v, int64_t lo, int64_t hi) {
  return lo >= 0 && hi >= lo && hi - lo <= v.max_len && hi <= v.total;
}

// The request of row r and the row's number in it, for a whole warp; -1 for a row of none.
__device__ __forceinline__ int row_request(const RowsView& v, int64_t r, int lane, int* j) {
  if (!v.cu) {
    const int b = static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(v.max_len));
    *j = static_cast<int>(r - static_cast<int64_t>(b) * v.max_len);
    return b;
  }
  // The last b with cu[b] <= r, 32 places at a time.
  int lo = 0, n = v.batch;  // among [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = lane * step < n && v.cu[at] <= r;
    const uint32_t any = __ballot_sync(0xffffffffu, le);
    const int k = any ? 31 - __clz(any) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  int found = -1, first = 0;
  auto look = [&](int b) {
    int32_t from = 0;
    bool mine = false;
    if (b < v.batch) {
      from = v.cu[b];
      const int32_t to = v.cu[b + 1];
      mine = range_ok(v, from, to) && from <= r && r < to;
    }
    const uint32_t any = __ballot_sync(0xffffffffu, mine);
    if (!any) return false;
    const int k = 31 - __clz(any);
    found = __shfl_sync(0xffffffffu, b, k);
    first = __shfl_sync(0xffffffffu, from, k);
    return true;
  };
  if (!look(lo + lane)) {
    // offsets that decrease somewhere mislead the search: every request is asked
#pragma unroll 1
    for (int b0 = 0; b0 < v.batch; b0 += 32)
      if (look(b0 + lane)) break;
  }
  *j = static_cast<int>(r - first);
  return found;
}

// Page and entry of a row's place.
struct Place {
  int32_t page, in;  // page -1: outside the cache
};
template <class C>  // KvView or PackedView
__device__ __forceinline__ Place slot_place(const C& c, int64_t slot) {
  if (slot < 0 || slot >= static_cast<int64_t>(c.pages) * c.page_size) return Place{-1, 0};
  const uint32_t s = static_cast<uint32_t>(slot), page = divide(s, c.div_mul, c.div_shift);
  return Place{static_cast<int32_t>(page), static_cast<int32_t>(s - page * c.page_size)};
}
template <class C>
__device__ __forceinline__ Place position_place(const C& c, int b, int64_t x) {
  if (x < 0 || x >= static_cast<int64_t>(c.max_pages) * c.page_size) return Place{-1, 0};
  const uint32_t s = static_cast<uint32_t>(x), p = divide(s, c.div_mul, c.div_shift);
  const int32_t page = c.table[b * c.ld_table + p];
  if (page < 0 || page >= c.pages) return Place{-1, 0};
  return Place{page, static_cast<int32_t>(s - p * c.page_size)};
}

// What is wrong with requests first, first + step, ... : flagged once a call.
__device__ __forceinline__ void flag_requests(const RowsView& v, uint32_t* status, int64_t first, int64_t step) {
  for (int64_t b = first; b < v.batch; b += step) {
    bool bad = v.seq_lens && v.seq_lens[b] < 0;
    if (v.cu) bad = bad || !range_ok(v, v.cu[b], v.cu[b + 1]);
    if (bad) atomicOr(status + b, kStBadLayout);
  }
}

}  // namespace sv
