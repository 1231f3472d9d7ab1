// What the attention kernels over the 4-bit cache share.  AttnParams.c describes the pages (table, sizes, heads); the memory is
// PackedView's.
#pragma once

#include <cstdint>

#include "sv_attention.cuh"
#include "sv_rows.cuh"

namespace sv {

// Page and entry of key x of a request, from the word that places it (key_word); page -1: not there.
__device__ __forceinline__ Place packed_place(const AttnParams& p, const PackedView& c, const AttnRequest& r, int x, int64_t word) {
  if (x < 0 || x >= r.len + r.n) return Place{-1, 0};
  if (x >= r.len && p.row_slots) return slot_place(c, word);
  if (word < 0 || word >= c.pages) return Place{-1, 0};
  const uint32_t page = divide(static_cast<uint32_t>(x), c.div_mul, c.div_shift);
  return Place{static_cast<int32_t>(word), static_cast<int32_t>(static_cast<uint32_t>(x) - page * c.page_size)};
}

cudaError_t launch_packed_attention_wide(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace sv
