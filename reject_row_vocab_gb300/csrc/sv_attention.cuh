// What the attention kernels share: the call's parameters, a request's
// layout, the division of the work over blocks, and the join of its parts.
//
// A unit is one request, one cache head and one tile of MT query rows (a
// request's new rows times the query heads that share the cache head).  Its
// keys are the request's committed positions followed by its new rows, cut
// into tiles of KT keys.  All units' tiles form one line; block c of g works
// on tiles [c T / g, (c + 1) T / g) of it.  So every block gets the same
// number of tiles whatever the requests' lengths are, a long history is split
// over many blocks and a short one is not split at all.  A unit that lies in
// one block is finished there; otherwise each block leaves its part (m, l, O)
// and the unit's last block to arrive joins the parts in block order.
#pragma once

#include <cstdint>

#include "sv_kv.cuh"

namespace sv {

constexpr int kAttnMaxBlocks = 512;     // upper bound on the grid (the workspace is laid out for it)
constexpr int kAttnCounterBytes = sizeof(uint32_t) * kAttnMaxBlocks;

struct AttnParams {
  const char* q;
  int64_t q_row, q_head;  // strides in elements
  char* out;
  int64_t o_row, o_head;
  float* lse;
  KvView c;  // k and v at the call's layer
  const int32_t* cu;
  const int64_t* seq_lens;
  const int64_t* row_slots;
  const uint8_t* mask;
  uint32_t* status;
  int32_t batch, max_len, heads, group;
  int64_t total_rows;
  float scale_log2;  // scale * log2(e)
  uint32_t* tickets;  // [kAttnMaxBlocks], zero between calls
  float* parts;       // [grid, 2, part_floats]
};

struct AttnRequest {
  int64_t row0;
  int32_t n;      // new rows; 0 when the row range is invalid
  int32_t len;    // committed positions
  uint32_t status;
};

__device__ __forceinline__ AttnRequest attn_request(const AttnParams& p, int b) {
  AttnRequest r{static_cast<int64_t>(b) * p.max_len, p.max_len, 0, 0u};
  if (p.cu) {
    const int64_t lo = p.cu[b], hi = p.cu[b + 1];
    r.row0 = lo;
    r.n = static_cast<int32_t>(hi - lo);
    if (lo < 0 || hi <= lo || hi - lo > p.max_len || hi > p.total_rows) {
      r.n = 0;
      r.status = kStBadLayout;
      return r;
    }
  }
  const int64_t len = p.seq_lens[b], most = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
  if (len < 0) {
    r.status = kStBadLayout;
  } else if (len > most) {
    r.status = kStSlotRange;
    r.len = static_cast<int32_t>(most);
  } else {
    r.len = static_cast<int32_t>(len);
  }
  return r;
}

// The raw word that places key x of a request (a page id or a slot), and what becomes of it.  Fetched a tile ahead
// of its use, so that the dependent loads of the K/V rows do not wait for it.
__device__ __forceinline__ int64_t key_word(const AttnParams& p, const AttnRequest& r, int b, int x) {
  if (x < 0 || x >= r.len + r.n) return -1;
  if (x >= r.len && p.row_slots) return p.row_slots[r.row0 + (x - r.len)];
  const uint32_t page = static_cast<uint32_t>(x) / static_cast<uint32_t>(p.c.page_size);
  if (page >= static_cast<uint32_t>(p.c.max_pages)) return -1;
  return p.c.table[b * p.c.ld_table + page];
}
__device__ __forceinline__ int64_t key_offset(const AttnParams& p, const AttnRequest& r, int x, int64_t word) {
  if (x < 0 || x >= r.len + r.n) return -1;
  if (x >= r.len && p.row_slots) return kv_slot_offset(p.c, word);
  if (word < 0 || word > INT32_MAX) return -1;
  return kv_page_offset(p.c, static_cast<int32_t>(word), static_cast<uint32_t>(x) % static_cast<uint32_t>(p.c.page_size));
}

// 16-byte asynchronous copy global -> shared; zero-fills when !valid (the source is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Whether new row i sees new row j of the same request.
__device__ __forceinline__ bool row_sees(const AttnParams& p, int b, int i, int j) {
  if (!p.mask) return j <= i;
  return p.mask[(static_cast<int64_t>(b) * p.max_len + i) * p.max_len + j] != 0;
}

}  // namespace sv
