// The ring that carries K and V to the attention kernels for bf16, and the warps around it: one that walks the line of
// tiles ahead of the others (the plan), four that load, one that fetches the next unit's Q.  The kernels differ in who
// consumes the tiles.
//
// A tile is 128 keys by DP (64 or 128) columns in blocks of 64 columns, 128 bytes a row, in the 128-byte swizzle that TMA
// writes and the matrix unit reads: piece c (16 bytes) of row r lies at (c ^ r) % 8 of its row.  Tile g's K is group 2 g
// of the ring, its V group 2 g + 1.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "sv_attention.cuh"

namespace sv {

constexpr int kKeys = 128;        // keys of a tile
constexpr int kLoadWarps = 4;
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kPlans = 4;         // segments the plan is ahead by
constexpr uint64_t kWaitNs = 1000000000ull;

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// K and V of the call's layer as [pages][page_size][heads][head_dim] tensors, in boxes of 64 columns of `rows` rows of a
// page (a power of two that divides the page's; 0: none, the pages are copied row by row).
struct KvMaps {
  CUtensorMap k, v;
  int32_t rows;
};

__device__ __forceinline__ void box_copy(uint32_t dst, const CUtensorMap* map, int x, int head, int row, int page,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(head), "r"(row), "r"(page), "r"(bar)
      : "memory");
}

// As mbar_try_wait, the thread suspended for up to about `ns`: warps that poll take issue slots from those that work.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

// The rest of a wait that is long.  (Out of line, like all that seldom runs: what the roles run by turns has to stay in the
// instruction cache.)
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_wait_bounded(bar, parity, abort, kWaitNs)) return true;
  *abort = 1;
  return false;
}

// An arrival that the thread's earlier asynchronous copies make, once they are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int DP, int NB>
struct KvRing {
  static constexpr int kBlock = kKeys * 128;        // 128 rows of 64 columns
  static constexpr int kTile = kBlock * (DP / 64);
  static constexpr int kPieces = DP / 8;            // 16-byte pieces of a row
  static constexpr int kInfo = 8;                   // tiles whose validity is kept
  // shared memory of the ring: the tiles, and behind them
  static constexpr int kValid = NB * kTile;                      // uint32 [kInfo][8]: four valid words, four bad
  static constexpr int kPlan = kValid + kInfo * 8 * 4;           // AttnSegment [kPlans]
  static constexpr int kBars = kPlan + kPlans * static_cast<int>(sizeof(AttnSegment));
  // full, empty [NB], plan, read [kPlans], q, q free [2]
  static constexpr int kSums = kBars + (2 * NB + 2 * kPlans + 4) * 8;  // int64 [34]: sums [32], find [2]
  static constexpr int kAbort = kSums + 34 * 8;
  static constexpr int kBytes = kAbort + 16;

  char* mem;       // of the ring
  uint32_t base;   // its shared address
  int lane;
  uint32_t plans;  // segments read (or planned)

  __device__ KvRing(char* at) : mem(at), base(smem_addr(at)), lane(threadIdx.x & 31), plans(0) {}

  __device__ uint32_t full(uint32_t group) const { return base + kBars + group % NB * 8; }
  __device__ uint32_t empty(uint32_t group) const { return base + kBars + (NB + group % NB) * 8; }
  __device__ uint32_t plan_bar(uint32_t i) const { return base + kBars + (2 * NB + i % kPlans) * 8; }
  __device__ uint32_t read_bar(uint32_t i) const { return base + kBars + (2 * NB + kPlans + i % kPlans) * 8; }
  __device__ uint32_t q_bar(int i) const { return base + kBars + (2 * NB + 2 * kPlans + i) * 8; }
  __device__ uint32_t q_free(int i) const { return base + kBars + (2 * NB + 2 * kPlans + 2 + i) * 8; }
  __device__ static uint32_t phase(uint32_t group) { return group / NB & 1; }
  __device__ uint32_t tile(uint32_t group) const { return base + group % NB * kTile; }
  __device__ char* tile_mem(uint32_t group) const { return mem + group % NB * kTile; }
  __device__ uint32_t* valid(uint32_t g) const { return reinterpret_cast<uint32_t*>(mem + kValid) + g % kInfo * 8; }
  __device__ AttnSegment* plan_slot(uint32_t i) const { return reinterpret_cast<AttnSegment*>(mem + kPlan) + i % kPlans; }
  __device__ int64_t* find() const { return sums() + 32; }
  __device__ int64_t* sums() const { return reinterpret_cast<int64_t*>(mem + kSums); }
  __device__ volatile int* abort() const { return reinterpret_cast<volatile int*>(mem + kAbort); }
  // 16-byte piece c of row r of a tile
  __device__ static uint32_t piece(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  }

  // By one thread: empties: arrivals that free a tile, readers: warps that read the plan, q_frees: arrivals that free a Q.
  __device__ void init(int empties, int readers, int q_frees) const {
    for (int i = 0; i < NB; ++i) mbar_init(full(i), kLoadThreads), mbar_init(empty(i), empties);
    for (int i = 0; i < kPlans; ++i) mbar_init(plan_bar(i), 1), mbar_init(read_bar(i), readers);
    for (int i = 0; i < 2; ++i) mbar_init(q_bar(i), 32), mbar_init(q_free(i), q_frees);
    *abort() = 0;
  }

  // A wait that gives up ends every role; the lanes of a warp leave together.
  __device__ bool wait_one(uint32_t bar, uint32_t parity) const {
    // (the call is the last resort: registers are saved around it)
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait_for(bar, parity, 10000)) return true;
    return wait_on(bar, parity, abort());
  }
  __device__ bool wait(uint32_t bar, uint32_t parity) const { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; }

  // The next segment of the plan, for a whole warp (or, with ONE, for its first lane alone); false at the end, or after a
  // wait that gave up.
  template <bool ONE = false>
  __device__ bool next(AttnSegment& s) {
    if (!(ONE ? wait_one(plan_bar(plans), plans / kPlans & 1) : wait(plan_bar(plans), plans / kPlans & 1))) return false;
    s = *plan_slot(plans);
    if (!ONE) __syncwarp();
    if (lane == 0) mbar_arrive(read_bar(plans));
    ++plans;
    return s.cnt > 0;
  }

  // The same, left in the plan until release() (for warps that have no registers to keep it in).
  __device__ const AttnSegment* peek() const {
    if (!wait(plan_bar(plans), plans / kPlans & 1)) return nullptr;
    const AttnSegment* s = plan_slot(plans);
    return s->cnt > 0 ? s : nullptr;
  }
  __device__ void release() {
    __syncwarp();
    if (lane == 0) mbar_arrive(read_bar(plans));
    ++plans;
  }

  // The planning warp: the block's segments in order; one without tiles ends them.  Segments that are only part of their
  // unit (two at most) are put down in `parts` too; their number is returned to every lane.
  template <int MT, int U>
  __device__ int plan(const AttnParams& p, const AttnSpan& span, AttnSegment* parts = nullptr) {
    int split = 0;
    if (lane == 0) {
      AttnWalk<MT, kKeys, U> walk(p, span);
      AttnSegment s{};
      for (bool more = true; more; ++plans) {
        more = walk.next(s);
        if (!more) s.cnt = 0;
        if (parts && more && s.cnt < s.nt) parts[split++] = s;
        if (plans >= kPlans && !wait_one(read_bar(plans), (plans / kPlans - 1) & 1)) break;
        *plan_slot(plans) = s;
        mbar_arrive(plan_bar(plans));
      }
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, split, 0);
  }

  // Loading warp lw.  A warp has 32 of a tile's keys, a lane one key's place, handed round by shuffles; the word that
  // places a lane's key of the next tile is on its way while this tile is copied.
  __device__ void load(const AttnParams& p, const KvMaps& maps, int lw) {
    AttnSegment s{};
    bool more = next(s);
    int t = s.t0;
    int64_t word = more ? key_word(p, s.r, s.b, t * kKeys + lw * 32 + lane) : -1;
    uint32_t q = 0;  // groups issued
    bool ok = true;
    const int c = lane % kPieces, sub = lane / kPieces;
    constexpr int kStep = 32 / kPieces;  // rows a warp copies at once
    const bool in_head = c * 8 < p.c.head_dim;
    while (more && ok) {
      const int x = t * kKeys + lw * 32 + lane;
      const int64_t off = key_offset(p, s.r, x, word);
      const uint32_t good = __ballot_sync(0xffffffffu, off >= 0);
      const uint32_t bad = __ballot_sync(0xffffffffu, x < s.r.len + s.r.n && off < 0);
      // a tile of history in boxes: this lane's box of the warp's 32 keys
      const bool boxes = maps.rows > 0 && (t + 1) * kKeys <= s.r.len;
      const int per = boxes ? 32 / maps.rows : 1;
      const int box_row = boxes ? lane % per * maps.rows : 0, box_col = boxes ? lane / per : 0;
      const int box_head = s.hkv;
      const int64_t box_page = __shfl_sync(0xffffffffu, word, box_row);
      const uint32_t box_key = static_cast<uint32_t>(t * kKeys + lw * 32 + box_row);
      const uint32_t box_in = box_key - divide(box_key, p.c.div_mul, p.c.div_shift) * p.c.page_size;
      const int64_t shift = (static_cast<int64_t>(s.hkv) * p.c.head_stride + c * 8) * 2;
      if (++t >= s.t0 + s.cnt) {
        more = next(s);
        t = s.t0;
      }
      if (more) word = key_word(p, s.r, s.b, t * kKeys + lw * 32 + lane);
#pragma unroll 1
      for (int which = 0; which < 2; ++which, ++q) {
        if (q >= NB && !wait(empty(q), phase(q - NB))) {
          ok = false;
          break;
        }
        if (which == 0 && lane == 0) {
          valid(q >> 1)[lw] = good;
          valid(q >> 1)[4 + lw] = bad;
        }
        const uint32_t dst = tile(q);
        if (boxes) {
          // (a page outside the cache is outside the tensor: the box is filled with zeros)
          if (lane == 0)
            mbar_arrive_expect_tx(full(q), 32 * 128 * (DP / 64));
          else
            mbar_arrive(full(q));
          __syncwarp();
          if (box_col < DP / 64)
            box_copy(dst + box_col * kBlock + (lw * 32 + box_row) * 128, which ? &maps.v : &maps.k, box_col * 64, box_head,
                     static_cast<int>(box_in), static_cast<int>(box_page), full(q));
          continue;
        }
        const char* src = (which ? p.c.v : p.c.k) + shift;
#pragma unroll 8
        for (int i = 0; i < 32; i += kStep) {
          const int64_t o = __shfl_sync(0xffffffffu, off, i + sub);
          const bool live = o >= 0 && in_head;
          cp_async16(dst + piece(lw * 32 + i + sub, c), live ? src + o * 2 : p.c.k, live);
        }
        cp_async_arrive(full(q));  // when this thread's copies so far are in place
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    if (*abort())  // copies in flight end before the block does
      for (uint32_t i = q > NB ? q - NB : 0; i < q; ++i)
        for (int n = 0; n < 100 && !mbar_try_wait_for(full(i), phase(i), 10000); ++n) {
        }
  }

  // The warp that fetches Q: rows of up to MT query rows a unit (rows that do not exist are 0), 64-column blocks of
  // `block` bytes at `at`, in the tiles' swizzle; slots Qs in turn, `slot_rows` rows apart.
  template <int MT>
  __device__ void load_q(const AttnParams& p, uint32_t at, int block, int slots, int slot_rows) {
    AttnSegment s;
    const int c = lane % kPieces, sub = lane / kPieces;
    const bool in_head = c * 8 < p.c.head_dim;
    for (uint32_t unit = 0; next(s); ++unit) {
      const int slot = static_cast<int>(unit % slots);
      const uint32_t turn = unit / slots;
      if (turn > 0 && !wait(q_free(slot), (turn - 1) & 1)) break;
      const int rows = s.r.n * p.group - s.rt * MT;
      const int upto = min(MT, (rows + 31) & ~31);  // rows of the warps that have any
      for (int r0 = 0; r0 < upto; r0 += 32) {       // a lane finds one row's place, the warp copies the 32 of them
        const int grow = s.rt * MT + r0 + lane, i = grow / p.group;
        const int64_t from = r0 + lane < rows
                                 ? (s.r.row0 + i) * p.q_row + (s.hkv * p.group + grow - i * p.group) * p.q_head
                                 : -1;
#pragma unroll 8
        for (int j = 0; j < (MT < 32 ? MT : 32); j += 32 / kPieces) {
          const int64_t o = __shfl_sync(0xffffffffu, from, j + sub);
          const bool live = o >= 0 && in_head;
          const int row = slot * slot_rows + r0 + j + sub;
          cp_async16(at + (c >> 3) * block + row * 128 + (((c & 7) ^ (row & 7)) << 4), live ? p.q + (o + c * 8) * 2 : p.q,
                     live);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_async();
      mbar_arrive(q_bar(slot));
    }
    cp_async_wait<0>();
  }

  // At the end, by every thread after the block's last barrier (never expected: see SV_DEV_TIMEOUT).
  __device__ void report_abort(const AttnParams& p) const {
    if (!*abort()) return;
    if (threadIdx.x == 0) atomicExch(p.err, 1u);
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x) p.status[b] = kStTimeout;
  }
};

// The maps of a call's layer (bf16).
KvMaps kv_maps(const KvView& c);

}  // namespace sv
