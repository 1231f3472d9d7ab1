// The ring that carries K and V to the attention kernels, and the warps around it: one that walks the line of tiles ahead
// of the others (the plan), four that load, one that fetches the next unit's Q.  The kernels differ in who consumes the
// tiles.
//
// A tile is 128 keys.  Its rows are cut into H entries of CB blocks of 128 bytes (64 columns of bf16, 32 of fp32) in the
// 128-byte swizzle that TMA writes and the matrix unit reads: piece c (16 bytes) of row r lies at (c ^ r) % 8 of its
// block's row.  The entries of tile g are groups 2 H g + h (K) and 2 H g + H + h (V) of the ring.
//
// The history's rows come in boxes of a page's rows, all of an entry's issued by one warp: what a warp does for an entry
// (find the pages, wait for room, issue) takes about a microsecond, and four entries are on their way at once.  New rows,
// the history's last, odd page sizes' and all beside them are gathered row by row, by all loading warps together.  (Rows that
// are gathered, the zeros behind them and the values taken out of V are written through the generic proxy, boxes through the
// asynchronous one: a place that the former wrote is fenced before a box goes there.  The barriers alone do not order the two.)
#pragma once

#include <cstdint>

#include <cuda.h>

#include "sv_attention.cuh"

namespace sv {

constexpr int kKeys = 128;        // keys of a tile
constexpr int kLoadWarps = 4;
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kPlans = 8;         // segments the plan is ahead by
constexpr uint64_t kWaitNs = 1000000000ull;

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// K and V of the call's layer as [pages][page_size][heads][head_dim] tensors, in boxes of 128 bytes of `rows` rows of a
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

__device__ __forceinline__ void mbar_arrive_times(uint32_t bar, uint32_t times) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(times) : "memory");
}

template <int ES, int CB, int NB, int H, bool EARLY = false>
struct KvRing {
  static constexpr int kEntries = NB;
  static constexpr int kBlock = kKeys * 128;        // 128 rows of 128 bytes
  static constexpr int kTile = kBlock * CB;         // an entry
  static constexpr int kPieces = CB * 8;            // 16-byte pieces of an entry's row
  static constexpr int kEach = 16 / ES;             // elements of a piece
  static constexpr int kInfo = 16;                  // tiles whose validity is kept
  // shared memory of the ring: the tiles, and behind them
  static constexpr int kValid = NB * kTile;                      // uint32 [kInfo][8]: four valid words, four bad
  static constexpr int kPlan = kValid + kInfo * 8 * 4;           // AttnSegment [kPlans]
  static constexpr int kBars = kPlan + kPlans * static_cast<int>(sizeof(AttnSegment));
  // full, empty [NB], plan, read [kPlans], q, q free [2], open [2 NB]
  static constexpr int kSums = kBars + (4 * NB + 2 * kPlans + 4) * 8;  // int64 [34]: sums [32], find [2]
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
  __device__ uint32_t open(uint32_t i) const { return base + kBars + (2 * NB + 2 * kPlans + 4 + i % (2 * NB)) * 8; }
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
    for (int i = 0; i < NB; ++i) mbar_init(full(i), 2 * kLoadThreads), mbar_init(empty(i), empties);
    for (int i = 0; i < 2 * NB; ++i) mbar_init(open(i), 1);
    for (int i = 0; i < kPlans; ++i) mbar_init(plan_bar(i), 1), mbar_init(read_bar(i), readers);
    for (int i = 0; i < kInfo * 8; ++i) valid(0)[i] = 0u;
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

  // What a loading warp knows of its next tile: the words that place the keys are long on their way.
  struct Ahead {
    int64_t word, box_word;  // of this lane's key, of this lane's box
    uint32_t g;              // tiles before it
    int x0, hkv;             // first key, cache head
    int len, n;              // the request's; n 0: no more tiles
    int boxed, row0, each;   // rows [0, boxed) come in boxes, the warp gathers rows row0 .. row0 + each - 1
  };

  // Rows of K or V, 32 keys' places being the lanes' `off`: the first `each` of them to the shared rows from dst on.
  __device__ void gather(const AttnParams& p, uint32_t dst, const char* from, int h, int hkv, int64_t off, int each) const {
    const int c = lane % kPieces, sub = lane / kPieces;
    constexpr int kStep = 32 / kPieces;  // rows a warp copies at once
    const char* src = from + (static_cast<int64_t>(hkv) * p.c.head_stride + c * kEach) * ES + h * CB * 128;
    const bool in_head = (h * kPieces + c) * kEach < p.c.head_dim;
    auto copy = [&](int i) {
      const int64_t o = __shfl_sync(0xffffffffu, off, i + sub);
      const bool live = o >= 0 && in_head;
      cp_async16(dst + piece(i + sub, c), live ? src + o * ES : p.c.k, live);
    };
    if (each == 32) {
#pragma unroll 8
      for (int i = 0; i < 32; i += kStep) copy(i);
    } else {
#pragma unroll 1
      for (int i = 0; i < each; i += kStep) copy(i);
    }
  }

  // The end of a loading warp that went through `groups` groups: copies in flight end before the block does.
  __device__ void drain(uint32_t groups) const {
    cp_async_commit();
    cp_async_wait<0>();
    if (*abort())
      for (uint32_t i = groups > NB ? groups - NB : 0; i < groups; ++i)
        for (int n = 0; n < 100 && !mbar_try_wait_for(full(i), phase(i), 10000); ++n) {
        }
  }

  // Loading warp lw where there are no boxes: a quarter of each tile's keys, a lane one key's place.
  __device__ void load_rows(const AttnParams& p, int lw) {
    AttnSegment s{};
    bool more = next(s);
    int t = s.t0;
    int64_t word = more ? key_word(p, s.r, s.b, t * kKeys + lw * 32 + lane) : -1;
    uint32_t q = 0;  // groups gone through
    for (bool ok = true; more && ok;) {
      const int x = t * kKeys + lw * 32 + lane, hkv = s.hkv;
      const int64_t off = key_offset(p, s.r, x, word);
      const uint32_t good = __ballot_sync(0xffffffffu, off >= 0);
      const uint32_t bad = __ballot_sync(0xffffffffu, x < s.r.len + s.r.n && off < 0);
      const uint32_t g = q / (2 * H);
      if (++t >= s.t0 + s.cnt) {
        more = next(s);
        t = s.t0;
      }
      if (more) word = key_word(p, s.r, s.b, t * kKeys + lw * 32 + lane);
#pragma unroll 1
      for (int e = 0; e < 2 * H; ++e, ++q) {
        if (q >= NB && !wait(empty(q), phase(q - NB))) {
          ok = false;
          break;
        }
        if (e == 0 && lane == 0) valid(g)[lw] = good, valid(g)[4 + lw] = bad;
        gather(p, tile(q) + lw * 32 * 128, e >= H ? p.c.v : p.c.k, e % H, hkv, off, 32);
        cp_async_arrive(full(q));  // when this thread's copies so far are in place
        mbar_arrive(full(q));
      }
    }
    drain(q);
  }

  // Loading warp lw with boxes.  A group is owned by the warp that is its number modulo the loading warps: it issues the
  // boxes.  Rows that do not come in boxes are gathered by all of the warps.
  // (A wait by parity is good where the barrier's phase before is known to be over, and where the next one cannot come
  // before the wait is done.  No group comes that a warp has not had its part in.  That a group's place is free follows a
  // wait for a group at most four before it; with that group, the place's own phase before is over, if the consumer frees
  // K and V in order, or at most K of the tile behind V's before V.  Where the places are too few for that (EARLY), the
  // owner waits, and opens the group to the others; the openings are gone through by every warp, and are twice as many as
  // the places.)
  __device__ void load(const AttnParams& p, const KvMaps& maps, int lw) {
    if (maps.rows == 0) return load_rows(p, lw);
    static_assert(NB >= kLoadWarps && kLoadWarps == 4, "parity of the places, owners of the groups");
    AttnSegment s{};
    bool more = next(s);
    int t = s.t0;
    uint32_t tiles = 0;
    const int nb = kKeys / maps.rows;  // boxes of a block
    const int box_row = lane % nb * maps.rows, box_col = lane / nb;
    auto ahead = [&](Ahead& a) {
      a.n = 0;
      for (; more; ++t, ++tiles) {
        if (t >= s.t0 + s.cnt) {
          more = next(s);
          t = s.t0;
          if (!more) return;
        }
        a.x0 = t * kKeys;
        a.boxed = max(min(s.r.len - a.x0, kKeys), 0) / maps.rows * maps.rows;
        // (boxes alone: with one entry a row, two of the four warps own them)
        if (a.boxed < kKeys || H > 1 || (tiles & 1) == (lw >> 1)) break;
      }
      if (!more) return;
      ++t;
      a.g = tiles++, a.hkv = s.hkv, a.len = s.r.len, a.n = s.r.n;
      a.each = ((kKeys - a.boxed) / kLoadWarps + 7) & ~7;  // (eight rows are the swizzle's period)
      a.row0 = min(a.boxed + lw * a.each, kKeys);
      a.each = min(a.each, kKeys - a.row0);
      if (a.boxed > 0) a.box_word = key_word(p, s.r, s.b, a.x0 + box_row);
      if (a.boxed < kKeys) a.word = key_word(p, s.r, s.b, a.x0 + a.row0 + lane);
    };
    const int c = lane % kPieces, sub = lane / kPieces;
    constexpr int kStep = 32 / kPieces;  // rows a warp copies at once
    uint32_t last = 0, opened = 0;              // groups before the next tile's; openings so far
    uint32_t gathered = 0;                      // groups up to the end of the last tile that had gathered rows
    bool ok = true;
    Ahead now;
    ahead(now);
    while (now.n > 0 && ok) {
      const Ahead a = now;
      ahead(now);
      last = (a.g + 1) * 2 * H;
      const bool whole = a.boxed == kKeys;
      if (!whole) gathered = last;
      uint32_t good = 0u;  // lane j < 4: of keys 32 j .. 32 j + 31, those in boxes
      if (a.boxed > 0) {
        const uint32_t found = __ballot_sync(0xffffffffu, a.box_word >= 0 && a.box_word < p.c.pages && box_row < a.boxed);
        for (int x = 0; x < 32; x += min(maps.rows, 32))
          if (found >> ((lane & 3) * 32 + x) / maps.rows & 1u)
            good |= (maps.rows >= 32 ? 0xffffffffu : (1u << maps.rows) - 1u) << x;
      }
      int64_t off = -1;
      uint32_t there = 0u, missing = 0u;  // of the warp's own rows
      if (!whole) {
        AttnRequest r{};
        r.len = a.len, r.n = a.n;
        const int x = a.x0 + a.row0 + lane;
        if (lane < a.each) off = key_offset(p, r, x, a.word);
        there = __ballot_sync(0xffffffffu, off >= 0);
        missing = __ballot_sync(0xffffffffu, lane < a.each && x < a.len + a.n && off < 0);
      }
      const uint32_t key = static_cast<uint32_t>(a.x0 + box_row);
      const int in = static_cast<int>(key - divide(key, p.c.div_mul, p.c.div_shift) * p.c.page_size);
#pragma unroll 1
      for (int e = 0; e < 2 * H; ++e) {
        const uint32_t q = a.g * 2 * H + e;
        const int h = e % H;
        const bool is_v = e >= H, own = q % kLoadWarps == lw;
        if (!own && whole) continue;
        if (q >= NB && (own || !EARLY) && !wait(empty(q), phase(q - NB))) {
          ok = false;
          break;
        }
        if (own) {
          if (e == 0 && lane < 4) {
            const int rest = a.boxed - lane * 32;  // of the word's keys, those that come in boxes
            const uint32_t boxes = rest >= 32 ? 0xffffffffu : rest <= 0 ? 0u : (1u << rest) - 1u;
            if (boxes) {
              atomicOr(valid(a.g) + lane, good);
              atomicOr(valid(a.g) + 4 + lane, boxes & ~good);
            }
          }
          // words are put together from 0: here those of a tile whose place was read long ago
          if (e == 0 && lane < 8) valid(a.g + kInfo / 2)[lane] = 0u;
          if (a.boxed > 0) {
            if (q >= NB && q - NB < gathered) fence_async();  // by the lanes that issue the boxes, behind their wait
            // (a page outside the cache is outside the tensor: the box is filled with zeros)
            if (lane == 0) mbar_expect_tx(full(q), a.boxed * 128 * CB);
            __syncwarp();
            if (box_col < CB && box_row < a.boxed)
              box_copy(tile(q) + box_col * kBlock + box_row * 128, is_v ? &maps.v : &maps.k,
                       (h * CB + box_col) * (128 / ES), a.hkv, in, static_cast<int>(a.box_word), full(q));
          }
          if (whole) {
            mbar_arrive_times(full(q), 2 * kLoadWarps);
            continue;
          }
        }
        if (EARLY && q >= NB) {
          __syncwarp();
          if (own && lane == 0) mbar_arrive(open(opened));
          if (!wait(open(opened), opened / (2 * NB) & 1)) {
            ok = false;
            break;
          }
          ++opened;
        }
        if (e == 0 && lane == 0) {
          uint32_t* v = valid(a.g) + (a.row0 >> 5);
          const int shift = a.row0 & 31;
          if (there << shift) atomicOr(v, there << shift);
          if (missing << shift) atomicOr(v + 4, missing << shift);
          if (shift && there >> (32 - shift)) atomicOr(v + 1, there >> (32 - shift));
          if (shift && missing >> (32 - shift)) atomicOr(v + 5, missing >> (32 - shift));
        }
        if (a.x0 + a.row0 < a.len + a.n) {
          gather(p, tile(q) + a.row0 * 128, is_v ? p.c.v : p.c.k, h, a.hkv, off, a.each);
        } else if (is_v) {  // a weight of 0 times what lay there before has to be 0 (a score of it is masked)
#pragma unroll 1
          for (int i = 0; i < a.each; i += kStep)
            *reinterpret_cast<uint4*>(tile_mem(q) + piece(a.row0 + i + sub, c)) = make_uint4(0u, 0u, 0u, 0u);
        }
        cp_async_arrive(full(q));  // when this thread's copies so far are in place
        mbar_arrive(full(q));
      }
    }
    drain(last);
  }

  // The warp that fetches Q: rows of up to MT query rows a unit (rows that do not exist are 0), 128-byte blocks of `block`
  // bytes at `at`, in the tiles' swizzle; slots Qs in turn, `slot_rows` rows apart.
  template <int MT>
  __device__ void load_q(const AttnParams& p, uint32_t at, int block, int slots, int slot_rows) {
    constexpr int kRowPieces = kPieces * H, kLanes = kRowPieces < 32 ? kRowPieces : 32;  // lanes on a row
    AttnSegment s;
    const int c0 = lane % kLanes, sub = lane / kLanes;
    for (uint32_t unit = 0; next(s); ++unit) {
      const int slot = static_cast<int>(unit % slots);
      const uint32_t turn = unit / slots;
      if (turn > 0 && !wait(q_free(slot), (turn - 1) & 1)) break;
      const int rows = s.r.n * p.group - s.rt * MT;
      const int upto = min(MT, (rows + 31) & ~31);  // rows of the warps that have any
      for (int r0 = 0; r0 < upto; r0 += 32) {       // a lane finds one row's place, the warp copies the 32 of them
        const int grow = s.rt * MT + r0 + lane, i = grow / p.group;
        const int64_t from = r0 + lane < min(rows, MT)
                                 ? (s.r.row0 + i) * p.q_row + (s.hkv * p.group + grow - i * p.group) * p.q_head
                                 : -1;
#pragma unroll 8
        for (int j = 0; j < (MT < 32 ? MT : 32); j += 32 / kLanes) {
          const int64_t o = __shfl_sync(0xffffffffu, from, j + sub);
          const int row = slot * slot_rows + r0 + j + sub;
#pragma unroll
          for (int c = c0; c < kRowPieces; c += kLanes) {
            const bool live = o >= 0 && c * kEach < p.c.head_dim;
            cp_async16(at + (c >> 3) * block + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                       live ? p.q + (o + c * kEach) * ES : p.q, live);
          }
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

// The NaN and infinite values that the products left out, added by a warp to the rows that it has just written: to its
// part of the unit, or, without one, to the output, where rows of `none` (a bit each) saw scores of -inf alone and stay 0.
// Units of MT rows, columns d0 .. d0 + COLS - 1.
template <bool BF16, int MT, int COLS>
__device__ __noinline__ void add_nonfinite(const AttnParams& p, const AttnSegment& s, int rows, int d0, uint32_t none, float* part) {
  __syncwarp();
  for (int x = threadIdx.x & 31; x < min(rows, MT) * (COLS / 4); x += 32) {
    const int row = x / (COLS / 4), d = d0 + x % (COLS / 4) * 4, grow = s.rt * MT + row, i = grow / p.group;
    if (d >= p.c.head_dim || (!part && (none >> row & 1u))) continue;
    const float4 f = nonfinite_seen<BF16, kKeys>(p, s, i, d);
    if (part) {
      float4* at = reinterpret_cast<float4*>(part) + (d / 4) * MT + row;
      const float4 v = *at;
      *at = make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w);
    } else {
      const int head = s.hkv * p.group + grow - i * p.group;
      char* at = p.out + ((s.r.row0 + i) * p.o_row + head * p.o_head + d) * (BF16 ? 2 : 4);
      float4 v;
      if (BF16) {
        const uint2 u = *reinterpret_cast<const uint2*>(at);
        v = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
      } else {
        v = *reinterpret_cast<const float4*>(at);
      }
      store4<BF16>(at, make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w));
    }
  }
  __syncwarp();
}

// The maps of a call's layer.
KvMaps kv_maps(const KvView& c);

}  // namespace sv
