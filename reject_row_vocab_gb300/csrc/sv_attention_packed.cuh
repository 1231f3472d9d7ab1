// What the attention kernels over the 4-bit cache share: how its tiles come to shared memory.  (AttnParams.c describes the pages:
// table, sizes, heads; the memory is PackedView's.)
//
// A tile is 128 keys of a cache head.  It lies in shared memory as the cache's own blocks, one after the other: a page's block
// is one bulk copy, K and V, codes and scales.  Of pages of a multiple of 128 entries a tile is a part, in four copies (codes
// and scales of K and of V), as a block of 128.  Rows that lie apart (new rows staged elsewhere; all rows where 128 and the page
// size do not divide one another) are gathered to the places that they would have, which takes a warp 40 turns a tile: one token of
// 128 requests of 64 to 8192 in pages of 48 to 200 such entries 1000 us (153 in pages of 16), blocks of 16 rows of 64 requests 103
// us (86).  Whatever lies in places of keys that are not
// there stands for finite numbers (every pattern of bits does): scores with it are masked, and its weights are 0.
#pragma once

#include <cstdint>

#include "sv_attention_ring.cuh"
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

// A cache and how its tiles are laid out.
struct PackedTiles {
  PackedView c;
  int32_t rows_log;  // a tile is blocks of 2^rows_log entries
  int32_t block;     // bytes from one of them to the next
  int32_t copies;    // bulk copies a block (1 or 4); 0: its rows are gathered
};

inline PackedTiles packed_tiles(const PackedView& c) {
  PackedTiles t{c, 7, 0, 0};
  if (c.page_size <= kKeys && kKeys % c.page_size == 0) {
    t.rows_log = 0;
    while ((1 << t.rows_log) < c.page_size) ++t.rows_log;
    t.copies = 1;
  } else if (c.page_size % kKeys == 0) {
    t.copies = 4;
  }
  t.block = static_cast<int32_t>(packed_block_bytes(1 << t.rows_log, c.head_dim));
  return t;
}

// A query row's way to half floats and back: its largest magnitude (the bits of a bf16 without the sign) goes to 2^14 .. 2^15, as far
// as a factor goes; and the factor of its scores, scale / up.
struct RowScale {
  float up, factor;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top, float scale) {
  const int e = min(static_cast<int>(top >> 7), 254), shift = min(14 + 127 - e, 126), half = shift / 2;
  // (back by two factors: one alone may be too large or too small)
  return RowScale{__uint_as_float(static_cast<uint32_t>(shift + 127) << 23),
                  scale * __uint_as_float(static_cast<uint32_t>(127 - half) << 23) *
                      __uint_as_float(static_cast<uint32_t>(127 - (shift - half)) << 23)};
}

// Bytes of a tile of heads of up to 64, 128 or 256 columns (blocks of one entry are padded: 80 bytes for 64 columns).
constexpr int packed_tile_bytes(int dim) { return kKeys * (dim <= 64 ? 80 : dim <= 128 ? 144 : 288); }

__device__ __forceinline__ void cp_async_n(uint32_t dst, const void* src, int bytes) {
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The places for tiles, and the warps that fill them.  A wait by parity needs the barrier's phase before to be known to be over,
// and the next one not to come before the wait is done.  So tile g has place g % NS, and a place is always loaded by the same
// warp (g % NL, NS a multiple of NL) and taken by the same ones.
template <int NS, int NL, int TILE>
struct PackedStage {
  static_assert(NS % NL == 0, "a place belongs to one loading warp");
  static constexpr int kTile = TILE;
  static constexpr int kInfo = NS * TILE;                        // uint32 [NS][8]: four valid words, four bad
  static constexpr int kBars = kInfo + NS * 8 * 4;               // full, empty [NS]
  static constexpr int kBytes = (kBars + 2 * NS * 8 + 127) / 128 * 128;

  char* mem;
  uint32_t base;

  __device__ explicit PackedStage(char* at) : mem(at), base(smem_addr(at)) {}
  __device__ uint32_t full(uint32_t g) const { return base + kBars + g % NS * 8; }
  __device__ uint32_t empty(uint32_t g) const { return base + kBars + (NS + g % NS) * 8; }
  __device__ static uint32_t phase(uint32_t g) { return g / NS & 1; }
  __device__ char* tile(uint32_t g) const { return mem + g % NS * TILE; }
  __device__ uint32_t* info(uint32_t g) const { return reinterpret_cast<uint32_t*>(mem + kInfo) + g % NS * 8; }

  // By one thread.  empties: arrivals that free a place.
  __device__ void init(int empties) const {
    for (int i = 0; i < NS; ++i) mbar_init(full(i), 64), mbar_init(empty(i), empties);
  }

  // Loading warp lw.  plan: the warps' way along the line of tiles.
  template <class Plan>
  __device__ void load(Plan& plan, const AttnParams& p, const PackedTiles& k, int lw) const {
    if (k.rows_log >= 2)
      load_tiles<1>(plan, p, k, lw);
    else
      load_tiles<4>(plan, p, k, lw);
  }

  // WORDS: pages that a lane has of a tile: one where the blocks are 32 at most, each of them a bulk copy; four of blocks of one
  // or two entries, which are copied 16 bytes a lane.
  template <int WORDS, class Plan>
  __device__ __forceinline__ void load_tiles(Plan& plan, const AttnParams& p, const PackedTiles& k, int lw) const {
    const PackedView& c = k.c;
    const int lane = threadIdx.x & 31;
    const int code_row = c.head_dim / 2, scale_row = c.head_dim / 16;
    const int blocks = kKeys >> k.rows_log;
    // (a block of one copy has the cache's padding, of four it has none)
    const int bytes = k.copies == 1 ? k.block : kKeys * (code_row + scale_row) * 2;
    AttnSegment s{};
    bool more = plan.next(s);
    int t = s.t0 + lw;       // this warp's next tile, if the segment has that many, and its number
    uint32_t g = lw;
    uint32_t gathered = 0u;  // places whose tile before had gathered rows: a bit each
    uint32_t last = 0;       // tiles up to this warp's last one
    // A tile, and the pages of its blocks lane, lane + 32, ...: the table's words are on their way a tile ahead, and are not
    // touched before they are needed.
    struct Tile {
      int32_t page[WORDS];
      uint32_t g;
      int x0, keys, hist, hkv, b;  // keys from x0 on, the committed ones among them; keys 0: no more tiles
      int64_t row0;
    };
    auto ahead = [&](Tile& a) {
      a.keys = 0;
      while (more && t >= s.t0 + s.cnt) {
        const int past = t - s.t0 - s.cnt;
        more = plan.next(s);
        t = s.t0 + past;
      }
      if (!more) return;
      a.g = g, a.x0 = t * kKeys, a.hkv = s.hkv, a.b = s.b, a.row0 = s.r.row0;
      a.keys = s.r.len + s.r.n - a.x0, a.hist = s.r.len - a.x0;
      const uint32_t first = divide(static_cast<uint32_t>(a.x0), c.div_mul, c.div_shift);
      const int32_t* table = c.table + a.b * c.ld_table + first;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        const int n = i * 32 + lane;
        a.page[i] = -1;
        if (n < blocks && (n << k.rows_log) < a.keys && first + n < static_cast<uint32_t>(c.max_pages)) a.page[i] = table[n];
      }
      t += NL, g += NL;
    };
    Tile now;
    ahead(now);
    while (now.keys > 0) {
      const Tile a = now;
      ahead(now);
      // (rows that lie apart: the request's last tiles', or all)
      const bool apart = k.copies == 0 || (p.row_slots && a.hist < kKeys && a.keys > a.hist);
      uint32_t found[WORDS];
#pragma unroll
      for (int i = 0; i < WORDS; ++i) found[i] = __ballot_sync(0xffffffffu, a.page[i] >= 0 && a.page[i] < c.pages);
      const uint32_t place = a.g % NS, to = base + place * TILE, bar = full(a.g), bit = 1u << place;
      if (a.g >= NS && !plan.wait(empty(a.g), phase(a.g - NS))) break;
      last = a.g + 1;
      if (gathered & bit) fence_async();  // what lanes wrote here, before bulk copies go over it (after the wait, by those that copy)
      gathered = apart || WORDS > 1 ? gathered | bit : gathered & ~bit;
      if (apart) {
        load_apart(p, k, a.b, a.x0, a.keys, a.hist, a.hkv, a.row0, to, bar, info(a.g));
        continue;
      }
      // All in blocks.  Keys that are there: lane w < 4 has word w of them.
      const int upto = a.keys - (lane & 3) * 32;
      const uint32_t range = upto >= 32 ? 0xffffffffu : upto <= 0 ? 0u : (1u << upto) - 1u;
      uint32_t good = range;
      const int need = min(blocks, (a.keys + (1 << k.rows_log) - 1) >> k.rows_log);  // blocks with keys
      int have = 0;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) have += __popc(found[i]);
      if (have < need) {
#pragma unroll 1
        for (int x = 0; x < 32; ++x) {
          const int n = ((lane & 3) * 32 + x) >> k.rows_log;
          uint32_t word = found[0];
#pragma unroll
          for (int i = 1; i < WORDS; ++i) word = n >> 5 == i ? found[i] : word;
          if (!(word >> (n & 31) & 1u)) good &= ~(1u << x);
        }
      }
      if (lane < 4) info(a.g)[lane] = good, info(a.g)[4 + lane] = range & ~good;
      const char* head = c.data + a.hkv * c.head_stride;
      if (WORDS > 1) {
        const int each = k.block / 16;
        const uint32_t mul = ((1u << 20) + each - 1) / each;  // exact for x below 2^20 / each: each at most 36, x 2335
#pragma unroll 2
        for (int y = 0; y < need * each; y += 32) {
          const int x = y + lane, n = static_cast<int>(x * mul >> 20);
          int32_t page = -1;
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            const int32_t v = __shfl_sync(0xffffffffu, a.page[i], n & 31);
            if (n >> 5 == i && (found[i] >> (n & 31) & 1u)) page = v;
          }
          if (page >= 0) cp_async16(to + x * 16, head + page * c.page_stride + (x - n * each) * 16, true);
        }
        cp_async_arrive(bar);  // when this lane's copies are in place
        mbar_arrive(bar);
        __syncwarp();
        continue;
      }
      if (lane == 0 && have > 0) mbar_expect_tx(bar, static_cast<uint32_t>(have * bytes));
      __syncwarp();
      if (k.copies == 1) {
        if (found[0] >> lane & 1u) bulk_copy_g2s(to + lane * k.block, head + a.page[0] * c.page_stride, bytes, bar);
      } else if (have > 0) {  // a part of one page: its four arrays, a lane each
        const char* from = head + __shfl_sync(0xffffffffu, a.page[0], 0) * c.page_stride;
        const int in = static_cast<int>(static_cast<uint32_t>(a.x0) -
                                        divide(static_cast<uint32_t>(a.x0), c.div_mul, c.div_shift) * c.page_size);
        const int n_code = kKeys * code_row, n_scale = kKeys * scale_row;
        if (lane < 4) {
          const int at = lane == 0 ? 0 : lane == 1 ? packed_v_codes(c.page_size, c.head_dim)
                         : lane == 2 ? packed_k_scales(c.page_size, c.head_dim) : packed_v_scales(c.page_size, c.head_dim);
          const int dst = lane == 0 ? 0 : lane == 1 ? n_code : lane == 2 ? 2 * n_code : 2 * n_code + n_scale;
          bulk_copy_g2s(to + dst, from + at + static_cast<int64_t>(in) * (lane < 2 ? code_row : scale_row), lane < 2 ? n_code : n_scale,
                        bar);
        }
      }
      if (lane == 0) mbar_arrive_times(bar, 64);
      __syncwarp();
    }
    // Copies in flight end before the block does.
    cp_async_commit();
    cp_async_wait<0>();
    if (*plan.abort())
      for (uint32_t i = last > NS ? last - NS : 0; i < last; ++i)
        if (static_cast<int>(i % NL) == lw)
          for (int n = 0; n < 100 && !mbar_try_wait_for(full(i), phase(i), 10000); ++n) {
          }
  }

  // A tile of which rows lie apart: blocks of the history that are whole, and the rest row by row.
  __device__ __noinline__ void load_apart(const AttnParams& p, const PackedTiles& k, int b, int x0, int keys, int hist, int hkv, int64_t row0,
                                          uint32_t to, uint32_t bar, uint32_t* words) const {
    const PackedView& c = k.c;
    const int lane = threadIdx.x & 31, rows = 1 << k.rows_log;
    const int code_row = c.head_dim / 2, scale_row = c.head_dim / 16, unit = scale_row & -scale_row;
    const int whole = k.copies == 1 ? min(max(hist, 0), kKeys) & ~(rows - 1) : 0;
    AttnRequest r{};
    r.row0 = row0, r.len = x0 + hist, r.n = keys - hist;
    const char* head = c.data + hkv * c.head_stride;
    Place at[4];
    uint32_t good[4], bad[4], boxes[4], rest = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = i * 32 + lane;
      at[i] = packed_place(p, c, r, x0 + x, key_word(p, r, b, x0 + x));
      const bool there = at[i].page >= 0;
      good[i] = __ballot_sync(0xffffffffu, there);
      bad[i] = __ballot_sync(0xffffffffu, x < keys && !there);
      boxes[i] = __ballot_sync(0xffffffffu, there && x < whole && (x & (rows - 1)) == 0);
      if (there && x >= whole) rest |= 1u << i;
    }
    if (lane < 4) {
      words[lane] = lane == 0 ? good[0] : lane == 1 ? good[1] : lane == 2 ? good[2] : good[3];
      words[4 + lane] = lane == 0 ? bad[0] : lane == 1 ? bad[1] : lane == 2 ? bad[2] : bad[3];
    }
    const int count = __popc(boxes[0]) + __popc(boxes[1]) + __popc(boxes[2]) + __popc(boxes[3]);
    if (lane == 0 && count > 0) mbar_expect_tx(bar, static_cast<uint32_t>(count * k.block));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (boxes[i] >> lane & 1u)
        bulk_copy_g2s(to + ((i * 32 + lane) >> k.rows_log) * k.block, head + at[i].page * c.page_stride, k.block, bar);
    // A key's pieces: 16 bytes of codes, `size` of scales, of K and then of V.
    const int size = unit > 16 ? 16 : unit, n_code = code_row / 16, n_scale = scale_row / size, pieces = 2 * (n_code + n_scale);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int page = i == 0 ? at[0].page : i == 1 ? at[1].page : i == 2 ? at[2].page : at[3].page;
      const int in = i == 0 ? at[0].in : i == 1 ? at[1].in : i == 2 ? at[2].in : at[3].in;
      if (!__any_sync(0xffffffffu, rest >> i & 1u)) continue;
#pragma unroll 1
      for (int y = 0; y < pieces; ++y) {  // 32 keys' pieces: `pieces` turns of 32 lanes
        const int z = y * 32 + lane, key = z / pieces, piece = z - key * pieces;
        const int64_t kpage = __shfl_sync(0xffffffffu, page, key);
        const int kin = __shfl_sync(0xffffffffu, in, key);
        const bool mine = __shfl_sync(0xffffffffu, rest >> i & 1u, key) != 0u;
        if (!mine) continue;
        const int x = i * 32 + key, row = x & (rows - 1);
        const char* from = head + kpage * c.page_stride;
        const uint32_t dst = to + (x >> k.rows_log) * k.block;
        if (piece < 2 * n_code) {
          const int v = piece >= n_code, o = (piece - v * n_code) * 16;
          cp_async16(dst + (v ? packed_v_codes(rows, c.head_dim) : 0) + row * code_row + o,
                     from + (v ? packed_v_codes(c.page_size, c.head_dim) : 0) + static_cast<int64_t>(kin) * code_row + o, true);
        } else {
          const int q = piece - 2 * n_code, v = q >= n_scale, o = (q - v * n_scale) * size;
          const uint32_t d = dst + (v ? packed_v_scales(rows, c.head_dim) : packed_k_scales(rows, c.head_dim)) + row * scale_row + o;
          const char* f = from + (v ? packed_v_scales(c.page_size, c.head_dim) : packed_k_scales(c.page_size, c.head_dim)) +
                          static_cast<int64_t>(kin) * scale_row + o;
          if (size >= 4)
            cp_async_n(d, f, size);
          else
            *reinterpret_cast<uint16_t*>(mem + (d - base)) = *reinterpret_cast<const uint16_t*>(f);
        }
      }
    }
    cp_async_arrive(bar);  // when this lane's copies are in place
    mbar_arrive(bar);
    __syncwarp();
  }
};

// The way along the line of tiles without a ring of whole numbers (as in KvRing): a warp walks it ahead of the others.
struct PlanQueue {
  static constexpr int kPlan = 0;  // AttnSegment [kPlans]
  static constexpr int kBars = kPlan + kPlans * static_cast<int>(sizeof(AttnSegment));  // plan, read [kPlans], q, q free [2]
  static constexpr int kWarps = 16;                           // of a block, at most
  static constexpr int kSums = kBars + (2 * kPlans + 4) * 8;  // int64: sums [2 kWarps], find [2]
  static constexpr int kAbort = kSums + (2 * kWarps + 2) * 8;
  static constexpr int kBytes = (kAbort + 16 + 127) / 128 * 128;

  char* mem;
  uint32_t base;
  int lane;
  uint32_t plans;

  __device__ explicit PlanQueue(char* at) : mem(at), base(smem_addr(at)), lane(threadIdx.x & 31), plans(0) {}
  __device__ uint32_t plan_bar(uint32_t i) const { return base + kBars + i % kPlans * 8; }
  __device__ uint32_t read_bar(uint32_t i) const { return base + kBars + (kPlans + i % kPlans) * 8; }
  __device__ uint32_t q_bar(int i) const { return base + kBars + (2 * kPlans + i) * 8; }
  __device__ uint32_t q_free(int i) const { return base + kBars + (2 * kPlans + 2 + i) * 8; }
  __device__ AttnSegment* plan_slot(uint32_t i) const { return reinterpret_cast<AttnSegment*>(mem + kPlan) + i % kPlans; }
  __device__ int64_t* sums() const { return reinterpret_cast<int64_t*>(mem + kSums); }
  __device__ int64_t* find() const { return sums() + 2 * kWarps; }
  __device__ volatile int* abort() const { return reinterpret_cast<volatile int*>(mem + kAbort); }

  // By one thread.  readers: warps that read the plan, q_frees: arrivals that free a Q.
  __device__ void init(int readers, int q_frees) const {
    for (int i = 0; i < kPlans; ++i) mbar_init(plan_bar(i), 1), mbar_init(read_bar(i), readers);
    for (int i = 0; i < 2; ++i) mbar_init(q_bar(i), 32), mbar_init(q_free(i), q_frees);
    *abort() = 0;
  }
  // A wait that gives up ends every role; the lanes of a warp leave together.
  __device__ bool wait_one(uint32_t bar, uint32_t parity) const {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait_for(bar, parity, 10000)) return true;
    return wait_on(bar, parity, abort());
  }
  __device__ bool wait(uint32_t bar, uint32_t parity) const { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; }
  __device__ bool next(AttnSegment& s) {
    if (!wait(plan_bar(plans), plans / kPlans & 1)) return false;
    s = *plan_slot(plans);
    __syncwarp();
    if (lane == 0) mbar_arrive(read_bar(plans));
    ++plans;
    return s.cnt > 0;
  }
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
  // At the end, by every thread after the block's last barrier (never expected: see SV_DEV_TIMEOUT).
  __device__ void report_abort(const AttnParams& p) const {
    if (threadIdx.x == 0) atomicExch(p.err, 1u);
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x) p.status[b] = kStTimeout;
  }
};

cudaError_t launch_packed_attention_few(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_packed_attention_wide(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace sv
