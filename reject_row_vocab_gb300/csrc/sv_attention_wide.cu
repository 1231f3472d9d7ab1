// Attention over the paged cache for many query rows, on the fifth-generation
// tensor cores: bf16, heads of up to 128, tiles of 128 rows and 128 keys.
//
//   S = Q K^T (128 x 128, tensor memory)     one thread issues the products
//   P = 2^(c S - m), l += sum P              one thread a row: no exchange
//   O += P V  (P from tensor memory)         accumulated in tensor memory
//
// Four softmax warps, four loading warps, one warp that issues the matrix
// instructions, one that loads the next unit's Q and one that walks the line
// of tiles ahead of them all, connected by mbarriers.  The loading warps gather K and V rows
// through the page table with 16-byte asynchronous copies into a ring of
// tiles in the 128-byte swizzle the matrix unit reads, and run ahead over the
// ends of units.  S has two buffers, so the next tile's scores are computed
// while this one's weights are taken; P overwrites its own S.  The reference m
// moves (and O is rescaled) only when a row's maximum has grown by more than
// 2^8: the weights stay below 2^8, the sums in fp32, and the result does not
// depend on the reference.
//
// Units that several blocks share are joined by a second kernel, spread over
// the whole GPU: two long requests leave 19 parts of a unit, which its last
// block alone took 35 us to join.
//
// Every wait is bounded; a wait that gives up raises SV_DEV_TIMEOUT, lets all
// warps leave, and the block frees its tensor memory.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>
#include <mutex>

#include <cuda.h>

#include "sv_attention.cuh"

namespace sv {
namespace {

constexpr int kRows = 128, kKeys = 128;  // a tile
constexpr int kSoftmaxThreads = 128, kLoadThreads = 128;
constexpr int kWideThreads = kSoftmaxThreads + kLoadThreads + 96;  // and a warp each to issue, to load Q, to plan
constexpr int kReaders = 10;      // warps that read the plan
constexpr int kUnitPlaces = 1;  // what a unit costs beside its key tiles, in tiles
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kSlack = 8.0f;  // log2 units a row's maximum may pass its reference by

// ---------------------------------------------------------------------------------------------------------------------
// Tensor memory and matrix instructions
// ---------------------------------------------------------------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of the calling warp's 32 lanes: one row's values a thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand in the 128-byte swizzle.  Stride: bytes between groups of eight rows (1024); lead: bytes between
// 64-element blocks of the contiguous axis (used where that axis is the operand's M or N).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>((lead >> 4) & 0x3fffu) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32, 128 rows, n columns; b_mn: B's contiguous axis is N (V as it lies), not K.
__host__ __device__ constexpr uint32_t instruction(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kRows >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {  // NaN and infinities replaced by 0
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
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

// As mbar_try_wait, the thread suspended for up to about `ns`.
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

// The rest of a wait that did not end at once.  Suspended meanwhile: warps that poll take issue slots from those that
// work.  (Out of line, like all that seldom runs: what the roles run by turns has to stay in the instruction cache.)
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_for(bar, parity, 10000)) return true;
  if (mbar_wait_bounded(bar, parity, abort, kWaitNs)) return true;
  *abort = 1;
  return false;
}

// An arrival that the thread's earlier asynchronous copies make, once they are complete.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The sum of the NaN and infinite values that new row i sees of columns d .. d + 3 of the segment's new rows' V.
__device__ __noinline__ float4 nonfinite_seen(const AttnParams& p, const AttnSegment& s, int i, int d) {
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < s.r.n; ++j) {
    const int x = s.r.len + j;
    if (x < s.t0 * kKeys || x >= (s.t0 + s.cnt) * kKeys || !row_sees(p, s.b, i, j)) continue;
    const int64_t off = key_offset(p, s.r, x, key_word(p, s.r, s.b, x));
    if (off < 0) continue;
    const uint16_t* v = reinterpret_cast<const uint16_t*>(p.c.v) + off + s.hkv * p.c.head_stride + d;
    for (int k = 0; k < 4 && d + k < p.c.head_dim; ++k) {
      const float x = __uint_as_float(static_cast<uint32_t>(v[k]) << 16);
      if (!(fabsf(x) < kInfF)) f[k] += x;
    }
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}

// ---------------------------------------------------------------------------------------------------------------------
// Layout
// ---------------------------------------------------------------------------------------------------------------------

template <int DP>
struct Wide {
  static constexpr int kBlock = kKeys * 128;          // 128 rows of 64 elements
  static constexpr int kTile = kBlock * (DP / 64);    // a K or V tile, or Q
  static constexpr int kRing = DP == 128 ? 6 : 8;     // tiles in the ring
  static constexpr int kInfo = 8;                     // tiles whose validity is kept
  static constexpr int kPieces = DP / 8;              // 16-byte pieces of a row
  static constexpr int kS = 0, kO = 256;              // tensor memory columns: two S of 128, then O
  // shared memory
  static constexpr int kQ = 0;
  static constexpr int kTiles = kTile;
  static constexpr int kValid = kTiles + kRing * kTile;     // uint32 [kInfo][8]: four valid words, four bad
  static constexpr int kPlan = kValid + kInfo * 8 * 4;       // AttnSegment [kPlans]
  static constexpr int kPlans = 4;
  static constexpr int kBars = kPlan + kPlans * static_cast<int>(sizeof(AttnSegment));
  // full, empty [kRing], s, p, q, q free, pv [2], soft, (pad), plan, plan free [kPlans]
  static constexpr int kMisc = kBars + (2 * kRing + 12 + 2 * kPlans) * 8;  // sums [22], find [2]; tmem, abort, careful
  static constexpr int kSmem = kMisc + 24 * 8 + 4 * 4;
  // 16-byte piece c of row r of a tile
  __device__ static uint32_t piece(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  }
};

template <int DP>
__global__ void __launch_bounds__(kWideThreads, 1)
    k_attention_wide(const AttnParams p, const __grid_constant__ KvMaps maps) {
  using W = Wide<DP>;
  constexpr int NB = W::kRing;
  extern __shared__ __align__(1024) char smem[];
  const uint32_t base = smem_addr(smem);
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(smem + W::kValid);
  int64_t* s_sum = reinterpret_cast<int64_t*>(smem + W::kMisc);
  int64_t* s_find = s_sum + 22;
  int* s_misc = reinterpret_cast<int*>(s_find + 2);
  volatile int* s_abort = s_misc + 1;
  volatile int* s_careful = s_misc + 2;
  AttnSegment* s_plan = reinterpret_cast<AttnSegment*>(smem + W::kPlan);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  auto bar_full = [&](int i) { return base + W::kBars + i * 8; };
  auto bar_empty = [&](int i) { return base + W::kBars + (NB + i) * 8; };
  auto bar_s = [&](int i) { return base + W::kBars + (2 * NB + i) * 8; };
  auto bar_p = [&](int i) { return base + W::kBars + (2 * NB + 2 + i) * 8; };
  auto bar_q = [&](int i) { return base + W::kBars + (2 * NB + 4 + i) * 8; };
  auto bar_qfree = [&](int i) { return base + W::kBars + (2 * NB + 6 + i) * 8; };
  // Two, in turn: a wait by parity is only good where the barrier's phase before is known to be over, and that S(g) has
  // come means that O has the products of tile g - 2, not those of g - 1.
  auto bar_pv = [&](uint32_t g) { return base + W::kBars + (2 * NB + 8 + (g & 1)) * 8; };
  const uint32_t bar_soft = base + W::kBars + (2 * NB + 10) * 8;
  auto bar_plan = [&](int i) { return base + W::kBars + (2 * NB + 12 + i) * 8; };
  auto bar_read = [&](int i) { return base + W::kBars + (2 * NB + 12 + W::kPlans + i) * 8; };
  // Units of up to 64 rows have two Qs, one in each half of Q's rows: the products of the lower half read on into what
  // lies behind it, but rows past 64 are nobody's then.
  const int twin = p.max_len * static_cast<int64_t>(p.group) <= 64 ? 1 : 0;
  auto q_slot = [&](uint32_t unit) { return twin ? static_cast<int>(unit & 1) : 0; };
  auto q_phase = [&](uint32_t unit) { return twin ? unit >> 1 : unit; };

  if (t == 0) {
    for (int i = 0; i < NB; ++i) mbar_init(bar_full(i), kLoadThreads), mbar_init(bar_empty(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar_s(i), 2), mbar_init(bar_p(i), kSoftmaxThreads);
    for (int i = 0; i < 2; ++i) mbar_init(bar_pv(i), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar_q(i), 32), mbar_init(bar_qfree(i), 1);
    mbar_init(bar_soft, kSoftmaxThreads);
    for (int i = 0; i < W::kPlans; ++i) mbar_init(bar_plan(i), 1), mbar_init(bar_read(i), kReaders);
    mbar_fence_init();
    *s_abort = 0;
    *s_careful = 0;
  }
  if (warp == 8) {
    tmem_alloc(base + W::kMisc + 24 * 8, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_misc[0]);

  grid_dependency_wait();
  allow_dependents();
  const AttnSpan span = attn_span<kRows, kKeys, kUnitPlaces, kWideThreads>(p, t, s_sum, s_find, [] { __syncthreads(); });
  // A wait that gives up ends every role; the lanes of a warp leave together.
  auto wait_one = [&](uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_on(bar, parity, s_abort);
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; };

  // The next segment of the plan, for a whole warp (or the issuing thread alone); false at the end, or after a wait that
  // gave up.
  uint32_t plans = 0;
  auto next = [&](AttnSegment& s, auto waiter) {
    const int slot = plans % W::kPlans;
    if (!waiter(bar_plan(slot), (plans / W::kPlans) & 1)) return false;
    s = s_plan[slot];
    __syncwarp(__activemask());
    if (lane == 0) mbar_arrive(bar_read(slot));
    ++plans;
    return s.cnt > 0;
  };

  if (warp == 10) {
    // ---- The plan: the block's segments in order, a few ahead of their readers; one without tiles ends it.
    if (lane == 0) {
      AttnWalk<kRows, kKeys, kUnitPlaces> walk(p, span);
      AttnSegment s{};
      for (bool more = true; more; ++plans) {
        more = walk.next(s);
        if (!more) s.cnt = 0;
        const int slot = plans % W::kPlans;
        if (plans >= W::kPlans && !wait_one(bar_read(slot), (plans / W::kPlans - 1) & 1)) break;
        s_plan[slot] = s;
        mbar_arrive(bar_plan(slot));
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ---- Loading warps: tile g's K is group 2 g of the ring, its V group 2 g + 1.  A warp has 32 of a tile's keys, a
    // lane one key's place, handed round by shuffles; the word that places a lane's key of the next tile is on its way
    // while this tile is copied.
    const int lw = warp - 4;
    AttnSegment s{};
    bool more = next(s, wait);
    int tile = s.t0;
    int64_t word = more ? key_word(p, s.r, s.b, tile * kKeys + lw * 32 + lane) : -1;
    uint32_t q = 0;  // groups issued
    bool ok = true;
    const int c = lane % W::kPieces, sub = lane / W::kPieces;
    constexpr int kStep = 32 / W::kPieces;  // rows a warp copies at once
    const bool in_head = c * 8 < p.c.head_dim;
    while (more && ok) {
      const int x = tile * kKeys + lw * 32 + lane;
      const int64_t off = key_offset(p, s.r, x, word);
      const uint32_t valid = __ballot_sync(0xffffffffu, off >= 0);
      const uint32_t bad = __ballot_sync(0xffffffffu, x < s.r.len + s.r.n && off < 0);
      // a tile of history in boxes: this lane's box of the warp's 32 keys
      const bool boxes = maps.rows > 0 && (tile + 1) * kKeys <= s.r.len;
      const int per = boxes ? 32 / maps.rows : 1;
      const int box_row = boxes ? lane % per * maps.rows : 0, box_col = boxes ? lane / per : 0;
      const int box_head = s.hkv;
      const int64_t box_page = __shfl_sync(0xffffffffu, word, box_row);
      const uint32_t box_key = static_cast<uint32_t>(tile * kKeys + lw * 32 + box_row);
      const uint32_t box_in = box_key - divide(box_key, p.c.div_mul, p.c.div_shift) * p.c.page_size;
      const int64_t shift = (static_cast<int64_t>(s.hkv) * p.c.head_stride + c * 8) * 2;
      if (++tile >= s.t0 + s.cnt) {
        more = next(s, wait);
        tile = s.t0;
      }
      if (more) word = key_word(p, s.r, s.b, tile * kKeys + lw * 32 + lane);
      const uint32_t g = q >> 1;
#pragma unroll 1
      for (int which = 0; which < 2; ++which, ++q) {
        if (q >= NB && !wait(bar_empty(q % NB), (q / NB - 1) & 1)) {
          ok = false;
          break;
        }
        if (which == 0 && lane == 0) {
          s_valid[(g % W::kInfo) * 8 + lw] = valid;
          s_valid[(g % W::kInfo) * 8 + 4 + lw] = bad;
        }
        if (boxes) {
          // (a page outside the cache is outside the tensor: the box is filled with zeros)
          if (lane == 0)
            mbar_arrive_expect_tx(bar_full(q % NB), 32 * 128 * (DP / 64));
          else
            mbar_arrive(bar_full(q % NB));
          __syncwarp();
          if (box_col < DP / 64)
            box_copy(base + W::kTiles + (q % NB) * W::kTile + box_col * W::kBlock + (lw * 32 + box_row) * 128,
                     which ? &maps.v : &maps.k, box_col * 64, box_head, static_cast<int>(box_in),
                     static_cast<int>(box_page), bar_full(q % NB));
          continue;
        }
        const char* src = (which ? p.c.v : p.c.k) + shift;
        const uint32_t dst = base + W::kTiles + (q % NB) * W::kTile;
#pragma unroll 8
        for (int i = 0; i < 32; i += kStep) {
          const int64_t o = __shfl_sync(0xffffffffu, off, i + sub);
          const bool live = o >= 0 && in_head;
          cp_async16(dst + W::piece(lw * 32 + i + sub, c), live ? src + o * 2 : p.c.k, live);
        }
        cp_async_arrive(bar_full(q % NB));  // when this thread's copies so far are in place
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    if (*s_abort)  // copies in flight end before the block does
      for (uint32_t i = q > NB ? q - NB : 0; i < q; ++i)
        for (int n = 0; n < 100 && !mbar_try_wait_for(bar_full(i % NB), (i / NB) & 1, 10000); ++n) {
        }
  } else if (warp == 9) {
    // ---- Q of the next unit, as soon as this unit's last scores are done.  Rows that do not exist are 0.
    AttnSegment s;
    for (uint32_t units = 0; next(s, wait); ++units) {
      const int slot = q_slot(units);
      if (q_phase(units) > 0 && !wait(bar_qfree(slot), (q_phase(units) - 1) & 1)) break;
      const int rows = s.r.n * p.group - s.rt * kRows;
      const int warps = min(kRows, (rows + 31) & ~31);  // rows of the warps that have any
      const int c = lane % W::kPieces, sub = lane / W::kPieces;
      const bool in_head = c * 8 < p.c.head_dim;
      for (int r0 = 0; r0 < warps; r0 += 32) {  // a lane finds one row's place, the warp copies the 32 of them
        const int grow = s.rt * kRows + r0 + lane, i = grow / p.group;
        const int64_t at = r0 + lane < rows
                               ? (s.r.row0 + i) * p.q_row + (s.hkv * p.group + grow - i * p.group) * p.q_head
                               : -1;
#pragma unroll 8
        for (int j = 0; j < 32; j += 32 / W::kPieces) {
          const int64_t o = __shfl_sync(0xffffffffu, at, j + sub);
          const bool live = o >= 0 && in_head;
          cp_async16(base + W::kQ + W::piece(slot * 64 + r0 + j + sub, c), live ? p.q + (o + c * 8) * 2 : p.q, live);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_async();
      mbar_arrive(bar_q(slot));
    }
    cp_async_wait<0>();
  } else if (warp == 8) {
    // ---- The issuing thread.
    if (lane == 0) {
      AttnSegment s;
      uint32_t g = 0, units = 0;
      bool ok = true;
      auto scores = [&](uint32_t n, bool last) {
        const int slot = q_slot(units);
        const uint32_t group = 2 * n;
        if (!wait_one(bar_full(group % NB), (group / NB) & 1)) return false;
        fence_async();  // the copies wrote through the generic proxy, the products read through the asynchronous one
        tc_fence_after();
        mbar_arrive(bar_s(n & 1));  // hands the tile's validity on
        const uint32_t k = base + W::kTiles + (group % NB) * W::kTile;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          const uint32_t at = (i >> 2) * W::kBlock + (i & 3) * 32;
          mma_ss(tmem + W::kS + (n & 1) * 128, operand(base + W::kQ + slot * 64 * 128 + at, 16), operand(k + at, 16),
                 instruction(kKeys, false), i > 0);
        }
        tc_commit(bar_empty(group % NB));
        tc_commit(bar_s(n & 1));
        if (last) tc_commit(bar_qfree(slot));
        return true;
      };
      while (ok && next(s, wait_one)) {
        if (!wait_one(bar_q(q_slot(units)), q_phase(units) & 1)) break;
        tc_fence_after();
        ok = scores(g, s.cnt == 1);
        for (int i = 0; ok && i < s.cnt; ++i) {
          const uint32_t n = g + i, group = 2 * n + 1;
          if (i + 1 < s.cnt && !scores(n + 1, i + 2 == s.cnt)) {
            ok = false;
            break;
          }
          if (!wait_one(bar_full(group % NB), (group / NB) & 1) || !wait_one(bar_p(n & 1), (n >> 1) & 1)) {
            ok = false;
            break;
          }
          fence_async();
          tc_fence_after();
          const uint32_t v = base + W::kTiles + (group % NB) * W::kTile;
#pragma unroll
          for (int j = 0; j < kKeys / 16; ++j)
            mma_ts(tmem + W::kO, tmem + W::kS + (n & 1) * 128 + j * 8, operand(v + j * 2048, W::kBlock),
                   instruction(DP, true), i > 0 || j > 0);
          tc_commit(bar_empty(group % NB));
          tc_commit(bar_pv(n));
        }
        g += s.cnt;
        ++units;
      }
    }
    __syncwarp();
  } else {
    // ---- Softmax warps: thread t has row t of the unit's tile.
    uint32_t meets = 0;
    auto meet = [&] {  // a barrier of the softmax warps, bounded like every wait
      mbar_arrive(bar_soft);
      wait(bar_soft, meets++ & 1);
    };
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const float c = fmaxf(p.scale_log2, 1e-30f);  // a scale of 0 by one too small to tell: 0 times a masked -inf is NaN
    AttnSegment s;
    uint32_t g = 0;
    bool ok = true, left = false;  // left: a unit that goes on behind this block
    while (ok && next(s, wait)) {
      const int rows = s.r.n * p.group - s.rt * kRows;  // rows of the unit from this tile on
      const bool idle = warp * 32 >= rows;              // none of the warp's rows exists
      const int my_row = (s.rt * kRows + t) / p.group;  // new row of this thread
      float m = -kInfF, l = 0.0f;
      uint32_t bad = 0u;
      bool mixed = false;  // a tile whose keys some rows see and others do not
      for (int i = 0; i < s.cnt; ++i, ++g) {
        const int x0 = (s.t0 + i) * kKeys;
        const uint32_t st = tmem + lanes + W::kS + (g & 1) * 128;
        if (!wait(bar_s(g & 1), (g >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint4 vv = *reinterpret_cast<const uint4*>(s_valid + (g % W::kInfo) * 8);
        const uint4 vb = *reinterpret_cast<const uint4*>(s_valid + (g % W::kInfo) * 8 + 4);
        uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
        bad |= vb.x | vb.y | vb.z | vb.w;
        const bool masked = (vw[0] & vw[1] & vw[2] & vw[3]) != 0xffffffffu || x0 + kKeys > s.r.len;
        if (masked && s.r.n > 1 && x0 + kKeys > s.r.len) {
          // A weight of 0 does not silence a V that is NaN or infinite: such values of new rows are taken out of the
          // products here, and added to the rows that see them at the end.
          mixed = true;
          const uint32_t group = 2 * g + 1;
          if (!wait(bar_full(group % NB), (group / NB) & 1)) {
            ok = false;
            break;
          }
          char* v = smem + W::kTiles + (group % NB) * W::kTile;
          const int from = max(s.r.len - x0, 0);
          bool found = false;
          for (int x = from * W::kPieces + t; x < kKeys * W::kPieces; x += kSoftmaxThreads) {
            uint4* at = reinterpret_cast<uint4*>(v + W::piece(x / W::kPieces, x % W::kPieces));
            const uint4 u = *at;
            const uint4 f = make_uint4(finite_pair(u.x), finite_pair(u.y), finite_pair(u.z), finite_pair(u.w));
            if (f.x != u.x || f.y != u.y || f.z != u.z || f.w != u.w) {
              *at = f;
              found = true;
            }
          }
          if (found) *s_careful = 1;
          fence_async();
        }
        if (!idle) {
          if (masked) {  // what the row does not see of the tile becomes -inf, in place
#pragma unroll
            for (int w = 0; w < 4; ++w) vw[w] = row_sees_of(p, s.r, s.b, t < rows ? my_row : s.r.n, x0 + w * 32, vw[w]);
            uint32_t word = vw[0];
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              float v[32];
              tmem_ld32(st + h * 32, reinterpret_cast<uint32_t*>(v));
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = (word >> j & 1u) ? v[j] : -kInfF;
              tmem_st32(st + h * 32, reinterpret_cast<const uint32_t*>(v));
              word = h == 0 ? vw[1] : h == 1 ? vw[2] : vw[3];
            }
            tmem_wait_st();
          }
          // The scores are read twice, for the maximum and for the weights: 128 of them do not fit beside the rest.
          float mx[4] = {-kInfF, -kInfF, -kInfF, -kInfF};
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            float v[64];
            tmem_ld32(st + h * 64, reinterpret_cast<uint32_t*>(v));
            tmem_ld32(st + h * 64 + 32, reinterpret_cast<uint32_t*>(v) + 32);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 64; ++j) mx[j & 3] = fmax_nan(mx[j & 3], v[j]);
          }
          const float top = fmax_nan(fmax_nan(mx[0], mx[1]), fmax_nan(mx[2], mx[3])) * c;
          const bool grow = !(top <= m + kSlack);  // also a first finite maximum, and NaN
          if (i == 0) {
            m = top;
          } else if (__any_sync(0xffffffffu, grow)) {
            const float a = grow ? ex2_fast(m - top) : 1.0f;
            if (grow) m = top;
            l *= a;
            if (!wait(bar_pv(g - 1), ((g - 1) >> 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < DP / 32; ++h) {
              float o[32];
              tmem_ld32(tmem + lanes + W::kO + h * 32, reinterpret_cast<uint32_t*>(o));
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= a;
              tmem_st32(tmem + lanes + W::kO + h * 32, reinterpret_cast<const uint32_t*>(o));
            }
          }
          const float ref = m == -kInfF ? 0.0f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            float v[64];
            uint32_t pk[32];
            tmem_ld32(st + h * 64, reinterpret_cast<uint32_t*>(v));
            tmem_ld32(st + h * 64 + 32, reinterpret_cast<uint32_t*>(v) + 32);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float a = ex2_fast(fmaf(v[2 * j], c, -ref));
              const float b = ex2_fast(fmaf(v[2 * j + 1], c, -ref));
              sum[(2 * j) & 3] += a;
              sum[(2 * j + 1) & 3] += b;
              pk[j] = pack_bf16(a, b);
            }
            tmem_st32(st + h * 32, pk);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(bar_p(g & 1));
      }
      if (!ok) break;
      // The unit's last product is done: this thread's row of O.
      if (!wait(bar_pv(g - 1), ((g - 1) >> 1) & 1)) break;
      tc_fence_after();
      bool careful = false;
      if (mixed) {
        meet();
        careful = *s_careful != 0;
        meet();
        if (t == 0) *s_careful = 0;
      }
      bad = (bad ? kStSlotRange : 0u) | s.r.status;
      const bool whole = s.cnt == s.nt;
      using P = AttnPart<kRows, DP>;
      float* part = whole ? nullptr : attn_part<kRows, DP>(p, blockIdx.x, s.t0 == 0);
      const int head = s.hkv * p.group + (s.rt * kRows + t) % p.group;
      char* out = p.out + ((s.r.row0 + my_row) * p.o_row + head * p.o_head) * 2;
      const bool none = m == -kInfF;  // nothing seen, or only scores of -inf
      const float inv = none ? 0.0f : 1.0f / l;
      if (!idle) {
#pragma unroll 1
        for (int h = 0; h < DP / 32; ++h) {
          float o[32];
          tmem_ld32(tmem + lanes + W::kO + h * 32, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
          if (t < rows) {
            if (careful) {
#pragma unroll
              for (int d = 0; d < 32; d += 4) {
                const float4 f = nonfinite_seen(p, s, my_row, h * 32 + d);
                o[d] += f.x, o[d + 1] += f.y, o[d + 2] += f.z, o[d + 3] += f.w;
              }
            }
            if (whole) {
#pragma unroll
              for (int d = 0; d < 32; d += 8)
                if (h * 32 + d < p.c.head_dim) {
                  uint4 u = make_uint4(0u, 0u, 0u, 0u);
                  if (!none)
                    u = make_uint4(pack_bf16(o[d] * inv, o[d + 1] * inv), pack_bf16(o[d + 2] * inv, o[d + 3] * inv),
                                   pack_bf16(o[d + 4] * inv, o[d + 5] * inv), pack_bf16(o[d + 6] * inv, o[d + 7] * inv));
                  *reinterpret_cast<uint4*>(out + (h * 32 + d) * 2) = u;
                }
            } else {
#pragma unroll
              for (int d = 0; d < 32; d += 4)
                reinterpret_cast<float4*>(part)[(h * 8 + d / 4) * kRows + t] =
                    make_float4(o[d], o[d + 1], o[d + 2], o[d + 3]);
            }
          }
        }
      }
      if (whole) {
        if (t < rows && p.lse) p.lse[(s.r.row0 + my_row) * p.heads + head] = none ? -kInfF : fmaf(m, kLn2, logf(l));
        if (s.reports && t == 0) p.status[s.b] = bad | attn_timeout(p);
      } else {
        part[P::kM + t] = m;
        part[P::kL + t] = l;
        if (t == 0) {
          part[P::kStatus] = __uint_as_float(bad);
          if (s.t0 == 0) {
            left = true;
            *reinterpret_cast<AttnSplit*>(part + P::kSplit) =
                AttnSplit{s.r.row0, s.r.n, s.b, s.hkv, s.rt, attn_owner(span, s.u0 + s.nt - 1), s.reports ? 1 : 0, {}};
          }
        }
      }
      tc_fence_before();
    }
    if (t == 0 && !left)
      reinterpret_cast<AttnSplit*>(attn_part<kRows, DP>(p, blockIdx.x, true) + AttnPart<kRows, DP>::kSplit)->last = 0;
  }
  __syncthreads();
  if (*s_abort) {  // never expected: see SV_DEV_TIMEOUT
    if (t == 0) atomicExch(p.err, 1u);
    for (int b = t; b < p.batch; b += kWideThreads) p.status[b] = kStTimeout;
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Block (c, i): rows 16 i .. of the unit that begins in block c of the attention kernel and goes on behind it, if any.
constexpr int kJoinRows = 16;

template <int DP>
__global__ void __launch_bounds__(kJoinRows * DP / 8) k_attention_join(AttnParams p) {
  using P = AttnPart<kRows, DP>;
  constexpr int PARTS = 8, E = 2;  // parts in flight, quads of columns a thread
  grid_dependency_wait();
  allow_dependents();
  const int c0 = blockIdx.x, t = threadIdx.x;
  const float* first = attn_part<kRows, DP>(p, c0, true);
  const float* rest = attn_part<kRows, DP>(p, 0, false);
  const AttnSplit s = *reinterpret_cast<const AttnSplit*>(first + P::kSplit);
  if (s.last <= c0) return;
  auto part_of = [&](int c) { return c == c0 ? first : rest + static_cast<int64_t>(c) * 2 * P::kFloats; };
  const int row = blockIdx.y * kJoinRows + t % kJoinRows, quad = t / kJoinRows;
  const int grow = s.rt * kRows + row;
  if (blockIdx.y == 0 && t == 0 && s.reports) {
    uint32_t any = 0u;
    for (int c = c0; c <= s.last; ++c) any |= __float_as_uint(part_of(c)[P::kStatus]);
    p.status[s.b] = any | attn_timeout(p);
  }
  if (grow >= s.n * p.group) return;
  const int i = grow / p.group, head = s.hkv * p.group + grow - i * p.group;
  float4 a[E];
  float M = -kInfF, L = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int cb = c0; cb <= s.last; cb += PARTS) {
    float m[PARTS], l[PARTS];
    float4 v[PARTS][E];
#pragma unroll
    for (int j = 0; j < PARTS; ++j)
      if (cb + j <= s.last) {
        const float* q = part_of(cb + j);
        m[j] = q[P::kM + row], l[j] = q[P::kL + row];
#pragma unroll
        for (int e = 0; e < E; ++e) v[j][e] = reinterpret_cast<const float4*>(q)[(quad + e * (DP / 8)) * kRows + row];
      }
#pragma unroll
    for (int j = 0; j < PARTS; ++j) {
      if (cb + j > s.last) break;
      const float N = fmax_nan(M, m[j]), ref = N == -kInfF ? 0.0f : N;
      const float wa = ex2_fast(M - ref), wb = ex2_fast(m[j] - ref);
      M = N;
      L = fmaf(L, wa, l[j] * wb);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        a[e].x = fmaf(a[e].x, wa, v[j][e].x * wb), a[e].y = fmaf(a[e].y, wa, v[j][e].y * wb);
        a[e].z = fmaf(a[e].z, wa, v[j][e].z * wb), a[e].w = fmaf(a[e].w, wa, v[j][e].w * wb);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    write_row<true>(p, s.row0 + i, head, (quad + e * (DP / 8)) * 4, a[e], M, L);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  return fn;
}

// Boxes need pages of a multiple of eight rows (the swizzle's period); a layout the driver takes no map of has none.
KvMaps kv_maps(const KvView& c) {
  KvMaps m{};
  int rows = 32;
  while (rows >= 8 && c.page_size % rows != 0) rows /= 2;
  const EncodeTiledFn encode = encode_tiled();
  if (rows < 8 || !encode) return m;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.pages)};
  // an axis of one entry may come without a step
  auto step = [&](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s : (c.head_dim + 7) / 8 * 8) * 2; };
  const cuuint64_t strides[3] = {step(c.head_stride), step(c.slot_stride), step(c.page_stride)};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(rows), 1}, ones[4] = {1, 1, 1, 1};
  char* const base[2] = {c.k, c.v};
  CUtensorMap* const map[2] = {&m.k, &m.v};
  for (int i = 0; i < 2; ++i)
    if (encode(map[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base[i], dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return m;
  m.rows = rows;
  return m;
}

template <int DP>
cudaError_t launch(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  static std::mutex mu;
  static bool have[64] = {};
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!have[d]) {
      e = cudaFuncSetAttribute(k_attention_wide<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<DP>::kSmem);
      if (e != cudaSuccess) return e;
      have[d] = true;
    }
  }
  static_assert(Wide<DP>::kSmem <= 227 * 1024, "shared memory of a block");
  const int grid = dev.sms < kAttnMaxBlocks / 2 ? dev.sms : kAttnMaxBlocks / 2;  // parts are laid out for 64-row tiles
  e = launch_pdl(k_attention_wide<DP>, dim3(static_cast<unsigned>(grid)), dim3(kWideThreads), Wide<DP>::kSmem, stream, p,
                 kv_maps(p.c));
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.max_len) * p.group;
  const int slices = static_cast<int>(((rows < kRows ? rows : kRows) + kJoinRows - 1) / kJoinRows);
  return launch_pdl(k_attention_join<DP>, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(slices)),
                    dim3(kJoinRows * DP / 8), 0, stream, p);
}

}  // namespace

cudaError_t launch_attention_wide(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  return p.c.head_dim <= 64 ? launch<64>(p, dev, stream) : launch<128>(p, dev, stream);
}

}  // namespace sv
