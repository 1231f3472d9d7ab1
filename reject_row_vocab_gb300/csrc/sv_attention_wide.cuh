// Attention over the paged cache for many query rows, on the fifth-generation
// tensor cores: tiles of 128 rows and 128 keys.  Where the tiles come from is the
// Source: a bf16 cache's rows as they are (sv_attention_wide.cu, and what follows), or
// a 4-bit cache's values in half floats (sv_attention_packed_wide.cu).
//
//   S = Q K^T (128 x 128, tensor memory)     one warp issues the products
//   P = 2^(c (S - m)), l += sum P            one thread a row: no exchange
//   O += P V  (P from tensor memory)         accumulated in tensor memory
//
// Four softmax warps, four loading warps, one warp that issues the matrix
// instructions (a lane of it, with what they take in uniform registers: by one
// thread alone an instruction took 70 clocks to issue, about as long as to run),
// one that loads the next unit's Q and one that walks the line of tiles ahead of
// them all, connected by mbarriers.  The loading warps bring
// K and V through the page table into a ring of tiles in the 128-byte swizzle
// the matrix unit reads, and run ahead over the ends of units.  S has two
// buffers, so the next tile's scores are computed while this one's weights are
// taken; P overwrites its own S.  The reference m moves (and O is rescaled) only
// when a row's maximum has grown by more than 2^8: the weights stay below 2^8,
// the sums in fp32, and the result does not depend on the reference.
//
// The weights are rounded to bf16 for the product with V (its operands have one
// type); l sums the unrounded ones, in fp32.  That leaves an error of 0.0022 of
// the outputs' norm, where rounding the outputs alone leaves 0.0017.  Two bf16
// values a weight, as the kernel for few rows has, would give 0.0017 here too,
// but lengthen the softmax warps' chain: 64 requests of 16 rows took 131 us
// instead of 102, two long ones 70 instead of 64.  (Half floats: below.)
//
// Bound by the bytes of K and V where histories are long, by the chain from
// scores to weights to sums at each unit's ends where they are short.
// Measured: blocks of 16 rows of 64 requests of up to 4000, 32 heads of 128 on 8
// in the cache: 100 us, 5.7 TB/s; 32 requests, heads of 256: 107 us; 5 rows of
// two requests of 60000 to 100000: 63 us, 5.0 TB/s (17 of them outside the
// stream); trees of 17 nodes of 16 requests in pages of one slot: 21 us; a
// causal block of 1024 rows of one request: 72 us without history, 148 (513
// TFLOP/s) behind 4000, all key tiles gone through by every tile of rows.
//
// Units that several blocks share are joined by a second kernel, spread over
// the whole GPU.  (By the last of the unit's blocks alone, two long requests
// took 90 us instead of 63, a 64-request block 127 instead of 118.)
//
// Every wait is bounded; a wait that gives up raises SV_DEV_TIMEOUT, lets all
// warps leave, and the block frees its tensor memory.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#pragma once

#include <cstdint>
#include <mutex>

#include "sv_attention_ring.cuh"

namespace sv {
namespace {

constexpr int kRows = 128;  // query rows of a tile
constexpr int kSoftmaxThreads = 128;
// What a unit costs beside its key tiles, in tiles (1 to 5 measure alike: 101 to 102 us for the 64-request block, 21.5 to 23
// for the trees).
constexpr int kUnitPlaces = 2;
// log2 units a row's maximum may pass its reference by.  (A largest weight that is not 1 is rounded like the others: the error
// is 0.0022 of the outputs' norm with 8, 0.0020 with 2, 0.0019 with 0; blocks of 16 rows of 64 requests take 102, 105.6 and
// 107 us, two long requests 63 each.)
constexpr float kSlack = 8.0f;
constexpr float kNear = 128.0f;  // log2 units of a reference that its factor's rounding may be left in

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
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand in the 128-byte swizzle: its lower word, which a part of the operand `bytes` further on only adds
// bytes / 16 to, and the operand.  (One warp issues all products, so what it computes for each of them counts.)  Stride: bytes
// between groups of eight rows (1024); lead: bytes between 64-element blocks of the contiguous axis (used where that axis is the
// operand's M or N).
__device__ __forceinline__ uint32_t operand_at(uint32_t addr, uint32_t lead) { return (addr >> 4) + ((lead >> 4) << 16); }
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t bytes) {
  constexpr uint32_t kUpper = (1024u >> 4) | (1u << 14) | (2u << 29);
  return static_cast<uint64_t>(kUpper) << 32 | (at + (bytes >> 4));
}
constexpr uint32_t kNegateA = 1u << 13;
// bf16 x bf16 (or half x half) -> fp32, 128 rows, n columns; b_mn: B's contiguous axis is N (V as it lies), not K.
__host__ __device__ constexpr uint32_t instruction(int n, bool b_mn, bool half) {
  return (1u << 4) | (half ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kRows >> 4) << 24);
}
// By a whole warp, of which the lane with `issues` acts: so the compiler sees operands and control flow that are the same in all
// lanes, and keeps them in uniform registers, which is where the instruction takes them from.
__device__ __forceinline__ void mma_ss(bool issues, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(issues ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(bool issues, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u), "r"(issues ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r)::"memory");
  return r != 0u;
}

// ---------------------------------------------------------------------------------------------------------------------
// Layout
// ---------------------------------------------------------------------------------------------------------------------

// Heads of up to 64 (CB 1), 128 (CB 2) and 256 (CB 2, H 2) columns.
template <int CB, int H, class Source>
struct Wide {
  static constexpr int kRing = Source::template entries<CB, H>();  // in the ring
  using R = KvRing<2, CB, kRing, H, kRing == 4>;
  static constexpr int kCols = CB * 64, kDP = kCols * H;
  static constexpr int kS = 0, kO = 256, kQ = kO + kDP;  // tensor memory columns: two S of 128, then O, and Q where there is room
  // Half floats' Q lies in tensor memory, where a thread of the softmax warps writes its row: the products read it there instead of
  // over the shared memory's bus, which limits, and it is written between a unit's last scores and its end.  (64 blocks of 16 rows
  // over 4 bits: 100 us, Q converted in shared memory by the unpacking warps 109.)
  static constexpr bool kTmemQ = Source::kHalf && H == 1;
  // shared memory: Q (as a tile's K), the ring, s, p, pv [2], soft, and tmem, careful [2]
  static constexpr int kQBytes = R::kTile * H;
  static constexpr int kBars = kQBytes + R::kBytes;
  static constexpr int kMisc = kBars + 7 * 8 + 8;
  static constexpr int kExtra = (kMisc + 16 + 127) / 128 * 128;  // the source's own
  static constexpr int kSmem = kExtra + Source::template extra_bytes<CB, H>();
};

// Rows of a cache of whole numbers.
struct RowSource {
  using Args = KvMaps;
  static constexpr int kWarps = kLoadWarps, kFulls = 2 * kLoadThreads;  // loading warps; arrivals that fill an entry
  // Half floats in the tiles (their values are finite, Q's rows have factors of their own, and one warp plans and fetches Q), or bf16.
  static constexpr bool kHalf = false;
  template <int CB, int H>
  static __host__ __device__ constexpr int entries() { return H == 2 ? 4 : CB == 2 ? 6 : 8; }
  template <int CB, int H>
  static __host__ __device__ constexpr int extra_bytes() { return 0; }
};

// Softmax warps, loading warps, and a warp each to issue, to load Q and to plan (with half floats one does both).
template <class Source>
constexpr int kWideThreads = kSoftmaxThreads + 32 * Source::kWarps + (Source::kHalf ? 64 : 96);
// Of half floats: a new reference lies this far below the maximum, in powers of two (weights reach 2^14; a half float's least is 2^-24).
constexpr float kTopHalf = 6.0f;

template <int CB, int H, class Source>
__global__ void __launch_bounds__(kWideThreads<Source>, 1)
    k_attention_wide(const __grid_constant__ AttnParams p, const __grid_constant__ typename Source::Args source) {
  using W = Wide<CB, H, Source>;
  constexpr int kIssue = 4 + Source::kWarps, kQueries = Source::kHalf ? -1 : kIssue + 1, kPlanner = kIssue + (Source::kHalf ? 1 : 2);
  using R = typename W::R;
  constexpr int DP = W::kDP;
  extern __shared__ __align__(1024) char smem[];
  const uint32_t base = smem_addr(smem);  // Q lies first
  R ring(smem + W::kQBytes);
  int* s_misc = reinterpret_cast<int*>(smem + W::kMisc);
  volatile uint32_t* s_careful = reinterpret_cast<volatile uint32_t*>(s_misc + 1);  // [2]: units that found NaN or infinities
  const int t = threadIdx.x, warp = __shfl_sync(0xffffffffu, t >> 5, 0);
  auto bar_s = [&](uint32_t g) { return base + W::kBars + (g & 1) * 8; };
  auto bar_p = [&](uint32_t g) { return base + W::kBars + (2 + (g & 1)) * 8; };
  // Two, in turn: a wait by parity is only good where the barrier's phase before is known to be over, and that S(g) has
  // come means that O has the products of tile g - 2, not those of g - 1.
  auto bar_pv = [&](uint32_t g) { return base + W::kBars + (4 + (g & 1)) * 8; };
  const uint32_t bar_soft = base + W::kBars + 6 * 8;
  auto half = [](uint32_t g) { return g >> 1 & 1; };  // parity of tile g at a pair of barriers
  // Units of up to 64 rows have two Qs, one in each half of Q's rows: the products of the lower half read on into what
  // lies behind it, but rows past 64 are nobody's then.
  const bool small = p.max_len * static_cast<int64_t>(p.group) <= 64;
  const int twins = small && (!Source::kHalf || W::kTmemQ) ? 2 : 1;
  // With half floats each row of Q is there twice, 64 rows apart (in tensor memory, or in shared memory, which then holds one Q), and
  // two threads have a row: the second takes the tiles' upper 64 keys, with a reference, a sum and an O of its own (its weights of the
  // lower keys are 0, as are the first one's of the upper); they are put together at the end of the unit.  (The softmax warps are
  // what limits there; the matrix unit multiplies 128 rows anyway.  64 blocks of 16 rows over 4 bits: 109 us, a thread a row 112;
  // two long requests 57 and 66.)
  const bool split = small && Source::kHalf;

  if (t == 0) {
    ring.init(1, kIssue + 2, W::kTmemQ ? 4 : 1, Source::kFulls);
    if constexpr (Source::kHalf) Source::template init<CB, H>(smem + W::kExtra);
    for (int i = 0; i < 2; ++i) mbar_init(bar_s(i), 2), mbar_init(bar_p(i), kSoftmaxThreads), mbar_init(bar_pv(i), 1);
    mbar_init(bar_soft, kSoftmaxThreads);
    mbar_fence_init();
    s_careful[0] = s_careful[1] = 0u;
  }
  if (warp == kIssue) {
    tmem_alloc(base + W::kMisc, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_misc[0]);

  grid_dependency_wait();
  allow_dependents();
  const AttnSpan span = attn_span<kRows, kKeys, kUnitPlaces, kWideThreads<Source>>(p, t, ring.sums(), ring.find(),
                                                                                   [] { __syncthreads(); });

  if (warp == kPlanner) {
    if constexpr (Source::kHalf)
      plan_and_load<kRows, kUnitPlaces>(ring, p, span, nullptr, twins, [&](const AttnSegment& s, int slot) {
        ring.template fetch_q<kRows>(p, s, base, R::kBlock, slot, 64);
      });
    else
      ring.template plan<kRows, kUnitPlaces>(p, span);
  } else if (warp >= 4 && warp < kIssue) {
    if constexpr (Source::kHalf)
      Source::template load<CB, H>(ring, p, source, smem, smem + W::kExtra, split, warp - 4);
    else
      ring.load(p, source, warp - 4);
  } else if (warp == kQueries) {
    ring.template load_q<kRows>(p, base, R::kBlock, twins, 64);
  } else if (warp == kIssue) {
    // ---- The issuing warp: one lane acts, all go along.
    AttnSegment s;
    uint32_t g = 0, units = 0;
    bool ok = true;
    const bool issues = elected();
    const uint32_t qk = instruction(kKeys, false, Source::kHalf) | (p.scale_log2 < 0.0f && !W::kTmemQ ? kNegateA : 0u);
    const uint32_t tmem_at = __shfl_sync(0xffffffffu, tmem, 0);
    auto commit = [&](uint32_t bar) {
      if (issues) tc_commit(bar);
    };
    // (rows of half floats are fenced by the warps that write them)
    auto see = [&] {
      if constexpr (!Source::kHalf) fence_async();  // the copies wrote through the generic proxy, the products read through the asynchronous one
      tc_fence_after();
    };
    auto scores = [&](uint32_t n, bool last) {
      const uint32_t slot = units % twins;
#pragma unroll 1
      for (int h = 0; h < H; ++h) {
        const uint32_t group = 2 * H * n + h;
        if (!ring.wait(ring.full(group), ring.phase(group))) return false;
        see();
        if (h == 0 && issues) mbar_arrive(bar_s(n));  // hands the tile's validity on
        const uint32_t q_at = operand_at(base + slot * 64 * 128 + h * R::kTile, 16), k_at = operand_at(ring.tile(group), 16);
        const uint32_t to = tmem_at + W::kS + (n & 1) * 128;
#pragma unroll
        for (int i = 0; i < W::kCols / 16; ++i) {
          const uint32_t at = (i >> 2) * R::kBlock + (i & 3) * 32;
          if constexpr (W::kTmemQ)
            mma_ts(issues, to, tmem_at + W::kQ + i * 8, operand(k_at, at), qk, i > 0);
          else
            mma_ss(issues, to, operand(q_at, at), operand(k_at, at), qk, h > 0 || i > 0);
        }
        commit(ring.empty(group));
      }
      commit(bar_s(n));
      if (last && !W::kTmemQ) commit(ring.q_free(slot));
      return true;
    };
    while (ok && ring.next(s)) {
      const int cnt = __shfl_sync(0xffffffffu, s.cnt, 0);
      const uint32_t q_slot = units % twins;
      uint32_t q_here = ring.q_bar(q_slot);
      if constexpr (Source::kHalf) q_here = Source::template q_ready<CB, H>(smem + W::kExtra);
      if (!ring.wait(q_here, (W::kTmemQ ? units : units / twins) & 1)) break;
      tc_fence_after();
      ok = scores(g, cnt == 1);
      for (int i = 0; ok && i < cnt; ++i) {
        const uint32_t n = g + i;
        if (i + 1 < cnt && !scores(n + 1, i + 2 == cnt)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int h = 0; h < H; ++h) {
          const uint32_t group = 2 * H * n + H + h;
          if (!ring.wait(ring.full(group), ring.phase(group)) || (h == 0 && !ring.wait(bar_p(n), half(n)))) {
            ok = false;
            break;
          }
          see();
          const uint32_t v_at = operand_at(ring.tile(group), R::kBlock);
          const uint32_t to = tmem_at + W::kO + h * W::kCols, weights = tmem_at + W::kS + (n & 1) * 128;
#pragma unroll
          for (int j = 0; j < kKeys / 16; ++j)
            mma_ts(issues, to, weights + j * 8, operand(v_at, j * 2048), instruction(W::kCols, true, Source::kHalf), i > 0 || j > 0);
          commit(ring.empty(group));
        }
        if (!ok) break;
        commit(bar_pv(n));
      }
      g += cnt;
      ++units;
    }
    __syncwarp();
  } else {
    // ---- Softmax warps: thread t has row t of the unit's tile.
    uint32_t meets = 0;
    auto meet = [&] {  // a barrier of the softmax warps, bounded like every wait
      mbar_arrive(bar_soft);
      ring.wait(bar_soft, meets++ & 1);
    };
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    // a negative scale's sign is in the products; a scale of 0 by the smallest number (0 times a masked -inf is NaN)
    float c = fmaxf(fabsf(p.scale_log2), 1e-45f);
    constexpr float kLow = Source::kHalf ? kTopHalf : 0.0f;  // the reference of the weights lies this far below c m
    uint32_t g = 0, units = 0;     // tiles and units so far, this one among them
    bool ok = true, left = false;  // left: a unit that goes on behind this block
    const int half_of = split ? t >> 6 : 0, mine = split ? t & 63 : t;  // this thread's half of a tile's keys, its row
    const int h0 = half_of, h1 = split ? half_of + 1 : 2;               // 64 keys each
    // With Q in tensor memory: the thread's row of unit n's, brought to half floats' range, and the factor of its scores.
    float c_next = c;
    auto put_q = [&](uint32_t n) {
      if constexpr (W::kTmemQ) {
        const int slot = static_cast<int>(n % twins), r = slot * 64 + mine;
        if (!ring.wait(ring.q_bar(slot), n / twins & 1)) return false;
        const char* const row = smem + r * 128;
        auto piece = [&](int x) { return *reinterpret_cast<const uint4*>(row + (x >> 3) * R::kBlock + (((x & 7) ^ (r & 7)) << 4)); };
        uint32_t top = 0u;
#pragma unroll
        for (int x = 0; x < W::kCols / 8; ++x) {
          const uint4 u = piece(x);
          top = __vmaxu2(__vmaxu2(top, u.x & 0x7fff7fffu), u.y & 0x7fff7fffu);
          top = __vmaxu2(__vmaxu2(top, u.z & 0x7fff7fffu), u.w & 0x7fff7fffu);
        }
        const float2 f = Source::row_range(max(top & 0xffffu, top >> 16), fabsf(p.scale_log2));
        const float up = p.scale_log2 < 0.0f ? -f.x : f.x;
        c_next = fmaxf(f.y, 1e-45f);
#pragma unroll 1
        for (int h = 0; h < W::kCols / 64; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint4 u = piece(h * 8 + x);
            w[4 * x] = pack_half(bf16_lo(u.x) * up, bf16_hi(u.x) * up), w[4 * x + 1] = pack_half(bf16_lo(u.y) * up, bf16_hi(u.y) * up);
            w[4 * x + 2] = pack_half(bf16_lo(u.z) * up, bf16_hi(u.z) * up), w[4 * x + 3] = pack_half(bf16_lo(u.w) * up, bf16_hi(u.w) * up);
          }
          tmem_st32(tmem + lanes + W::kQ + h * 32, w);
        }
        __syncwarp();
        if ((t & 31) == 0) mbar_arrive(ring.q_free(slot));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(Source::template q_ready<CB, H>(smem + W::kExtra));
      }
      return true;
    };
    if (W::kTmemQ && ring.peek()) ok = put_q(0);
    while (ok) {
      const AttnSegment* const seg = ring.peek();
      if (!seg) break;
      const AttnSegment& s = *seg;
      ++units;
      if (W::kTmemQ) c = c_next;
      const int rows = s.r.n * p.group - s.rt * kRows;  // rows of the unit from this tile on
      const bool idle = (mine & ~31) >= rows;           // none of the warp's rows exists
      const int my_row = (s.rt * kRows + mine) / p.group;  // new row of this thread, and its head
      const int head = s.hkv * p.group + (s.rt * kRows + mine) - my_row * p.group;
      float m = -kInfF, l = 0.0f;  // m: a score without its factor c
      uint32_t bad = 0u;
      bool mixed = false;  // a tile whose keys some rows see and others do not
      const int cnt = s.cnt, t0 = s.t0;
      for (int i = 0; i < cnt; ++i, ++g) {
        const int x0 = (t0 + i) * kKeys;
        const uint32_t st = tmem + lanes + W::kS + (g & 1) * 128;
        if (!ring.wait(bar_s(g), half(g))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if constexpr (Source::kHalf && !W::kTmemQ) {  // the row's factor is there with its scores
          if (i == 0) c = Source::template row_factor<CB, H>(smem + W::kExtra, units - 1, mine);
        }
        const uint4 vv = *reinterpret_cast<const uint4*>(ring.valid(g));
        const uint4 vb = *reinterpret_cast<const uint4*>(ring.valid(g) + 4);
        uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
        bad |= vb.x | vb.y | vb.z | vb.w;
        const bool masked = (vw[0] & vw[1] & vw[2] & vw[3]) != 0xffffffffu || x0 + kKeys > s.r.len;
        if (!Source::kHalf && masked && new_rows_differ(p, s.r) && x0 + kKeys > s.r.len) {
          mixed = true;
          const int from = max(s.r.len - x0, 0), upto = min(s.r.len + s.r.n - x0, kKeys);  // the new rows
          bool found = false;
          // With one tile's entries in the ring V(g) lies where V(g - 1) did, which S(g) does not wait for: the phase before
          // the one waited for here is known to be over once V(g - 1) has been used.  (A unit's first tile comes after the
          // end of the unit before; larger rings have V(g - 2) or an older one in the place, and S(g) comes behind its use.)
          if (R::kEntries == 2 * H && i > 0 && !ring.wait(bar_pv(g - 1), half(g - 1))) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (int h = 0; ok && h < H; ++h) {
            const uint32_t group = 2 * H * g + H + h;
            ok = ring.wait(ring.full(group), ring.phase(group));
            char* v = ring.tile_mem(group);
            for (int x = from * R::kPieces + t; ok && x < upto * R::kPieces; x += kSoftmaxThreads) {
              if (make_finite<true>(reinterpret_cast<uint4*>(v + R::piece(x / R::kPieces, x % R::kPieces)))) found = true;
            }
          }
          if (!ok) break;
          if (found) s_careful[units & 1] = units;
          fence_async();
        }
        if (!idle) {
          if (masked) {  // what the row does not see of the tile becomes -inf, in place
#pragma unroll
            for (int w = 0; w < 4; ++w) if (w >= 2 * h0 && w < 2 * h1)
                vw[w] = row_sees_of(p, s.r, s.b, mine < rows ? my_row : s.r.n, x0 + w * 32, vw[w]);
            uint32_t word = h0 ? vw[2] : vw[0];
#pragma unroll 1
            for (int h = 2 * h0; h < 2 * h1; ++h) {
              if (!__all_sync(0xffffffffu, word == 0xffffffffu)) {
                float v[32];
                if (__any_sync(0xffffffffu, word != 0u)) {
                  tmem_ld32(st + h * 32, reinterpret_cast<uint32_t*>(v));
                  tmem_wait_ld();
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = (word >> j & 1u) ? v[j] : -kInfF;
                tmem_st32(st + h * 32, reinterpret_cast<const uint32_t*>(v));
              }
              word = h == 0 ? vw[1] : h == 1 ? vw[2] : vw[3];
            }
            tmem_wait_st();
          }
          // The scores are read twice, for the maximum and for the weights: 128 of them do not fit beside the rest.
          float mx[4] = {-kInfF, -kInfF, -kInfF, -kInfF};
#pragma unroll 1
          for (int h = h0; h < h1; ++h) {
            float v[64];
            tmem_ld32(st + h * 64, reinterpret_cast<uint32_t*>(v));
            tmem_ld32(st + h * 64 + 32, reinterpret_cast<uint32_t*>(v) + 32);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) mx[j & 3] = fmax_nan(mx[j & 3], v[2 * j], v[2 * j + 1]);
          }
          const float top = fmax_nan(fmax_nan(mx[0], mx[1]), fmax_nan(mx[2], mx[3]));
          const bool grow = !(top <= m) && !((top - m) * c <= kSlack);  // also a first finite maximum, and NaN
          if (i == 0) {
            m = top;
          } else if (__any_sync(0xffffffffu, grow)) {
            const float a = grow ? ex2_fast((m - top) * c) : 1.0f;
            if (grow) m = top;
            l *= a;
            if (!ring.wait(bar_pv(g - 1), half(g - 1))) {
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
          // c S - c m, one multiply-add with c m rounded (by 2^-18 at most), as long as c m is small enough; where a row's is
          // not, the warp's rows are moved to their references first, in place: at 2^31 the rounding alone would be past the
          // exponent's range.
          float ref = m == -kInfF ? 0.0f : m * c;
          if (__any_sync(0xffffffffu, !(fabsf(ref) < kNear))) {
            const float from = m == -kInfF ? 0.0f : m;
#pragma unroll 1
            for (int h = 2 * h0; h < 2 * h1; ++h) {
              float v[32];
              tmem_ld32(st + h * 32, reinterpret_cast<uint32_t*>(v));
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] -= from;
              tmem_st32(st + h * 32, reinterpret_cast<const uint32_t*>(v));
            }
            tmem_wait_st();
            ref = 0.0f;
          }
          ref -= kLow;
          uint64_t sum[2] = {0u, 0u};  // of each fourth weight, in pairs
          const uint64_t c2 = pair(c, c), ref2 = pair(-ref, -ref);
#pragma unroll 1
          for (int h = h0; h < h1; ++h) {
            float v[64];
            tmem_ld32(st + h * 64, reinterpret_cast<uint32_t*>(v));
            tmem_ld32(st + h * 64 + 32, reinterpret_cast<uint32_t*>(v) + 32);
            tmem_wait_ld();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t pk[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float a, b;
                unpair(fma_pair(pair(v[part * 32 + 2 * j], v[part * 32 + 2 * j + 1]), c2, ref2), a, b);
                a = ex2_fast(a), b = ex2_fast(b);
                sum[j & 1] = add_pair(sum[j & 1], pair(a, b));
                pk[j] = Source::kHalf ? pack_half(a, b) : pack_bf16(a, b);
              }
              tmem_st16(st + h * 32 + part * 16, pk);
            }
          }
          if (split) {  // the other half of the keys is the other thread's
            uint32_t none[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) none[j] = 0u;
            tmem_st32(st + (1 - h0) * 32, none);
          }
          float of[4];
          unpair(sum[0], of[0], of[1]), unpair(sum[1], of[2], of[3]);
          l += (of[0] + of[1]) + (of[2] + of[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(bar_p(g));
      }
      if (!ok) break;
      // The next unit's Q, now that this one's last scores are there: its products begin while this one's end.
      if (W::kTmemQ && ring.another() && !put_q(units)) break;
      // The unit's last product is done: this thread's row of O.
      if (!ring.wait(bar_pv(g - 1), half(g - 1))) break;
      tc_fence_after();
      bool careful = false;
      if (mixed) {
        meet();
        careful = s_careful[units & 1] == units;  // (a unit's products wait for every thread: none is two units ahead)
      }
      bad = (bad ? kStSlotRange : 0u) | s.r.status;
      const bool whole = s.cnt == s.nt;
      using P = AttnPart<kRows, DP>;
      float* part = whole ? nullptr : attn_part<kRows, DP>(p, blockIdx.x, s.t0 == 0);
      char* out = p.out + ((s.r.row0 + my_row) * p.o_row + head * p.o_head) * 2;
      float top = m * c - kLow, weight = 1.0f;  // the reference, and what O is to be multiplied by
      if constexpr (Source::kHalf) {
        if (split) {
          float2* const pairs = Source::template pairs<CB, H>(smem + W::kExtra);
          pairs[t] = make_float2(top, l);
          meet();
          const float2 other = pairs[t ^ 64];
          const float both = fmax_nan(top, other.x), from = both == -kInfF ? 0.0f : both;
          weight = ex2_fast(top - from);
          l = fmaf(l, weight, other.y * ex2_fast(other.x - from));
          top = both;
        }
      }
      const bool none = (split ? top : m) == -kInfF;  // nothing seen, or only scores of -inf
      const float inv = none ? 0.0f : 1.0f / l;
      if (!idle || split) {
#pragma unroll 1
        for (int h = 0; h < DP / 32; ++h) {
          float o[32];
          tmem_ld32(tmem + lanes + W::kO + h * 32, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
          if constexpr (Source::kHalf) {
            if (split) {  // 32 columns go through shared memory (two places, in turn): the second thread's to the first
              float4* const row = Source::template exchange<CB, H>(smem, smem + W::kExtra, h & 1) + mine * 8;
              if (half_of) {
#pragma unroll
                for (int d = 0; d < 8; ++d)
                  row[d ^ (mine & 7)] = make_float4(o[4 * d] * weight, o[4 * d + 1] * weight, o[4 * d + 2] * weight, o[4 * d + 3] * weight);
              }
              meet();
              if (!half_of) {
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                  const float4 v = row[d ^ (mine & 7)];
                  o[4 * d] = fmaf(o[4 * d], weight, v.x), o[4 * d + 1] = fmaf(o[4 * d + 1], weight, v.y);
                  o[4 * d + 2] = fmaf(o[4 * d + 2], weight, v.z), o[4 * d + 3] = fmaf(o[4 * d + 3], weight, v.w);
                }
              }
              if (W::kTmemQ) meet();  // (there is one place)
            }
          }
          if (mine < rows && !half_of) {
            if (!Source::kHalf && careful) {
#pragma unroll
              for (int d = 0; d < 32; d += 4) {
                const float4 f = nonfinite_seen<true, kKeys>(p, s, my_row, h * 32 + d);
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
                reinterpret_cast<float4*>(part)[(h * 8 + d / 4) * kRows + mine] =
                    make_float4(o[d], o[d + 1], o[d + 2], o[d + 3]);
            }
          }
        }
      }
      if (whole) {
        if (mine < rows && !half_of && p.lse) p.lse[(s.r.row0 + my_row) * p.heads + head] = none ? -kInfF : fmaf(top, kLn2, logf(l));
        if (s.reports && t == 0) p.status[s.b] = bad | attn_timeout(p);
      } else {
        if (!half_of) part[P::kM + mine] = top, part[P::kL + mine] = l;
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
      if constexpr (Source::kHalf && !W::kTmemQ) mbar_arrive(Source::template unit_done<CB, H>(smem + W::kExtra));
      ring.release();
    }
    if (t == 0 && !left)
      reinterpret_cast<AttnSplit*>(attn_part<kRows, DP>(p, blockIdx.x, true) + AttnPart<kRows, DP>::kSplit)->last = 0;
  }
  __syncthreads();
  ring.report_abort(p);
  if (warp == kIssue) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Block (c, i): rows 8 i .. of the unit that begins in block c of the attention kernel and goes on behind it, if any.
// (Rows a block, quads a thread, parts in flight; two requests of 60000 to 100000 and a block of 64 requests: 16, 2, 8: 66
// and 119 us; 8, 2, 4: 63 and 118; 8, 2, 10: 62 and 119; 4, 2, 8: 62 and 120; 8, 1, 20: 63 and 127.)
constexpr int kJoinRows = 8;

template <int DP>
__global__ void __launch_bounds__(kJoinRows * DP / 8) k_attention_join(AttnParams p) {
  using P = AttnPart<kRows, DP>;
  constexpr int PARTS = 4, E = 2;  // parts in flight, quads of columns a thread
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

template <int CB, int H, class Source>
cudaError_t launch_wide(const AttnParams& p, const typename Source::Args& source, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int DP = Wide<CB, H, Source>::kDP;
  static std::mutex mu;
  static bool have[64] = {};
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!have[d]) {
      e = cudaFuncSetAttribute(k_attention_wide<CB, H, Source>, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<CB, H, Source>::kSmem);
      if (e != cudaSuccess) return e;
      have[d] = true;
    }
  }
  static_assert(Wide<CB, H, Source>::kSmem <= 227 * 1024, "shared memory of a block");
  const int grid = dev.sms < kAttnMaxBlocks / 2 ? dev.sms : kAttnMaxBlocks / 2;  // parts are laid out for 64-row tiles
  e = launch_pdl(k_attention_wide<CB, H, Source>, dim3(static_cast<unsigned>(grid)), dim3(kWideThreads<Source>),
                 Wide<CB, H, Source>::kSmem, stream, p, source);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.max_len) * p.group;
  const int slices = static_cast<int>(((rows < kRows ? rows : kRows) + kJoinRows - 1) / kJoinRows);
  return launch_pdl(k_attention_join<DP>, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(slices)),
                    dim3(kJoinRows * DP / 8), 0, stream, p);
}

}  // namespace
}  // namespace sv
