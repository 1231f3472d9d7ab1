// Attention over the 4-bit cache for few query rows (a decoded token's heads, a
// short chain's), in tiles of 8 or 16 rows.
//
//   S^T = K Q^T   (16 keys x 8 rows a matrix instruction)
//   O^T += V^T P^T
//
// Codes become half floats in registers, on their way from shared memory to
// the matrix unit: an instruction converts two of them, another multiplies them
// by their scales, and the product is exact.  So that keys fill the 16 rows of
// the instruction and the few query rows its 8 columns, both products are taken
// transposed.  The order of a contraction is free, so a lane's columns of K and of
// V are those that lie together: 16 bytes of a key's codes for K, 8 bytes of each of
// four keys for V, whose codes are paired (two keys, one column) before they
// are converted.  P^T is S^T with its 8 x 8 parts turned.
//
// The queries are brought to the range of half floats by a power of two a row,
// which the scores' factor takes back; the weights are half floats (2^-12 of
// themselves, below the rounding of the output), their sum l is in fp32.  A warp's
// reference m moves only when a score passes it by 2^14, the largest weight
// that a half float has room for; so there is no exchange between lanes in a
// usual tile.
//
// A tile's slices of 16 keys are dealt out to the warps of a team; teams take
// tiles in turn.  A warp that is through with a unit leaves its (m, l, O) in
// shared memory and goes on; the last one joins them and writes the rows, or
// the block's part of the unit.
//
// Bound by its instructions' order: of the 330 for a slice of 16 keys (64 conversions, 64
// products with scales) most wait for the one before, and two warps on each
// scheduler, all that the registers hold, issue one at every other clock (no pipe is
// busy for more than 42 % of the time).  The bytes are there in time (the same pages
// again and again, out of L2, take as long).  One token of 128 requests of 64 to 8192, 32 heads of 128 on 8: 153 us,
// 4.0 TB/s (over bf16 320, for 3.6 times the bytes); bringing the tiles in alone
// takes 110 us.  Two slices a warp side by side: 153, one
// after the other by twelve warps 157, one by sixteen 166; one team of four warps 171;
// tiles brought in with 16-byte copies 315.  One request of 500: 11 us, which is latency.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "sv_attention_packed.cuh"

namespace sv {
namespace {

constexpr int kSlice = 16;              // keys that a warp takes at once
constexpr int kSlices = kKeys / kSlice;
constexpr int kUnitPlaces = 2;   // what a unit costs beside its key tiles, in tiles
constexpr float kTop = 6.0f;     // a new reference lies this far below the maximum, in powers of two ...
constexpr float kSlack = 14.0f;  // ... and scores may pass it by this much: weights are below 2^14

// Heads of up to D (64, 128, 256) columns, 8 NT rows.
template <int D, int NT>
struct Few4 {
  static constexpr int kRows = 8 * NT;
  // A tile is taken by kWarps warps, kTogether slices each: as many as their registers hold.  Tile g is that of team g % kTeams.
  static constexpr bool kLarge = D == 256 || NT == 2;
  static constexpr int kTogether = kLarge ? 1 : 2, kWarps = kSlices / kTogether, kTeams = kLarge ? 1 : 2;
  static constexpr int kTakers = kWarps * kTeams;
  static constexpr int kHelpers = 4, kStageWarps = D == 256 ? 2 : 3;  // those that load tiles; the last helper plans and fetches Q
  static constexpr int kThreads = 32 * (kHelpers + kTakers);
  static constexpr int kPlaces = D == 256 ? 4 : 6;
  static_assert(kPlaces % kTeams == 0, "a place belongs to one team");
  using Stage = PackedStage<kPlaces, kStageWarps, packed_tile_bytes(D)>;
  static constexpr int KW = D / 32;   // words of codes that a lane has of a key's K
  static constexpr int VW = D / 64;   // and of a key's V
  static constexpr int MT = D / 16;   // tiles of 16 columns of O
  static constexpr int kLeave = (MT + 1) * NT * 32 * 16;  // a warp's O, m and l
  static constexpr int kQRow = D * 2 + 16;
  // shared memory: the places; the plan; two Qs; what the warps leave; their flags; counters and barriers; split segments
  static constexpr int kPlan = Stage::kBytes;
  static constexpr int kQ = kPlan + PlanQueue::kBytes;
  static constexpr int kLeft = kQ + 2 * kRows * kQRow;
  static constexpr int kFlags = kLeft + kTakers * kLeave;
  static constexpr int kMisc = kFlags + kTakers * 4 + (kTakers * 4) % 16;  // left free barrier, last, split, count
  static constexpr int kParts = kMisc + 32;
  static constexpr int kSmem = kParts + 2 * static_cast<int>(sizeof(AttnSegment));
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// N words (1, 2, 4 or 8: of two pieces that lie `far` bytes apart) from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N], int far = 0) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(at + i * far));
  }
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at));
  return r;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(at));
  return r;
}

// DENSE: heads of D columns in pages of a multiple of 16, whose steps in shared memory are constants.
template <int D, int NT, bool DENSE>
__global__ void __launch_bounds__(Few4<D, NT>::kThreads, 1)
    k_packed_few(const __grid_constant__ AttnParams p, const __grid_constant__ PackedTiles tiles) {
  using W = Few4<D, NT>;
  constexpr int KW = W::KW, VW = W::VW, MT = W::MT, kRows = W::kRows, kTakers = W::kTakers;
  extern __shared__ __align__(128) char smem[];
  const uint32_t base = smem_addr(smem);
  typename W::Stage stage(smem);
  PlanQueue plan(smem + W::kPlan);
  const uint32_t bar_left = base + W::kMisc;  // what the warps leave has been joined
  int* s_last = reinterpret_cast<int*>(smem + W::kMisc + 8);
  int* s_split = s_last + 1;                  // segments of the block that are only part of their unit
  unsigned* s_count = reinterpret_cast<unsigned*>(s_last + 2);
  uint32_t* s_flags = reinterpret_cast<uint32_t*>(smem + W::kFlags);
  AttnSegment* s_parts = reinterpret_cast<AttnSegment*>(smem + W::kParts);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    stage.init(W::kWarps);
    plan.init(kTakers + W::kStageWarps + 1, kTakers);
    mbar_init(bar_left, 1);
    *s_count = 0u;
    mbar_fence_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const AttnSpan span = attn_span<kRows, kKeys, kUnitPlaces, W::kThreads>(p, t, plan.sums(), plan.find(), [] { __syncthreads(); });
  const int dim = p.c.head_dim;
  if (warp < W::kHelpers) {
    if (warp < W::kStageWarps) {
      stage.load(plan, p, tiles, warp);
    } else if (warp == W::kHelpers - 1) {
      const int split = plan_and_load<kRows, kUnitPlaces>(plan, p, span, s_parts, 2, [&](const AttnSegment& s, int at) {
        // rows that do not exist are 0
        const int rows = s.r.n * p.group - s.rt * kRows;
        for (int x = lane; x < kRows * (D / 8); x += 32) {
          const int row = x / (D / 8), piece = x % (D / 8), grow = s.rt * kRows + row, i = grow / p.group;
          const bool live = row < rows && piece * 8 < dim;
          const int64_t from = (s.r.row0 + i) * p.q_row + (s.hkv * p.group + grow - i * p.group) * p.q_head + piece * 8;
          cp_async16(base + W::kQ + (at * kRows + row) * W::kQRow + piece * 16, live ? p.q + from * 2 : p.q, live);
        }
        cp_async_commit();
        cp_async_wait<0>();
        mbar_arrive(plan.q_bar(at));
      });
      if (lane == 0) *s_split = split;
    }
  } else {
    const int taker = warp - W::kHelpers, team = taker / W::kWarps, x_own = taker % W::kWarps * W::kTogether * kSlice;
    const int g8 = lane >> 2, t4 = lane & 3;  // a fragment's row, and its pair of columns
    const int rows_log = tiles.rows_log, block = tiles.block, in_block = (1 << rows_log) - 1;
    const int code_row = DENSE ? D / 2 : dim / 2, scale_row = DENSE ? D / 16 : dim / 16;
    // Where key x of a tile lies, and how far keys 1, 8 and 16 further on are from a slice's first.
    auto code_at = [&](int x) { return (x >> rows_log) * block + (x & in_block) * code_row; };
    auto scale_at = [&](int x) { return (x >> rows_log) * block + (x & in_block) * scale_row; };
    const int code8 = DENSE ? 8 * code_row : code_at(8), scale8 = DENSE ? 8 * scale_row : scale_at(8);
    const int code1 = (t4 & 1 ? -1 : 1) * (DENSE ? code_row : code_at(1)), scale1 = (t4 & 1 ? -1 : 1) * (DENSE ? scale_row : scale_at(1));
    const int code16 = code_at(kSlice), scale16 = scale_at(kSlice);
    // Row m of a product's 16 is key m ^ (m >> 1 & 1) of the slice: so lanes that read K together read neighbouring keys, and those
    // that read V together keys of both parities, which lie in different banks.
    const int key = g8 ^ (g8 >> 1 & 1);
    // K: keys key and key + 8, this lane's columns (16 or 32 from k_col on; of 256 columns 32 more, 128 further on).  Columns
    // that a head does not have are others' codes times 0.
    constexpr int kCols = D == 64 ? 16 : 32;
    const int k_col = t4 * kCols;
    const bool k_live = k_col < dim, k_live2 = D == 256 && k_col + 128 < dim;
    const uint32_t k_code = base + code_at(x_own + key) + (k_live ? k_col / 2 : 0);
    const uint32_t k_scale = base + packed_k_scales(in_block + 1, dim) + scale_at(x_own + key) + (k_live ? k_col / 16 : 0);
    const uint32_t k_one = k_live ? 128u : 0u, k_one2 = k_live2 ? 128u : 0u;
    // V: the keys of rows 2 t4, + 1, + 8, + 9, columns v_col .. v_col + D / 8 - 1.
    const int v_col = g8 * (D / 8);
    const bool v_live = v_col < dim;
    const uint32_t v_code = base + packed_v_codes(in_block + 1, dim) + code_at(x_own + 2 * t4 + (t4 & 1)) + (v_live ? v_col / 2 : 0);
    const uint32_t v_scale = base + packed_v_scales(in_block + 1, dim) + scale_at(x_own + 2 * t4 + (t4 & 1)) + (v_live ? v_col / 16 : 0);
    const uint32_t v_one = v_live ? 128u : 0u;
    uint32_t g = 0;             // tiles of the segments before
    int place = team;           // of the team's next tile, and its phase there
    uint32_t parity = 0u;
    bool ok = true;
    for (uint32_t unit = 0; ok; ++unit) {
      const AttnSegment* const seg = plan.peek();
      if (!seg) break;
      const AttnSegment& s = *seg;
      const int rows = s.r.n * p.group - s.rt * kRows;
      const int q_slot = unit & 1;
      if (!plan.wait(plan.q_bar(q_slot), unit >> 1 & 1)) break;
      // Q's fragments: row g8 of each tile of 8 rows, the columns that this lane has of K.
      uint32_t qf[NT][KW][4];
      float factor[NT][2];  // of the scores of rows 2 t4 and 2 t4 + 1
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t at = base + W::kQ + (q_slot * kRows + n * 8 + g8) * W::kQRow + k_col * 2;
        uint32_t top = 0u;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint4 u = lds16(at + (w & 3) * 16 + (w >> 2) * 256);
          qf[n][w][0] = u.x, qf[n][w][1] = u.y, qf[n][w][2] = u.z, qf[n][w][3] = u.w;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = __vmaxu2(top, qf[n][w][i] & 0x7fff7fffu);
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const RowScale f = row_scale(top, p.scale_log2);
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[n][w][i] = pack_half(bf16_lo(qf[n][w][i]) * f.up, bf16_hi(qf[n][w][i]) * f.up);
#pragma unroll
        for (int c = 0; c < 2; ++c) factor[n][c] = __shfl_sync(0xffffffffu, f.factor, (2 * t4 + c) * 4);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(plan.q_free(q_slot));
      // Of rows 2 t4 and 2 t4 + 1: the reference (0 at first), what scores may reach before it moves, the sum, O.
      float ref[NT][2], most[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        ref[n][0] = ref[n][1] = l[n][0] = l[n][1] = 0.0f, most[n][0] = most[n][1] = -kInfF;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
      }
      uint32_t bad = 0u;
      // The warp's slices of tile i of the segment, side by side.
      constexpr int N = W::kTogether;
      const int cnt = s.cnt, len = s.r.len, end = s.r.len + s.r.n, first = s.t0 * kKeys + x_own;
#pragma unroll 1
      for (int i = (team + W::kTeams - static_cast<int>(g % W::kTeams)) % W::kTeams; i < cnt; i += W::kTeams) {
        if (!plan.wait(stage.full(place), parity)) {
          ok = false;
          break;
        }
        uint32_t kw[N][2][KW], ks[N][2][D == 256 ? 2 : 1], vw[N][4][VW], vs[N][4], good[N];
        const uint32_t tile_at = place * W::Stage::kTile, info = base + W::Stage::kInfo + place * 32 + x_own / 8;
        if constexpr (N == 2) {  // keys that are there, and that are not
          uint32_t both, none;
          asm volatile("ld.shared.u32 %0, [%2];\n\tld.shared.u32 %1, [%2 + 16];" : "=r"(both), "=r"(none) : "r"(info));
          good[0] = both & 0xffffu, good[N - 1] = both >> 16;
          bad |= none;
        } else {
          good[0] = lds_u16(info);
          bad |= lds_u16(info + 16);
        }
#pragma unroll
        for (int z = 0; z < N; ++z) {
          const uint32_t at_code = tile_at + z * code16, at_scale = tile_at + z * scale16;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = at_code + k_code + h * code8, b = at_scale + k_scale + h * scale8;
            if constexpr (D == 256) {
              lds_words<KW>(a, kw[z][h], k_live2 ? 64 : 0);
              ks[z][h][0] = lds_u16(b);
              ks[z][h][D == 256 ? 1 : 0] = lds_u16(b + (k_live2 ? 8 : 0));
            } else {
              lds_words<KW>(a, kw[z][h]);
              ks[z][h][0] = D == 64 ? lds_u8(b) : lds_u16(b);
            }
          }
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            lds_words<VW>(at_code + v_code + (h & 1) * code1 + (h >> 1) * code8, vw[z][h]);
            const uint32_t b = at_scale + v_scale + (h & 1) * scale1 + (h >> 1) * scale8;
            vs[z][h] = D == 256 ? lds_u16(b) : lds_u8(b);
          }
        }
        const int x0 = first + i * kKeys;  // the first key
        auto done = [&] {  // all that the warp needs of the tile is in its registers
          __syncwarp();
          if (lane == 0) mbar_arrive(stage.empty(place));
          place += W::kTeams;
          if (place >= W::kPlaces) place -= W::kPlaces, parity ^= 1u;
        };
        done();
        if (x0 >= end) continue;
        // Scores: two chains of products a slice.
        float sc[N][NT][4], other[N][NT][4];
#pragma unroll
        for (int z = 0; z < N; ++z)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[z][n][j] = other[z][n][j] = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int z = 0; z < N; ++z) {
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              unpack_codes(kw[z][h][w], a[h]);
              const uint32_t s2 = scale_pair(__byte_perm(ks[z][h][w >> 2], 0u, D == 64 || (w & 2) == 0 ? 0x4040 : 0x4141),
                                             w < 4 ? k_one : k_one2);
#pragma unroll
              for (int j = 0; j < 4; ++j) a[h][j] = mul_half2(a[h][j], s2);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(sc[z][n], a[0][0], a[1][0], a[0][1], a[1][1], qf[n][w][0], qf[n][w][1]);
              mma_f16(other[z][n], a[0][2], a[1][2], a[0][3], a[1][3], qf[n][w][2], qf[n][w][3]);
            }
          }
#pragma unroll
        for (int z = 0; z < N; ++z)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[z][n][j] = (sc[z][n][j] + other[z][n][j]) * factor[n][j & 1];
#pragma unroll
        for (int z = 0; z < N; ++z)
          if (good[z] != 0xffffu || x0 + z * kSlice + kSlice > len) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t see =
                    row_sees_of(p, s.r, s.b, (s.rt * kRows + n * 8 + 2 * t4 + c) / p.group, x0 + z * kSlice, good[z]);
                if (!(see >> key & 1u)) sc[z][n][c] = -kInfF;
                if (!(see >> (key + 8) & 1u)) sc[z][n][2 + c] = -kInfF;
              }
          }
        float top[NT][2];
        bool grow = false;  // also at a first finite score, and at NaN
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            top[n][c] = fmax_nan(sc[0][n][c], sc[0][n][2 + c]);
#pragma unroll
            for (int z = 1; z < N; ++z) top[n][c] = fmax_nan(top[n][c], fmax_nan(sc[z][n][c], sc[z][n][2 + c]));
            grow = grow || !(top[n][c] <= most[n][c]);
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top[n][c] = fmax_nan(top[n][c], __shfl_xor_sync(0xffffffffu, top[n][c], x));
              if (!(top[n][c] <= most[n][c])) {
                const float to = top[n][c] - kTop, a = most[n][c] == -kInfF ? 0.0f : ex2_fast(ref[n][c] - to);
                // (rounded down: of a score beyond 2^25 the next float may be 16 higher, whose weight a half float has no room for)
                ref[n][c] = to, most[n][c] = __fadd_rd(to, kSlack);
                l[n][c] *= a;
#pragma unroll
                for (int d = 0; d < MT; ++d) o[n][d][c] *= a, o[n][d][2 + c] *= a;
              }
            }
        }
        uint32_t pt[N][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int z = 0; z < N; ++z) {
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = ex2_fast(sc[z][n][j] - ref[n][j & 1]);
            l[n][0] += w[0] + w[2];
            l[n][1] += w[1] + w[3];
            pt[z][n][0] = turn8(pack_half(w[0], w[1]));
            pt[z][n][1] = turn8(pack_half(w[2], w[3]));
          }
        }
        // V: word w of a pair of keys holds eight columns of both.
        uint32_t s2[N][D == 256 ? 2 : 1][2];  // scales, by group of columns, by pair of keys
#pragma unroll
        for (int z = 0; z < N; ++z)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s2[z][0][h] = scale_pair(__byte_perm(vs[z][2 * h], vs[z][2 * h + 1], D == 256 ? 0x7430 : 0x1410), v_one);
            if constexpr (D == 256) s2[z][1][h] = scale_pair(__byte_perm(vs[z][2 * h], vs[z][2 * h + 1], 0x7531), v_one);
          }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int z = 0; z < N; ++z) {
            uint32_t even[2][4], odd[2][4];  // by pair of keys: the codes' even and odd columns
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a = vw[z][2 * h][w], b = vw[z][2 * h + 1][w];
              unpack_codes((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even[h]);
              unpack_codes(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odd[h]);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                even[h][j] = mul_half2(even[h][j], s2[z][w / 2][h]), odd[h][j] = mul_half2(odd[h][j], s2[z][w / 2][h]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(o[n][w * 4 + j], even[0][j], odd[0][j], even[1][j], odd[1][j], pt[z][n][0], pt[z][n][1]);
          }
      }
      g += s.cnt;
      if (!ok) break;

      // What the warp has is left to the unit's last warp.  A lane has the same rows and columns in every warp.
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
      if (unit > 0 && !plan.wait(bar_left, (unit - 1) & 1)) break;
      auto left = [&](int w) { return reinterpret_cast<float4*>(smem + W::kLeft + w * W::kLeave) + lane; };
      float4* to = left(taker);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int d = 0; d < MT; ++d) to[(n * (MT + 1) + d) * 32] = make_float4(o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]);
        const float m[2] = {most[n][0] == -kInfF ? -kInfF : ref[n][0], most[n][1] == -kInfF ? -kInfF : ref[n][1]};
        to[(n * (MT + 1) + MT) * 32] = make_float4(m[0], m[1], l[n][0], l[n][1]);
      }
      if (lane == 0) s_flags[taker] = bad;
      __syncwarp();
      unsigned before = 0u;
      if (lane == 0) asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(before) : "r"(smem_addr(s_count)) : "memory");
      before = __shfl_sync(0xffffffffu, before, 0);
      if (before == kTakers - 1) {
        __syncwarp();
        uint32_t any = 0u;
        for (int w = 0; w < kTakers; ++w) any |= s_flags[w];
        const uint32_t status = (any ? kStSlotRange : 0u) | s.r.status;
        const bool whole = s.cnt == s.nt;
        using P = AttnPart<kRows, D>;
        float* part = attn_part<kRows, D>(p, blockIdx.x, s.t0 == 0);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float M[2] = {-kInfF, -kInfF}, L[2] = {0.0f, 0.0f};
#pragma unroll
          for (int w = 0; w < kTakers; ++w) {
            const float4 x = left(w)[(n * (MT + 1) + MT) * 32];
            M[0] = fmax_nan(M[0], x.x), M[1] = fmax_nan(M[1], x.y);
          }
          const float ref[2] = {M[0] == -kInfF ? 0.0f : M[0], M[1] == -kInfF ? 0.0f : M[1]};
          float4 sum[MT];
#pragma unroll
          for (int d = 0; d < MT; ++d) sum[d] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int w = 0; w < kTakers; ++w) {
            const float4* from = left(w) + n * (MT + 1) * 32;
            const float4 x = from[MT * 32];
            const float w0 = ex2_fast(x.x - ref[0]), w1 = ex2_fast(x.y - ref[1]);
            L[0] = fmaf(x.z, w0, L[0]), L[1] = fmaf(x.w, w1, L[1]);
#pragma unroll
            for (int d = 0; d < MT; ++d) {
              const float4 v = from[d * 32];
              sum[d].x = fmaf(v.x, w0, sum[d].x), sum[d].y = fmaf(v.y, w1, sum[d].y);
              sum[d].z = fmaf(v.z, w0, sum[d].z), sum[d].w = fmaf(v.w, w1, sum[d].w);
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = n * 8 + 2 * t4 + c, grow = s.rt * kRows + row;
            if (row >= rows) continue;
            // column v_col + 2 d + h of the row
            auto at = [&](int d, int h) { return c ? (h ? sum[d].w : sum[d].y) : (h ? sum[d].z : sum[d].x); };
            if (whole) {
              const int i = grow / p.group, head = s.hkv * p.group + grow - i * p.group;
              const bool none = M[c] == -kInfF;  // nothing seen, or only scores of -inf
              const float inv = none ? 0.0f : 1.0f / L[c];
              if (v_live) {
                char* out = p.out + ((s.r.row0 + i) * p.o_row + head * p.o_head + v_col) * 2;
#pragma unroll
                for (int d = 0; d < MT; d += 4) {
                  uint4 u = make_uint4(0u, 0u, 0u, 0u);
                  if (!none)
                    u = make_uint4(pack_bf16(at(d, 0) * inv, at(d, 1) * inv), pack_bf16(at(d + 1, 0) * inv, at(d + 1, 1) * inv),
                                   pack_bf16(at(d + 2, 0) * inv, at(d + 2, 1) * inv), pack_bf16(at(d + 3, 0) * inv, at(d + 3, 1) * inv));
                  *reinterpret_cast<uint4*>(out + d * 4) = u;
                }
              }
              if (g8 == 0 && p.lse) p.lse[(s.r.row0 + i) * p.heads + head] = none ? -kInfF : fmaf(M[c], kLn2, logf(L[c]));
            } else {
#pragma unroll
              for (int d = 0; d < MT; d += 2)
                *(reinterpret_cast<float4*>(part) + (v_col / 4 + d / 2) * kRows + row) =
                    make_float4(at(d, 0), at(d, 1), at(d + 1, 0), at(d + 1, 1));
              if (g8 == 0) part[P::kM + row] = M[c], part[P::kL + row] = L[c];
            }
          }
        }
        if (lane == 0) {
          if (!whole)
            part[P::kStatus] = __uint_as_float(status);
          else if (s.reports)
            p.status[s.b] = status | attn_timeout(p);
          *s_count = 0u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_left);
      }
      plan.release();
    }
  }
  __syncthreads();
  if (*plan.abort())
    plan.report_abort(p);
  else
    attn_join<true, kRows, D, W::kThreads>(p, span, s_parts, *s_split, s_last);
}

template <int D, int NT, bool DENSE>
cudaError_t launch_as(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream) {
  using W = Few4<D, NT>;
  const auto kernel = k_packed_few<D, NT, DENSE>;
  static std::mutex mu;
  static bool have[64] = {};
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!have[d]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
      if (e != cudaSuccess) return e;
      have[d] = true;
    }
  }
  static_assert(W::kSmem <= 227 * 1024, "shared memory of a block");
  const int grid = dev.sms < kAttnMaxBlocks ? dev.sms : kAttnMaxBlocks;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(W::kThreads), W::kSmem, stream, p, packed_tiles(c));
}

template <int D, int NT>
cudaError_t launch(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream) {
  const bool dense = c.head_dim == D && c.page_size % kSlice == 0 && (c.page_size % kKeys == 0 || kKeys % c.page_size == 0);
  return dense ? launch_as<D, NT, true>(p, c, dev, stream) : launch_as<D, NT, false>(p, c, dev, stream);
}

}  // namespace

cudaError_t launch_packed_attention_few(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream) {
  const bool one = static_cast<int64_t>(p.max_len) * p.group <= 8;
  const int dim = c.head_dim;
  if (dim <= 64) return one ? launch<64, 1>(p, c, dev, stream) : launch<64, 2>(p, c, dev, stream);
  if (dim <= 128) return one ? launch<128, 1>(p, c, dev, stream) : launch<128, 2>(p, c, dev, stream);
  return launch<256, 1>(p, c, dev, stream);
}

}  // namespace sv
