// Attention over the paged cache for few query rows (a decoded token's heads, a
// short chain's): bf16, tiles of 16 rows and 128 keys.
//
// Bound by the bytes of K and V: of the 16 x 8 x 16 matrix instructions' rows
// most are often empty, and their rate is still not what limits.  So the layout
// serves the loads: the ring of sv_attention_ring.cuh runs ahead, eight warps
// take 16 keys of a tile each, with their own running (m, l, O) in registers,
// and meet only at the end of a unit, where they join by halves, and the first
// of them writes the rows while the others go on.  The units that a block
// shares with others are joined at its end, by all its threads.
//
// The matrix unit takes operands of one type, so the weights go to the product
// with V as two bf16 values, their upper half and the rounding of what it leaves
// (16 bits together); their sum l is in fp32.  Where the weight is above 0 both
// are: an infinity of V times one of 0, or of the other sign, would be NaN.  The
// second value costs little where the bytes are what limits: heads of 128 321.9
// us with one and 323.5 with two, of 256 327 and 330, of 96 276 and 284, of 64
// 224 and 231.
//
// Measured: one token of 128 requests of up to 8192, 32 heads of 128 on 8 in the
// cache: 318 to 323 us, 6.7 TB/s; 64 requests, heads of 256: 330 us, 6.7 TB/s; one
// of a single request of 100000: 77 us, 5.3 TB/s; of 500: 12 us, latency.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>
#include <mutex>

#include "sv_attention_ring.cuh"

namespace sv {
namespace {

constexpr int kRows = 16;
constexpr int kTakers = 8;                                      // warps that take the tiles
constexpr int kFewThreads = 32 * (kTakers + kLoadWarps + 2);    // and a warp each to plan, to load Q
constexpr int kUnitPlaces = 2;  // what a unit costs beside its key tiles, in tiles (1 to 3 measure alike)

// Heads of up to 64 (CB 1), 128 (CB 2) and 256 (CB 2, H 2) columns.  With H of 2 a warp has the scores of 32 keys and one
// entry's columns of O: the scores are taken twice, O would not fit the registers otherwise.
template <int CB, int H>
struct Few {
  static constexpr int kRing = CB == 2 ? 5 : 10;  // entries in the ring
  using R = KvRing<2, CB, kRing, H>;
  static constexpr int kCols = CB * 64, kDP = kCols * H;
  static constexpr int kGroups = kTakers / H;        // key groups
  static constexpr int kOwn = kKeys / kGroups;       // keys of a warp
  static constexpr int DT = kCols / 8, KS = kCols / 16, NT = kOwn / 8;
  static constexpr int kStage = (DT + 1) * 32 * 16;  // a warp's O, m and l
  // shared memory: the ring; two Qs of 16 rows; half the warps' results; the warps' flags; the meeting point; last; split segments
  static constexpr int kQBlock = 2 * kRows * 128;
  static constexpr int kQ = (R::kBytes + 1023) / 1024 * 1024;
  static constexpr int kStages = kQ + kQBlock * CB * H;
  static constexpr int kFlags = kStages + kTakers / 2 * kStage;
  static constexpr int kMeet = kFlags + 2 * kTakers * 8;
  static constexpr int kParts = kMeet + 2 * 8;
  static constexpr int kSmem = kParts + 2 * static_cast<int>(sizeof(AttnSegment));
};

template <int CB, int H>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_attention_few(const AttnParams p, const __grid_constant__ KvMaps maps) {
  using W = Few<CB, H>;
  using R = typename W::R;
  constexpr int DT = W::DT, KS = W::KS, NT = W::NT, DP = W::kDP;
  extern __shared__ __align__(1024) char smem[];
  R ring(smem);
  const uint32_t base = smem_addr(smem);
  const uint32_t bar_meet = base + W::kMeet;
  uint32_t* s_flags = reinterpret_cast<uint32_t*>(smem + W::kFlags);  // [2][kTakers][2], by turns: keys outside the cache, careful
  AttnSegment* s_parts = reinterpret_cast<AttnSegment*>(smem + W::kParts);
  int* s_last = reinterpret_cast<int*>(smem + W::kMeet + 8);
  int* s_split = s_last + 1;  // segments of the block that are only part of their unit
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    ring.init(kTakers, kTakers + kLoadWarps + 1, kTakers);
    mbar_init(bar_meet, 32 * kTakers);
    mbar_fence_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const AttnSpan span = attn_span<kRows, kKeys, kUnitPlaces, kFewThreads>(p, t, ring.sums(), ring.find(),
                                                                          [] { __syncthreads(); });
  if (warp == kTakers + kLoadWarps) {
    const int split = ring.template plan<kRows, kUnitPlaces>(p, span, s_parts);
    if (lane == 0) *s_split = split;
  } else if (warp == kTakers + kLoadWarps + 1) {
    ring.template load_q<kRows>(p, base + W::kQ, W::kQBlock, 2, kRows);
  } else if (warp >= kTakers) {
    ring.load(p, maps, warp - kTakers);
  } else {
    const int group = warp % W::kGroups, part_of_row = warp / W::kGroups;  // its keys, its columns of O
    const int k0 = group * W::kOwn, d0 = part_of_row * W::kCols;
    // What this lane addresses for ldmatrix within a tile (piece(row, column)): the pieces of a row further on differ from
    // it in bits 5 and 6 of the address, or by a block.
    const int mi = lane >> 3, mr = lane & 7;  // matrix and row
    const uint32_t k_at = R::piece(k0 + (mi >> 1) * 8 + mr, mi & 1), v_at = R::piece(k0 + (mi & 1) * 8 + mr, mi >> 1);
    uint32_t meets = 0, g = 0;
    auto meet = [&] {  // a barrier of the taking warps, bounded like every wait
      mbar_arrive(bar_meet);
      return ring.wait(bar_meet, meets++ & 1);
    };
    auto done = [&](uint32_t bar) {  // this warp needs the buffer no more
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    for (uint32_t unit = 0; ok; ++unit) {
      const AttnSegment* const seg = ring.peek();
      if (!seg) break;
      const AttnSegment& s = *seg;
      const int rows = s.r.n * p.group - s.rt * kRows;  // rows of the unit from this tile on
      const int slot = unit & 1;
      if (!ring.wait(ring.q_bar(slot), unit >> 1 & 1)) break;
      const int q_row = slot * kRows + (lane & 15);  // this lane's row of Q for ldmatrix
      const uint32_t q_at = base + W::kQ + q_row * 128 + (((lane >> 4) ^ (q_row & 7)) << 4);
      float m[2] = {-kInfF, -kInfF}, l[2] = {0.0f, 0.0f};
      float o[DT][4];
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
      uint32_t bad = 0u;
      bool careful = false;
#pragma unroll 1
      for (int i = 0; i < s.cnt; ++i, ++g) {
        const int x0 = (s.t0 + i) * kKeys + k0;  // the warp's first key
        if (!ring.wait(ring.full(2 * H * g), ring.phase(2 * H * g))) {
          ok = false;
          break;
        }
        const uint32_t all = W::kOwn == 32 ? 0xffffffffu : 0xffffu;
        const uint32_t good = ring.valid(g)[k0 / 32] >> (k0 & 31) & all;
        bad |= ring.valid(g)[4 + k0 / 32];
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const uint32_t group_k = 2 * H * g + h;
          if (h > 0 && !ring.wait(ring.full(group_k), ring.phase(group_k))) ok = false;
          const uint32_t kt = ring.tile(group_k) + k_at;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t qf[4];  // (Q stays in shared memory: O, the scores and Q do not fit the registers together)
            ldmatrix4((q_at ^ (ks & 3) << 5) + (h * CB + (ks >> 2)) * W::kQBlock, qf);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
              uint32_t kb[4];
              ldmatrix4((kt ^ (ks & 3) << 5) + (ks >> 2) * R::kBlock + n * 1024, kb);
              mma_bf16(sc[n], qf, kb[0], kb[1]);
              mma_bf16(sc[n + 1], qf, kb[2], kb[3]);
            }
          }
          done(ring.empty(group_k));
        }
        if (!ok) break;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[n][c] *= p.scale_log2;
        if (good != all || x0 + W::kOwn > s.r.len) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = (s.rt * kRows + (lane >> 2) + h * 8) / p.group;
            const uint32_t see = row_sees_of(p, s.r, s.b, row, x0, good) >> ((lane & 3) * 2);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (!(see >> (n * 8 + c) & 1u)) sc[n][h * 2 + c] = -kInfF;
          }
        }
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = m[h];
#pragma unroll
          for (int n = 0; n < NT; ++n) mx = fmax_nan(mx, fmax_nan(sc[n][h * 2], sc[n][h * 2 + 1]));
          mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float ref = mx == -kInfF ? 0.0f : mx;
          alpha[h] = ex2_fast(m[h] - ref);
          m[h] = mx;
          l[h] *= alpha[h];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = ex2_fast(sc[n][h * 2 + c] - ref);
              sc[n][h * 2 + c] = x;
              l[h] += x;
            }
        }
        // O moves to the new maximum only when one of the warp's rows has a new one
        if (__any_sync(0xffffffffu, !(alpha[0] == 1.0f && alpha[1] == 1.0f))) {
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[d][0] *= alpha[0], o[d][1] *= alpha[0];
            o[d][2] *= alpha[1], o[d][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const uint32_t group_v = 2 * H * g + H + h;
          if (!ring.wait(ring.full(group_v), ring.phase(group_v))) {
            ok = false;
            break;
          }
          if (h != part_of_row) {  // (a warp that does not need the entry has still to know that it came)
            done(ring.empty(group_v));
            continue;
          }
          if (new_rows_differ(p, s.r) && x0 + W::kOwn > s.r.len) {
            char* v = ring.tile_mem(group_v);
            bool found = false;
#pragma unroll 1
            for (int x = max(s.r.len - x0, 0) * R::kPieces + lane; x < min(s.r.len + s.r.n - x0, W::kOwn) * R::kPieces; x += 32)
              if (make_finite<true>(reinterpret_cast<uint4*>(v + R::piece(k0 + x / R::kPieces, x % R::kPieces)))) found = true;
            __syncwarp();  // what a lane took out, another reads (a vote orders no memory)
            careful = __any_sync(0xffffffffu, found) || careful;
          }
          const uint32_t vt = ring.tile(group_v) + v_at;
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t a[4], rest[4];  // the weights' upper halves, and what is left
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = sc[n + (i >> 1)][(i & 1) * 2], y = sc[n + (i >> 1)][(i & 1) * 2 + 1];
              a[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
              // (a weight above 0 is 2^-126 at least)
              rest[i] = pack_bf16(fmaxf(x - bf16_lo(a[i]), fminf(x, 0x1p-126f)), fmaxf(y - bf16_hi(a[i]), fminf(y, 0x1p-126f)));
            }
#pragma unroll
            for (int d = 0; d < DT; d += 2) {
              uint32_t vb[4];
              ldmatrix4_trans((vt ^ (d & 6) << 4) + (d >> 3) * R::kBlock + n * 1024, vb);
              mma_bf16(o[d], a, vb[0], vb[1]);
              mma_bf16(o[d + 1], a, vb[2], vb[3]);
              mma_bf16(o[d], rest, vb[0], vb[1]);
              mma_bf16(o[d + 1], rest, vb[2], vb[3]);
            }
          }
          done(ring.empty(group_v));
        }
        if (!ok) break;
      }
      if (!ok) break;
      done(ring.q_free(slot));

      // The warps' results, joined by halves: warp w + h into warp w for h = 4, 2, 1.  A lane has the same rows and columns
      // in every warp.  (What h leaves lies where no warp of the step before reads: the steps meet in between.)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      }
      uint32_t* const flags = s_flags + slot * kTakers * 2;
      if (lane == 0) flags[warp * 2] = bad, flags[warp * 2 + 1] = careful ? 1u : 0u;
      auto stage = [&](int i) { return reinterpret_cast<float4*>(smem + W::kStages + i * W::kStage) + lane; };
      auto leave = [&](float4* to) {
#pragma unroll
        for (int d = 0; d < DT; ++d) to[d * 32] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
        to[DT * 32] = make_float4(m[0], m[1], l[0], l[1]);
      };
      auto take = [&](const float4* from) {
        const float4 x = from[DT * 32];
        float wa[2], wb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mb = h ? x.y : x.x, N = fmax_nan(m[h], mb), ref = N == -kInfF ? 0.0f : N;
          wa[h] = ex2_fast(m[h] - ref), wb[h] = ex2_fast(mb - ref);
          m[h] = N;
          l[h] = fmaf(l[h], wa[h], (h ? x.w : x.z) * wb[h]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const float4 v = from[d * 32];
          o[d][0] = fmaf(o[d][0], wa[0], v.x * wb[0]), o[d][1] = fmaf(o[d][1], wa[0], v.y * wb[0]);
          o[d][2] = fmaf(o[d][2], wa[1], v.z * wb[1]), o[d][3] = fmaf(o[d][3], wa[1], v.w * wb[1]);
        }
      };
      ok = true;
#pragma unroll 1
      for (int h = W::kGroups / 2; h > 0; h /= 2) {
        if (group >= h && group < 2 * h) leave(stage(part_of_row * (W::kGroups / 2) + group - h));
        ok = meet();
        if (!ok) break;
        if (group < h) take(stage(part_of_row * (W::kGroups / 2) + group));
        ok = meet();
        if (!ok) break;
      }
      if (!ok) break;
      if (group == 0) {
        uint32_t any = 0u, odd = 0u;
#pragma unroll
        for (int w = 0; w < kTakers; ++w) any |= flags[w * 2], odd |= flags[w * 2 + 1];
        bad = (any ? kStSlotRange : 0u) | s.r.status;
        const bool whole = s.cnt == s.nt;
        using P = AttnPart<kRows, DP>;
        float* part = attn_part<kRows, DP>(p, blockIdx.x, s.t0 == 0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = (lane >> 2) + h * 8, grow = s.rt * kRows + row;
          if (row >= rows) continue;
          if (whole) {
            const int i = grow / p.group, head = s.hkv * p.group + grow - i * p.group;
            const bool none = m[h] == -kInfF;  // nothing seen, or only scores of -inf
            const float inv = none ? 0.0f : 1.0f / l[h];
            char* out = p.out + ((s.r.row0 + i) * p.o_row + head * p.o_head + d0 + (lane & 3) * 2) * 2;
#pragma unroll
            for (int d = 0; d < DT; ++d)
              if (d0 + d * 8 < p.c.head_dim)
                *reinterpret_cast<uint32_t*>(out + d * 16) = none ? 0u : pack_bf16(o[d][h * 2] * inv, o[d][h * 2 + 1] * inv);
            if (d0 == 0 && (lane & 3) == 0 && p.lse) p.lse[(s.r.row0 + i) * p.heads + head] = none ? -kInfF : fmaf(m[h], kLn2, logf(l[h]));
          } else {
#pragma unroll
            for (int d = 0; d < DT; ++d)  // quads of columns, a quad by two lanes
              *reinterpret_cast<float2*>(part + ((d0 / 4 + d * 2 + (lane >> 1 & 1)) * kRows + row) * 4 + (lane & 1) * 2) =
                  make_float2(o[d][h * 2], o[d][h * 2 + 1]);
            if (d0 == 0 && (lane & 3) == 0) part[P::kM + row] = m[h], part[P::kL + row] = l[h];
          }
        }
        if (odd) {
          uint32_t none = 0u;
#pragma unroll
          for (int h = 0; h < 2; ++h) none |= __reduce_or_sync(0xffffffffu, m[h] == -kInfF ? 1u << ((lane >> 2) + h * 8) : 0u);
          add_nonfinite<true, kRows, W::kCols>(p, s, rows, d0, none, whole ? nullptr : part);
        }
        if (whole) {
          if (s.reports && warp == 0 && lane == 0) p.status[s.b] = bad | attn_timeout(p);
        } else {
          if (warp == 0 && lane == 0) part[P::kStatus] = __uint_as_float(bad);
        }
      }
      ring.release();
    }
  }
  __syncthreads();
  if (*ring.abort())
    ring.report_abort(p);
  else
    attn_join<true, kRows, DP, kFewThreads>(p, span, s_parts, *s_split, s_last);
}

template <int CB, int H>
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
      e = cudaFuncSetAttribute(k_attention_few<CB, H>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<CB, H>::kSmem);
      if (e != cudaSuccess) return e;
      have[d] = true;
    }
  }
  static_assert(Few<CB, H>::kSmem <= 227 * 1024, "shared memory of a block");
  const int grid = dev.sms < kAttnMaxBlocks ? dev.sms : kAttnMaxBlocks;
  return launch_pdl(k_attention_few<CB, H>, dim3(static_cast<unsigned>(grid)), dim3(kFewThreads), Few<CB, H>::kSmem, stream, p,
                    kv_maps(p.c));
}

}  // namespace

cudaError_t launch_attention_few(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int dim = p.c.head_dim;
  return dim <= 64 ? launch<1, 1>(p, dev, stream) : dim <= 128 ? launch<2, 1>(p, dev, stream) : launch<2, 2>(p, dev, stream);
}

}  // namespace sv
