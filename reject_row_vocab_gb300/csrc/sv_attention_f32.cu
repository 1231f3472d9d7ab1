// Attention over the paged cache in fp32, plain arithmetic throughout: tiles of
// 4 or 8 query rows and 128 keys.
//
// One unit for a request and cache head is bound by the bytes of K and V: 8 rows
// and 128 keys of 128 columns are 2048 cycles of an SM's multiply-adds, their K
// and V 5500 cycles of its share of the memory's bandwidth.  Several units read
// them again from L2, and are bound by issue and latency, two such warps to a
// scheduler.  Shared memory stands between, so a value taken from it serves
// several: in the scores a lane has
// four keys and eight rows of its eighth of the columns (12 reads of 16 bytes
// for 128 multiply-adds; the eighths are summed by halving exchanges, after
// which a lane has one row's scores of its keys), in the sums four columns of
// every row.  Eight warps take 16 keys of a tile each, with their own running
// (m, l, O), joined at the end of a unit.
//
// Measured: one token of 64 requests of up to 8192, 32 heads of 128 on 8 in the
// cache: 339 us, 6.5 TB/s; 64 heads on 8: 366 us; blocks of 16 rows of 32 requests
// of up to 4000, 64 rows a request and cache head: 742 us, 24 TFLOP/s; ragged
// blocks of 1 to 8 rows of 24 requests of up to 900, heads of 64: 24 us, latency.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>
#include <mutex>

#include "sv_attention_ring.cuh"

namespace sv {
namespace {

constexpr int kTakers = 8;                                    // warps that take the tiles
constexpr int kThreads = 32 * (kTakers + kLoadWarps + 2);     // and a warp each to plan, to load Q
constexpr int kOwn = kKeys / kTakers;                         // keys of a warp
constexpr int kUnitPlaces = 1;                                // what a unit costs beside its key tiles, in tiles

// Heads of up to 64 H columns, units of R rows.
template <int H, int R>
struct Plain {
  static constexpr int kRing = 5;
  using Ring = KvRing<4, 2, kRing, H>;
  static constexpr int kDP = 64 * H;
  static constexpr int kVals = R / 2;               // scores that a lane is left with
  static constexpr int kPairs = H < 2 ? 1 : H / 2;  // a lane's quads of columns: one of each pair of entries
  static constexpr int kQRows = 8;                  // rows a Q has (the swizzle's period)
  // shared memory: the ring; two Qs; half the warps' results; each warp's weights [16][R] and row scales [R]; the warps' m,
  // l and flags; the unit's m and l; meeting point, last, split; split segments
  static constexpr int kQBlock = 2 * kQRows * 128;
  static constexpr int kQ = (Ring::kBytes + 1023) / 1024 * 1024;
  static constexpr int kStage = R * kPairs * 32 * 16;
  static constexpr int kStages = kQ + kQBlock * 2 * H;
  static constexpr int kWeights = kStages + kTakers / 2 * kStage;
  static constexpr int kWarpWeights = (kOwn + 1) * R * 4;
  static constexpr int kM = kWeights + kTakers * kWarpWeights;  // m, then l: [2 by turns][kTakers][R] each
  static constexpr int kFlags = kM + 4 * kTakers * R * 4;
  static constexpr int kMeet = kFlags + 2 * kTakers * 8;
  static constexpr int kParts = kMeet + 2 * 8;
  static constexpr int kSmem = kParts + 2 * static_cast<int>(sizeof(AttnSegment));
};

template <int H, int R>
__global__ void __launch_bounds__(kThreads, 1) k_attention_f32(const AttnParams p, const __grid_constant__ KvMaps maps) {
  using W = Plain<H, R>;
  using Ring = typename W::Ring;
  constexpr int DP = W::kDP, VALS = W::kVals, PAIRS = W::kPairs;
  extern __shared__ __align__(1024) char smem[];
  Ring ring(smem);
  const uint32_t base = smem_addr(smem);
  const uint32_t bar_meet = base + W::kMeet;
  int* s_last = reinterpret_cast<int*>(smem + W::kMeet + 8);
  int* s_split = s_last + 1;  // segments of the block that are only part of their unit
  uint32_t* s_flags = reinterpret_cast<uint32_t*>(smem + W::kFlags);  // [2][kTakers][2], by turns: keys outside the cache, careful
  AttnSegment* s_parts = reinterpret_cast<AttnSegment*>(smem + W::kParts);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) {
    ring.init(kTakers, kTakers + kLoadWarps + 1, kTakers);
    mbar_init(bar_meet, 32 * kTakers);
    mbar_fence_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const AttnSpan span = attn_span<R, kKeys, kUnitPlaces, kThreads>(p, t, ring.sums(), ring.find(), [] { __syncthreads(); });
  if (warp == kTakers + kLoadWarps) {
    const int split = ring.template plan<R, kUnitPlaces>(p, span, s_parts);
    if (lane == 0) *s_split = split;
  } else if (warp == kTakers + kLoadWarps + 1) {
    ring.template load_q<R>(p, base + W::kQ, W::kQBlock, 2, W::kQRows);
  } else if (warp >= kTakers) {
    ring.load(p, maps, warp - kTakers);
  } else {
    const int k0 = warp * kOwn;  // this warp's keys of a tile
    // For the scores: keys key + 4 j, and of each block of eight pieces the piece `eighth` (in the order in which eight
    // lanes side by side find their pieces in different banks).
    const int key = lane & 3, eighth = (lane >> 2 & 1) << 2 | lane >> 3;
    // What the exchanges leave a lane with: row `row`, keys key + 4 (j0 + j), j < VALS.
    const int row = R == 8 ? lane >> 2 : lane >> 3, j0 = R == 8 ? 0 : (lane >> 2 & 1) * 2;
    const bool leads = key == 0 && (R == 8 || (lane >> 2 & 1) == 0);  // one lane a row
    // For the sums: piece lane of the 32 of a pair of entries, or (one entry) piece lane & 15, every other key.
    const int piece = H == 1 ? lane & 15 : lane, odd = H == 1 ? lane >> 4 : 0;
    float* const pw = reinterpret_cast<float*>(smem + W::kWeights + warp * W::kWarpWeights);  // [kOwn][R]
    float* const scales = pw + kOwn * R;                                                      // [R]
    uint32_t meets = 0, g = 0;
    auto meet = [&] {                     // a barrier of the taking warps, bounded like every wait
      mbar_arrive(bar_meet);
      return ring.wait(bar_meet, meets++ & 1);
    };
    auto done = [&](uint32_t bar) {  // this warp needs the buffer no more
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // every row's O times its entry of `scales`
    float4 o[PAIRS][R];
    auto rescale = [&](const float* by) {
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 a4 = *reinterpret_cast<const float4*>(by + r);
        const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < PAIRS; ++x) {
            float4& v = o[x][r + i];
            v.x *= a[i], v.y *= a[i], v.z *= a[i], v.w *= a[i];
          }
      }
    };
    bool ok = true;
    for (uint32_t unit = 0; ok; ++unit) {
      const AttnSegment* const seg = ring.peek();
      if (!seg) break;
      const AttnSegment& s = *seg;
      const int rows = s.r.n * p.group - s.rt * R;  // rows of the unit from this tile on
      const int slot = unit & 1;
      if (!ring.wait(ring.q_bar(slot), unit >> 1 & 1)) break;
      const char* const q_at = smem + W::kQ + slot * W::kQRows * 128;
      float m = -kInfF, l = 0.0f;  // of the lane's row
#pragma unroll
      for (int x = 0; x < PAIRS; ++x)
#pragma unroll
        for (int r = 0; r < R; ++r) o[x][r] = make_float4(0.f, 0.f, 0.f, 0.f);
      uint32_t bad = 0u;
      bool careful = false;
#pragma unroll 1
      for (int i = 0; i < s.cnt; ++i, ++g) {
        const int x0 = (s.t0 + i) * kKeys + k0;  // the warp's first key
        uint32_t good = 0u;
        float acc[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = acc[r][2] = acc[r][3] = 0.0f;
#pragma unroll 1
        for (int h = 0; h < H; ++h) {
          const uint32_t group = 2 * H * g + h;
          if (!ring.wait(ring.full(group), ring.phase(group))) {
            ok = false;
            break;
          }
          const char* kt = ring.tile_mem(group) + (k0 + key) * 128;
          const char* qt = q_at + h * 2 * W::kQBlock;
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // blocks of 32 columns
            float4 k[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              k[j] = *reinterpret_cast<const float4*>(kt + b * Ring::kBlock + j * 512 + ((eighth ^ key ^ (j & 1) << 2) << 4));
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float4 a = *reinterpret_cast<const float4*>(qt + b * W::kQBlock + r * 128 + ((eighth ^ r) << 4));
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                acc[r][j] = fmaf(a.x, k[j].x, acc[r][j]);
                acc[r][j] = fmaf(a.y, k[j].y, acc[r][j]);
                acc[r][j] = fmaf(a.z, k[j].z, acc[r][j]);
                acc[r][j] = fmaf(a.w, k[j].w, acc[r][j]);
              }
            }
          }
          if (h == H - 1) good = ring.valid(g)[warp / 2] >> (k0 & 16) & 0xffffu, bad |= ring.valid(g)[4 + warp / 2];
          done(ring.empty(group));
        }
        if (!ok) break;
        // The eighths' sums: each exchange halves what a lane has left, the rows first, by lane bits 4, 3, 2.
        float sc[VALS];
        {
          float a2[R / 2][4], a1[R / 4][4];
          const bool hi = lane >> 4 & 1, mid = lane >> 3 & 1, lo = lane >> 2 & 1;
#pragma unroll
          for (int r = 0; r < R / 2; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float give = hi ? acc[r][j] : acc[r + R / 2][j], keep = hi ? acc[r + R / 2][j] : acc[r][j];
              a2[r][j] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
            }
#pragma unroll
          for (int r = 0; r < R / 4; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float give = mid ? a2[r][j] : a2[r + R / 4][j], keep = mid ? a2[r + R / 4][j] : a2[r][j];
              a1[r][j] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
            }
#pragma unroll
          for (int j = 0; j < VALS; ++j) {
            float give, keep;
            if (R == 8)
              give = lo ? a1[0][j] : a1[R / 4 - 1][j], keep = lo ? a1[R / 4 - 1][j] : a1[0][j];
            else
              give = lo ? a1[0][j] : a1[0][(j + 2) & 3], keep = lo ? a1[0][(j + 2) & 3] : a1[0][j];
            sc[j] = (keep + __shfl_xor_sync(0xffffffffu, give, 4)) * p.scale_log2;
          }
        }
        if (good != 0xffffu || x0 + kOwn > s.r.len) {
          const uint32_t see = row_sees_of(p, s.r, s.b, (s.rt * R + row) / p.group, x0, good);
#pragma unroll
          for (int j = 0; j < VALS; ++j)
            if (!(see >> (key + 4 * (j0 + j)) & 1u)) sc[j] = -kInfF;
        }
        float mx = m;
#pragma unroll
        for (int j = 0; j < VALS; ++j) mx = fmax_nan(mx, sc[j]);
        mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (R == 4) mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        const float ref = mx == -kInfF ? 0.0f : mx;
        const float alpha = ex2_fast(m - ref);
        m = mx;
        l *= alpha;
        __syncwarp();  // the weights of the tile before are no longer read
#pragma unroll
        for (int j = 0; j < VALS; ++j) {
          const float x = ex2_fast(sc[j] - ref);
          l += x;
          pw[(key + 4 * (j0 + j)) * R + row] = x;
        }
        if (leads) scales[row] = alpha;
        const bool moved = __any_sync(0xffffffffu, !(alpha == 1.0f));
        __syncwarp();
        // O moves to the new maximum only when one of the warp's rows has a new one
        if (moved) rescale(scales);
#pragma unroll
        for (int x = 0; x < PAIRS; ++x) {
          constexpr int E = H < 2 ? 1 : 2;  // entries of a pair
          const uint32_t group = 2 * H * g + H + x * E;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (!ring.wait(ring.full(group + e), ring.phase(group + e))) ok = false;
          if (!ok) break;
          if (new_rows_differ(p, s.r) && x0 + kOwn > s.r.len) {
            bool found = false;
#pragma unroll 1
            for (int y = max(s.r.len - x0, 0) * Ring::kPieces * E + lane; y < min(s.r.len + s.r.n - x0, kOwn) * Ring::kPieces * E;
                 y += 32) {
              const int c = y % (Ring::kPieces * E);
              if (make_finite<false>(reinterpret_cast<uint4*>(ring.tile_mem(group + c / Ring::kPieces) +
                                                              Ring::piece(k0 + y / (Ring::kPieces * E), c % Ring::kPieces))))
                found = true;
            }
            __syncwarp();  // what a lane took out, another reads (a vote orders no memory)
            careful = __any_sync(0xffffffffu, found) || careful;
          }
          const char* vt = ring.tile_mem(group + (H == 1 ? 0 : lane >> 4)) + (piece >> 3 & 1) * Ring::kBlock + k0 * 128;
#pragma unroll 4
          for (int kk = 0; kk < kOwn; kk += H == 1 ? 2 : 1) {
            const int r0 = kk + odd;
            const float4 v = *reinterpret_cast<const float4*>(vt + r0 * 128 + (((piece & 7) ^ (r0 & 7)) << 4));
#pragma unroll
            for (int r = 0; r < R; r += 4) {
              const float4 w4 = *reinterpret_cast<const float4*>(pw + r0 * R + r);
              const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float4& a = o[x][r + y];
                a.x = fmaf(w[y], v.x, a.x), a.y = fmaf(w[y], v.y, a.y);
                a.z = fmaf(w[y], v.z, a.z), a.w = fmaf(w[y], v.w, a.w);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < E; ++e) done(ring.empty(group + e));
        }
        if (!ok) break;
      }
      if (!ok) break;
      done(ring.q_free(slot));

      // The warps' results: m and l of every warp first, then each warp's O on the unit's maximum, added by halves (warp
      // w + h to warp w for h = 4, 2, 1; what h leaves lies where no warp of the step before reads).
      float* const sm = reinterpret_cast<float*>(smem + W::kM) + slot * 2 * kTakers * R;
      float* const sl = sm + kTakers * R;
      float sum = l;
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (R == 4) sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      if (leads) sm[warp * R + row] = m, sl[warp * R + row] = sum;
      uint32_t* const flags = s_flags + slot * kTakers * 2;
      if (lane == 0) flags[warp * 2] = bad, flags[warp * 2 + 1] = careful ? 1u : 0u;
      if (H == 1) {  // the odd keys' sums
#pragma unroll
        for (int r = 0; r < R; ++r) {
          o[0][r].x += __shfl_xor_sync(0xffffffffu, o[0][r].x, 16);
          o[0][r].y += __shfl_xor_sync(0xffffffffu, o[0][r].y, 16);
          o[0][r].z += __shfl_xor_sync(0xffffffffu, o[0][r].z, 16);
          o[0][r].w += __shfl_xor_sync(0xffffffffu, o[0][r].w, 16);
        }
      }
      if (!meet()) break;
      float M = -kInfF, L = 0.0f;  // of row lane
      if (lane < R) {
#pragma unroll
        for (int w = 0; w < kTakers; ++w) M = fmax_nan(M, sm[w * R + lane]);
        const float ref = M == -kInfF ? 0.0f : M;
#pragma unroll
        for (int w = 0; w < kTakers; ++w) L = fmaf(ex2_fast(sm[w * R + lane] - ref), sl[w * R + lane], L);
        scales[lane] = ex2_fast(sm[warp * R + lane] - ref);
      }
      __syncwarp();
      rescale(scales);
#pragma unroll 1
      for (int h = kTakers / 2; h > 0; h /= 2) {
        float4* const stage = reinterpret_cast<float4*>(smem + W::kStages + (warp >= h ? warp - h : warp) * W::kStage) + lane;
        if (warp >= h && warp < 2 * h) {
#pragma unroll
          for (int x = 0; x < PAIRS; ++x)
#pragma unroll
            for (int r = 0; r < R; ++r) stage[(x * R + r) * 32] = o[x][r];
        }
        ok = meet();
        if (!ok) break;
        if (warp < h) {
#pragma unroll
          for (int x = 0; x < PAIRS; ++x)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float4 v = stage[(x * R + r) * 32];
              o[x][r].x += v.x, o[x][r].y += v.y, o[x][r].z += v.z, o[x][r].w += v.w;
            }
        }
        ok = meet();
        if (!ok) break;
      }
      if (!ok) break;
      if (warp == 0) {
        uint32_t any = 0u, odd_ones = 0u;
#pragma unroll
        for (int w = 0; w < kTakers; ++w) any |= flags[w * 2], odd_ones |= flags[w * 2 + 1];
        bad = (any ? kStSlotRange : 0u) | s.r.status;
        const bool whole = s.cnt == s.nt;
        using P = AttnPart<R, DP>;
        float* part = attn_part<R, DP>(p, blockIdx.x, s.t0 == 0);
        // lane r: where row r goes, and what its sums are multiplied by
        const int grow = s.rt * R + lane, new_row = grow / p.group, head = s.hkv * p.group + grow - new_row * p.group;
        const bool none = M == -kInfF;  // nothing seen, or only scores of -inf
        const float inv = none ? 0.0f : 1.0f / L;
        const int64_t to = ((s.r.row0 + new_row) * p.o_row + head * p.o_head) * 4;
        if (whole && lane < min(rows, R) && p.lse)
          p.lse[(s.r.row0 + new_row) * p.heads + head] = none ? -kInfF : fmaf(M, kLn2, logf(L));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float by = __shfl_sync(0xffffffffu, inv, r);
          char* at = p.out + __shfl_sync(0xffffffffu, to, r);
          const bool zero = __shfl_sync(0xffffffffu, none ? 1 : 0, r) != 0;
#pragma unroll
          for (int x = 0; x < PAIRS; ++x) {
            const int quad = x * 32 + piece;
            float4 v = o[x][r];
            if (whole) {
              v = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
              if (r < rows && !odd && quad * 4 < p.c.head_dim) *reinterpret_cast<float4*>(at + quad * 16) = v;
            } else if (!odd) {
              reinterpret_cast<float4*>(part)[quad * R + r] = v;
            }
          }
        }
        if (!whole && lane < R) part[P::kM + lane] = M, part[P::kL + lane] = L;
        if (odd_ones) add_nonfinite<false, R, DP>(p, s, rows, 0, __ballot_sync(0xffffffffu, none), whole ? nullptr : part);
        if (whole) {
          if (s.reports && lane == 0) p.status[s.b] = bad | attn_timeout(p);
        } else {
          if (lane == 0) part[P::kStatus] = __uint_as_float(bad);
        }
      }
      ring.release();
    }
  }
  __syncthreads();
  if (*ring.abort())
    ring.report_abort(p);
  else
    attn_join<false, R, DP, kThreads>(p, span, s_parts, *s_split, s_last);
}

template <int H, int R>
cudaError_t launch(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  static std::mutex mu;
  static bool have[64] = {};
  int d = 0;
  cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess) return e;
  if (d < 0 || d >= 64) return cudaErrorInvalidDevice;
  constexpr int kSmem = Plain<H, R>::kSmem;
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!have[d]) {
      e = cudaFuncSetAttribute(k_attention_f32<H, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      have[d] = true;
    }
  }
  const int grid = dev.sms < kAttnMaxBlocks ? dev.sms : kAttnMaxBlocks;
  return launch_pdl(k_attention_f32<H, R>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmem, stream, p, kv_maps(p.c));
}

// Units of 4 rows where they hold a request's rows of a cache head, else of 8: what a unit of 16 saves in reading, it
// loses in registers (O alone would be 64 of a lane's 128: blocks of 16 rows took 911 us instead of 849, ragged ones 40
// instead of 24).
template <int H>
cudaError_t launch_rows(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  return static_cast<int64_t>(p.max_len) * p.group <= 4 ? launch<H, 4>(p, dev, stream) : launch<H, 8>(p, dev, stream);
}

}  // namespace

cudaError_t launch_attention_f32(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int dim = p.c.head_dim;
  return dim <= 64 ? launch_rows<1>(p, dev, stream)
                   : dim <= 128 ? launch_rows<2>(p, dev, stream) : launch_rows<4>(p, dev, stream);
}

}  // namespace sv
