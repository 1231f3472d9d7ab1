// Attention over the 4-bit cache for many query rows: the kernel of
// sv_attention_wide.cuh on tiles that eight of its warps unpack to half floats,
// which hold the cache's values exactly.
//
// Each unpacking warp has 16 keys of a tile; a lane has 32 columns of one key
// in each block of 64: 16 bytes of codes, two scales, 64 bytes of half floats in
// the swizzle that the matrix unit reads.  Its operands have one type, so the
// queries are half floats too: each row of a unit's Q is brought to their range by
// a power of two, which the row's factor of the scores takes back (by the softmax
// warps, to tensor memory; of heads of more than 128 columns, for which that has no
// room, by the unpacking warps in shared memory).  The weights are half floats, below 2^14 with the sums in fp32 (their
// rounding, 2^-12, is below that of the output).
//
// A tile's bytes come by bulk copies (sv_attention_packed.cuh), some tiles ahead.
// Heads of more than 128 columns have no room for that, and pages of one or two
// entries no blocks worth a copy: there the unpacking warps fetch a tile ahead into
// registers (trees of 16 requests in pages of one slot: 24 us, by way of shared
// memory 41; 64 blocks of 16 rows in pages of 64 the other way round, 137 and 109,
// both with Q in shared memory).
//
// Bound by the softmax warps' chain, about 1700 clocks a tile (64 keys a thread), beside
// 1100 of the matrix unit, which multiplies 128 rows whether there are as many or not,
// and by a unit's end (5400 clocks: two threads' halves of a row are put together by
// way of 8 KB).  Measured: blocks of 16 rows of 64 requests of up to 4000, 32 heads of
// 128 on 8, pages of 64: 86 us (100 over bf16, for 3.6 times the bytes); trees of 17
// nodes of 16 requests in pages of one slot: 22 us; 5 rows of two requests of 60000 to
// 100000: 49 us (63); a causal block of 1024 rows of one request, pages of 16: 51 us
// without history, 118 behind 4000 (heads of 256: 90 and 300), K and V unpacked again for
// every tile of rows and all key tiles gone through.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include "sv_attention_packed.cuh"
#include "sv_attention_wide.cuh"

namespace sv {
namespace {

constexpr int kUnpackWarps = 8;

// Eight codes times a scale (both halves).
__device__ __forceinline__ uint4 unpack_half(uint32_t w, uint32_t scale2) {
  uint32_t h[4];
  unpack_codes(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = mul_half2(h[i], scale2);
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// 32 columns of one key, of codes `w` and two scales, to half floats at pieces c0 .. c0 + 3 of row r of a tile.
template <class R>
__device__ __forceinline__ void store_half(char* tile, int r, int c0, uint4 w, uint32_t scales) {
  const uint32_t s0 = scale_pair(__byte_perm(scales, 0u, 0x4040)), s1 = scale_pair(__byte_perm(scales, 0u, 0x4141));
  *reinterpret_cast<uint4*>(tile + R::piece(r, c0)) = unpack_half(w.x, s0);
  *reinterpret_cast<uint4*>(tile + R::piece(r, c0 + 1)) = unpack_half(w.y, s0);
  *reinterpret_cast<uint4*>(tile + R::piece(r, c0 + 2)) = unpack_half(w.z, s1);
  *reinterpret_cast<uint4*>(tile + R::piece(r, c0 + 3)) = unpack_half(w.w, s1);
}

// STAGED: through shared memory, by a warp that loads.
template <bool STAGED>
struct HalfSource {
  using Args = PackedTiles;
  static constexpr int kWarps = kUnpackWarps + (STAGED ? 1 : 0), kFulls = STAGED ? kUnpackWarps / 2 : kUnpackWarps;
  static constexpr bool kHalf = true;
  template <int CB, int H>
  static __host__ __device__ constexpr int entries() { return CB == 2 ? 4 : 8; }
  template <int CB, int H>
  using Stage = PackedStage<CB == 2 ? 3 : 4, 1, packed_tile_bytes(CB * 64 * H)>;
  // The source's shared memory: the places; what threads of one row tell each other, and 8 KB through which the second thread's O
  // goes to the first (where Q is in shared memory, its second copy is used for that); the rows' factors of the last eight
  // units, where Q is in shared memory (the unpacking warps are at most six tiles ahead of the softmax warps: a tile of K needs the
  // place of one four before it, whose product is issued behind the weights two before that); the barriers of a converted Q and
  // of a unit's end.
  template <int CB, int H>
  static __host__ __device__ constexpr int pairs_at() { return STAGED ? Stage<CB, H>::kBytes : 0; }
  template <int CB, int H>
  static __host__ __device__ constexpr int factors() { return pairs_at<CB, H>() + kRows * 8; }
  template <int CB, int H>
  static __host__ __device__ constexpr int ready() { return factors<CB, H>() + (H == 1 ? 64 * 128 : 8 * kRows * 4); }
  template <int CB, int H>
  static __host__ __device__ constexpr int extra_bytes() { return ready<CB, H>() + 16; }

  template <int CB, int H>
  static __device__ __forceinline__ void init(char* extra) {
    if constexpr (STAGED) Stage<CB, H>(extra).init(kUnpackWarps);
    mbar_init(smem_addr(extra) + ready<CB, H>(), H == 1 ? kSoftmaxThreads : kUnpackWarps);
    mbar_init(unit_done<CB, H>(extra), kSoftmaxThreads);
  }
  template <int CB, int H>
  static __device__ __forceinline__ uint32_t q_ready(char* extra) {
    return smem_addr(extra) + ready<CB, H>();
  }
  template <int CB, int H>
  static __device__ __forceinline__ uint32_t unit_done(char* extra) {
    return smem_addr(extra) + ready<CB, H>() + 8;
  }
  template <int CB, int H>
  static __device__ __forceinline__ float2* pairs(char* extra) {
    return reinterpret_cast<float2*>(extra + pairs_at<CB, H>());
  }
  // Of H = 2 there are two places: the second copy's rows of two blocks of Q, which are not used between a unit's last product and its end.
  template <int CB, int H>
  static __device__ __forceinline__ float4* exchange(char* q, char* extra, int i) {
    return reinterpret_cast<float4*>(H == 1 ? extra + factors<CB, H>() : q + 64 * 128 + i * kKeys * 128);
  }
  static __device__ __forceinline__ float2 row_range(uint32_t top, float scale) {
    const RowScale f = row_scale(top, scale);
    return make_float2(f.up, f.factor);
  }
  template <int CB, int H>
  static __device__ __forceinline__ float row_factor(char* extra, uint32_t unit, int t) {
    return reinterpret_cast<const volatile float*>(extra + factors<CB, H>())[unit % 8 * kRows + t];
  }

  // A warp's share of a unit's Q: rows of bf16 to half floats, in place, and (of units of up to 64 rows) once more 64 rows
  // further on, where the end of the unit before has to be over.
  template <int CB, int H, class R>
  static __device__ __forceinline__ bool convert_q(R& ring, const AttnParams& p, char* q, char* extra, const AttnSegment& s, uint32_t unit,
                                                   bool split, int lw) {
    constexpr int kPieces = R::kPieces * H, kAtOnce = 32 / kPieces;
    const int lane = ring.lane;
    if (!ring.wait(ring.q_bar(0), unit & 1)) return false;
    if (split && unit > 0 && !ring.wait(unit_done<CB, H>(extra), (unit - 1) & 1)) return false;
    // (with the rows of 0 that fill the last warp's)
    const int rows = min((s.r.n * p.group - s.rt * kRows + 31) & ~31, kRows), c = lane % kPieces;
    float* const factor = reinterpret_cast<float*>(extra + factors<CB, H>()) + unit % 8 * kRows;
    for (int r0 = lw * kAtOnce; r0 < rows; r0 += kUnpackWarps * kAtOnce) {
      const int r = r0 + lane / kPieces;
      char* const at = q + (c >> 3) * R::kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (r < rows) {
        const uint4 u = *reinterpret_cast<const uint4*>(at);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      }
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
      top = max(top & 0xffffu, top >> 16);
#pragma unroll
      for (int x = 1; x < kPieces; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
      const RowScale f = row_scale(top, fabsf(p.scale_log2));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_half(bf16_lo(w[i]) * f.up, bf16_hi(w[i]) * f.up);
      if (r < rows) {
        *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        if (split) *reinterpret_cast<uint4*>(at + 64 * 128) = make_uint4(w[0], w[1], w[2], w[3]);
        if (c == 0) factor[r] = fmaxf(f.factor, 1e-45f);
      }
    }
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_ready<CB, H>(extra));
    return true;
  }

  template <int CB, int H, class R>
  static __device__ __forceinline__ void load(R& ring, const AttnParams& p, const Args& k, char* q, char* extra, bool split, int lw) {
    if constexpr (STAGED) {
      const Stage<CB, H> stage(extra);
      if (lw == kUnpackWarps)
        stage.load(ring, p, k, 0);
      else
        unpack<CB, H>(ring, k, stage, lw);
    } else {
      fetch<CB, H>(ring, p, k.c, q, extra, split, lw);
    }
  }

  // A tile from its place, K by one half of the warps, V by the other.  (K's place is free again when its scores are there, V's only
  // behind the weights: by the same warps in turn, the next K waits for that: 64 blocks of 16 rows took 100 us that way and 96 this.)
  template <int CB, int H, class R, class S>
  static __device__ __forceinline__ void unpack(R& ring, const Args& k, const S& stage, int lw) {
    constexpr int kEntries = R::kEntries;
    static_assert(H == 1 && kEntries % 2 == 0, "one entry for K and one for V, in places of their own; Q is in tensor memory");
    const int lane = ring.lane, dim = k.c.head_dim, in_block = (1 << k.rows_log) - 1;
    const int is_v = lw / kFulls, quarter = lw % kFulls;  // 32 keys, 16 at once
    int code[2], scale[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int key = quarter * 32 + r * 16 + (lane >> 1), at_block = (key >> k.rows_log) * k.block;
      code[r] = at_block + (key & in_block) * (dim / 2) + (lane & 1) * 16 + (is_v ? packed_v_codes(in_block + 1, dim) : 0);
      scale[r] = at_block + (key & in_block) * (dim / 16) + (lane & 1) * 2 +
                 (is_v ? packed_v_scales(in_block + 1, dim) : packed_k_scales(in_block + 1, dim));
    }
    AttnSegment s;
    uint32_t g = 0;
    bool ok = true;
    while (ok && ring.next(s)) {
#pragma unroll 1
      for (int i = 0; i < s.cnt; ++i, ++g) {
        if (!ring.wait(stage.full(g), stage.phase(g))) {
          ok = false;
          break;
        }
        const char* place = stage.tile(g);
        uint4 w[2][CB];
        uint32_t b[2][CB];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int n = 0; n < CB; ++n) {
            const bool live = n * 64 + (lane & 1) * 32 < dim;
            w[r][n] = *reinterpret_cast<const uint4*>(place + code[r] + (live ? n * 32 : 0));
            b[r][n] = *reinterpret_cast<const uint16_t*>(place + scale[r] + (live ? n * 4 : 0));
            if (!live) b[r][n] = 0u;  // columns that a head does not have are 0
          }
        const uint32_t good = stage.info(g)[quarter], bad = stage.info(g)[4 + quarter];
        __syncwarp();
        if (lane == 0) mbar_arrive(stage.empty(g));
        const uint32_t entry = 2 * g + is_v;
        if (entry >= kEntries && !ring.wait(ring.empty(entry), R::phase(entry - kEntries))) {
          ok = false;
          break;
        }
        if (!is_v && lane == 0) ring.valid(g)[quarter] = good, ring.valid(g)[4 + quarter] = bad;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int n = 0; n < CB; ++n)
            store_half<R>(ring.tile_mem(entry), quarter * 32 + r * 16 + (lane >> 1), n * 8 + (lane & 1) * 4, w[r][n], b[r][n]);
        fence_async();  // (the matrix unit reads through the asynchronous proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.full(entry));
      }
    }
  }

  // A tile from the cache: the next one's bytes are fetched while this one's are unpacked.
  template <int CB, int H, class R>
  static __device__ __forceinline__ void fetch(R& ring, const AttnParams& p, const PackedView& c, char* q_mem, char* extra, bool split, int lw) {
    constexpr int kBlocks = CB * H;
    const int lane = ring.lane, mine = lw * 16 + (lane >> 1);
    const int v_codes = packed_v_codes(c.page_size, c.head_dim), k_scales = packed_k_scales(c.page_size, c.head_dim);
    const int v_scales = packed_v_scales(c.page_size, c.head_dim);
    struct Tile {
      uint4 codes[2][kBlocks];      // of K, of V
      uint32_t scales[2][kBlocks];  // two bytes
      uint32_t good, bad;           // two bits for each of the warp's keys
      bool first;                   // of its unit
    };
    AttnSegment s{};
    bool more = ring.next(s);
    int t = s.t0;
    uint32_t unit = 0;
    bool ok = H == 1 || !more || convert_q<CB, H>(ring, p, q_mem, extra, s, unit, split, lw);
    int64_t word = more ? key_word(p, s.r, s.b, t * kKeys + mine) : -1;
    auto ahead = [&](Tile& f) {  // the next tile's bytes; false behind the last tile
      if (!more || !ok) return false;
      const int x = t * kKeys + mine, keys = s.r.len + s.r.n;
      const Place at = packed_place(p, c, s.r, x, word);
      const bool there = at.page >= 0;
      f.good = __ballot_sync(0xffffffffu, there), f.bad = __ballot_sync(0xffffffffu, x < keys && !there);
      const char* block = c.data + at.page * c.page_stride + s.hkv * c.head_stride;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int d = i * 64 + (lane & 1) * 32;
          f.codes[e][i] = make_uint4(0u, 0u, 0u, 0u);
          f.scales[e][i] = 0u;
          if (there && d < c.head_dim) {
            f.codes[e][i] = *reinterpret_cast<const uint4*>(block + (e ? v_codes : 0) + at.in * (c.head_dim / 2) + d / 2);
            f.scales[e][i] = *reinterpret_cast<const uint16_t*>(block + (e ? v_scales : k_scales) +
                                                                at.in * (c.head_dim / 16) + d / 16);
          }
        }
      return true;
    };
    uint32_t q = 0;
    Tile next_tile;
    bool have = ahead(next_tile);
    while (have && ok) {
      const Tile f = next_tile;
      // The walk's next tile.  (A unit's Q is converted before its first tile is unpacked, and after the last of the unit before:
      // only then is its place sure to be given back.)
      bool turn = false;
      if (++t >= s.t0 + s.cnt) {
        more = ring.next(s);
        t = s.t0;
        turn = more;
      }
      if (more) word = key_word(p, s.r, s.b, t * kKeys + mine);
      have = ahead(next_tile);
      const uint32_t g = q / (2 * H);
#pragma unroll
      for (int e = 0; e < 2 * H; ++e, ++q) {
        if (q >= R::kEntries && !ring.wait(ring.empty(q), R::phase(q - R::kEntries))) {
          ok = false;
          break;
        }
        if (e == 0 && lane < 16) {  // (a key is two lanes' bits)
          const uint32_t there = __ballot_sync(0xffffu, f.good >> (2 * lane) & 1u);
          const uint32_t missing = __ballot_sync(0xffffu, f.bad >> (2 * lane) & 1u);
          if (lane == 0) {
            reinterpret_cast<uint16_t*>(ring.valid(g))[lw] = static_cast<uint16_t>(there);
            reinterpret_cast<uint16_t*>(ring.valid(g) + 4)[lw] = static_cast<uint16_t>(missing);
          }
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
          const int n = (e % H) * CB + i;
          store_half<R>(ring.tile_mem(q), mine, i * 8 + (lane & 1) * 4, f.codes[e >= H ? 1 : 0][n], f.scales[e >= H ? 1 : 0][n]);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.full(q));
      }
      if (H > 1 && ok && turn) ok = convert_q<CB, H>(ring, p, q_mem, extra, s, ++unit, split, lw);
    }
  }
};

}  // namespace

cudaError_t launch_packed_attention_wide(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream) {
  const PackedTiles tiles = packed_tiles(c);
  const int dim = c.head_dim;
  if (tiles.copies == 0 || tiles.rows_log < 2)
    return dim <= 64    ? launch_wide<1, 1, HalfSource<false>>(p, tiles, dev, stream)
           : dim <= 128 ? launch_wide<2, 1, HalfSource<false>>(p, tiles, dev, stream)
                        : launch_wide<2, 2, HalfSource<false>>(p, tiles, dev, stream);
  return dim <= 64    ? launch_wide<1, 1, HalfSource<true>>(p, tiles, dev, stream)
         : dim <= 128 ? launch_wide<2, 1, HalfSource<true>>(p, tiles, dev, stream)
                      : launch_wide<2, 2, HalfSource<false>>(p, tiles, dev, stream);
}

}  // namespace sv
