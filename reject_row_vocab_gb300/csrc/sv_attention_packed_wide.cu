// Attention over the 4-bit cache for many query rows: the kernel of
// sv_attention_wide.cu on tiles that the loading warps unpack to bf16 (which
// holds the cache's values exactly).
//
// Eight loading warps take 16 keys of a tile each.  A lane has one key's 32
// columns (16 bytes of codes, two scales) of each block of 64: it fetches them
// a tile ahead, and writes 64 bytes of bf16 in the swizzle that the matrix unit
// reads.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include "sv_attention_packed.cuh"
#include "sv_attention_wide.cuh"

namespace sv {
namespace {

// Four pairs of bf16 from eight codes: a code's half float, its exponent moved to bf16's place, is the value times 2^-112,
// which the scale brings back.
__device__ __forceinline__ uint4 unpack_bf16(uint32_t w, uint32_t scale2) {
  uint32_t h[4];
  unpack_codes(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((h[i] >> 3) & 0x0fff0fffu) | (h[i] & 0x80008000u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(m), "r"(scale2));
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// A scale times 2^112 in both halves.
__device__ __forceinline__ uint32_t bf16_scale2(uint32_t byte) {
  uint32_t r;
  const float s = scale_value(byte) * 0x1p112f;
  asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(s));
  return r;
}

struct PackedSource {
  using Args = PackedView;
  static constexpr int kWarps = 8, kFulls = kWarps;
  static constexpr bool kFinite = true;

  template <class R>
  static __device__ void load(R& ring, const AttnParams& p, const Args& c, int lw) {
    constexpr int kEntries = R::kPieces / 8;  // blocks of 64 columns in an entry
    constexpr int H = R::kHalves, kBlocks = kEntries * H;
    const int lane = ring.lane, mine = lw * 16 + (lane >> 1);  // this lane's key of a tile
    const int v_codes = packed_v_codes(c.page_size, c.head_dim), k_scales = packed_k_scales(c.page_size, c.head_dim);
    const int v_scales = packed_v_scales(c.page_size, c.head_dim);
    struct Tile {
      uint4 codes[2][kBlocks];       // of K, of V
      uint32_t scales[2][kBlocks];   // two bytes
      uint32_t good, bad;            // a bit for each of the warp's keys
    };
    AttnSegment s{};
    bool more = ring.next(s);
    int t = s.t0;
    int64_t word = more ? key_word(p, s.r, s.b, t * kKeys + mine) : -1;
    // The next tile's bytes; false behind the last tile.
    auto fetch = [&](Tile& f) {
      if (!more) return false;
      const int x = t * kKeys + mine, hkv = s.hkv, keys = s.r.len + s.r.n;
      const Place at = packed_place(p, c, s.r, x, word);
      const bool there = at.page >= 0;
      const uint32_t good = __ballot_sync(0xffffffffu, there), bad = __ballot_sync(0xffffffffu, x < keys && !there);
      f.good = good, f.bad = bad;
      if (++t >= s.t0 + s.cnt) {
        more = ring.next(s);
        t = s.t0;
      }
      if (more) word = key_word(p, s.r, s.b, t * kKeys + mine);
      const char* block = c.data + at.page * c.page_stride + hkv * c.head_stride;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int d = i * 64 + (lane & 1) * 32;
          f.codes[k][i] = make_uint4(0u, 0u, 0u, 0u);
          f.scales[k][i] = 0u;
          if (there && d < c.head_dim) {
            f.codes[k][i] = *reinterpret_cast<const uint4*>(block + (k ? v_codes : 0) + at.in * (c.head_dim / 2) + d / 2);
            f.scales[k][i] = *reinterpret_cast<const uint16_t*>(block + (k ? v_scales : k_scales) +
                                                                at.in * (c.head_dim / 16) + d / 16);
          }
        }
      return true;
    };
    uint32_t q = 0;
    Tile next_tile;
    bool have = fetch(next_tile);
    for (bool ok = true; have && ok;) {
      const Tile f = next_tile;
      have = fetch(next_tile);
      const uint32_t g = q / (2 * H);
#pragma unroll
      for (int e = 0; e < 2 * H; ++e, ++q) {
        if (q >= R::kEntries && !ring.wait(ring.empty(q), R::phase(q - R::kEntries))) {
          ok = false;
          break;
        }
        if (e == 0 && lane < 16) {
          // (a key is two lanes' bits)
          const uint32_t there = __ballot_sync(0xffffu, f.good >> (2 * lane) & 1u);
          const uint32_t missing = __ballot_sync(0xffffu, f.bad >> (2 * lane) & 1u);
          if (lane == 0) {
            reinterpret_cast<uint16_t*>(ring.valid(g))[lw] = static_cast<uint16_t>(there);
            reinterpret_cast<uint16_t*>(ring.valid(g) + 4)[lw] = static_cast<uint16_t>(missing);
          }
        }
        char* tile = ring.tile_mem(q);
        constexpr int kK = 0;
        const int which = e >= H ? 1 : kK;
#pragma unroll
        for (int i = 0; i < kEntries; ++i) {
          const int n = (e % H) * kEntries + i;
          const uint4 w = f.codes[which][n];
          const uint32_t s0 = bf16_scale2(f.scales[which][n] & 0xffu), s1 = bf16_scale2(f.scales[which][n] >> 8);
          const int c0 = i * 8 + (lane & 1) * 4;
          *reinterpret_cast<uint4*>(tile + R::piece(mine, c0)) = unpack_bf16(w.x, s0);
          *reinterpret_cast<uint4*>(tile + R::piece(mine, c0 + 1)) = unpack_bf16(w.y, s0);
          *reinterpret_cast<uint4*>(tile + R::piece(mine, c0 + 2)) = unpack_bf16(w.z, s1);
          *reinterpret_cast<uint4*>(tile + R::piece(mine, c0 + 3)) = unpack_bf16(w.w, s1);
        }
        fence_async();  // (the matrix unit reads through the asynchronous proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.full(q));
      }
    }
  }
};

}  // namespace

cudaError_t launch_packed_attention_wide(const AttnParams& p, const PackedView& c, const DeviceInfo& dev, cudaStream_t stream) {
  const int dim = c.head_dim;
  return dim <= 64    ? launch_wide<1, 1, PackedSource>(p, c, dev, stream)
         : dim <= 128 ? launch_wide<2, 1, PackedSource>(p, c, dev, stream)
                      : launch_wide<2, 2, PackedSource>(p, c, dev, stream);
}

}  // namespace sv
