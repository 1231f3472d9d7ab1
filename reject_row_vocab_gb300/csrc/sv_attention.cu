// Attention of the verify rows over the paged cache ([E2D] §2.4: each node
// sees the committed history, its ancestors and itself).
//
//   s_x = scale q.k_x,  m = max s,  l = sum e^(s_x - m),  o = sum e^(s_x - m) v_x / l
//
// kept as running (m, l, O) over tiles of keys, in base 2 (scale log2(e) is
// folded into q), in fp32.  The division of the work and the join of its parts
// are described in sv_attention.cuh.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cmath>
#include <cstdint>
#include <mutex>

#include "sv_attention.cuh"

namespace sv {
namespace {

constexpr float kLn2 = 0.693147180559945309417f;

// ---------------------------------------------------------------------------------------------------------------------
// Engine: plain fp32 arithmetic.  Four warps of four rows each; a lane scores one key of the tile, then gathers columns.
// ---------------------------------------------------------------------------------------------------------------------

template <bool BF16>
__device__ __forceinline__ float4 load4(const char* p) {  // four elements as floats
  if (BF16) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  }
  return *reinterpret_cast<const float4*>(p);
}

template <bool BF16, int DP>
struct SimtEngine {
  static constexpr bool kBf16 = BF16;
  static constexpr int kDP = DP;
  static constexpr int MT = 16, KT = 32, WK = 1, THREADS = 128;
  static constexpr int ES = BF16 ? 2 : 4;
  static constexpr int ROW = DP * ES;              // bytes of a staged row
  static constexpr int STAGE = 2 * KT * ROW;       // K then V
  static constexpr int STAGES = STAGE > 32768 ? 2 : 3;
  static constexpr int NQ = DP >= 128 ? DP / 128 : 1;  // column quads a lane owns
  static constexpr int KS = DP == 64 ? 2 : 1;          // keys a warp's lanes work on side by side
  static constexpr int EXTRA = MT * DP * 4 + KT * MT * 4;  // Q as fp32, P

  float m[4], l[4];
  float4 o[4][NQ];
  float* q;
  float* pt;

  // 16-byte pieces of a row are swizzled over the banks by the row's number.
  __device__ static int piece(int row, int c) { return row * ROW + ((c ^ (row & 7)) << 4); }

  __device__ void init(const AttnParams& p, const AttnRequest& r, int hkv, int rt, char* extra) {
    q = reinterpret_cast<float*>(extra);
    pt = q + MT * DP;
    const int rows = r.n * p.group;
    for (int x = threadIdx.x; x < MT * (DP / 4); x += THREADS) {
      const int row = rt * MT + x / (DP / 4), d = (x % (DP / 4)) * 4;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < rows && d < p.c.head_dim) {
        const int64_t at = (r.row0 + row / p.group) * p.q_row + (hkv * p.group + row % p.group) * p.q_head + d;
        f = load4<BF16>(p.q + at * ES);
      }
      f.x *= p.scale_log2, f.y *= p.scale_log2, f.z *= p.scale_log2, f.w *= p.scale_log2;
      *reinterpret_cast<float4*>(q + x * 4) = f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -kInfF, l[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < NQ; ++j) o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
  }

  // One tile: keys x0 .. x0 + KT - 1; valid: which of them exist.
  __device__ void tile(const AttnParams& p, const AttnRequest& r, int b, int rt, int x0, const char* stage,
                       const uint32_t* valid) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const char* ks = stage;
    const char* vs = stage + KT * ROW;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < DP * ES / 16; ++c) {
      const char* kp = ks + piece(lane, c);
#pragma unroll
      for (int h = 0; h < 16 / (4 * ES); ++h) {
        const float4 k = load4<BF16>(kp + h * 4 * ES);
        const int d = c * (16 / ES) + h * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 a = *reinterpret_cast<const float4*>(q + (warp * 4 + i) * DP + d);
          s[i] = fmaf(a.x, k.x, s[i]);
          s[i] = fmaf(a.y, k.y, s[i]);
          s[i] = fmaf(a.z, k.z, s[i]);
          s[i] = fmaf(a.w, k.w, s[i]);
        }
      }
    }
    const bool masked = valid[0] != 0xffffffffu || x0 + KT > r.len;
    if (masked) {
      const int x = x0 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = (rt * MT + warp * 4 + i) / p.group;
        bool see = (valid[0] >> lane & 1u) != 0u && row < r.n;
        if (see && x >= r.len) see = row_sees(p, b, row, x - r.len);
        if (!see) s[i] = -kInfF;
      }
    }
    float pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = s[i];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      mx = fmax_nan(mx, m[i]);
      const float ref = mx == -kInfF ? 0.0f : mx;
      const float a = ex2_fast(m[i] - ref);
      pr[i] = ex2_fast(s[i] - ref);
      m[i] = mx;
      l[i] = fmaf(l[i], a, pr[i]);
#pragma unroll
      for (int j = 0; j < NQ; ++j) o[i][j].x *= a, o[i][j].y *= a, o[i][j].z *= a, o[i][j].w *= a;
      if (masked && s[i] == -kInfF) pr[i] = -1.0f;  // not seen: its V has no part, whatever it holds
    }
    *reinterpret_cast<float4*>(pt + lane * MT + warp * 4) = make_float4(pr[0], pr[1], pr[2], pr[3]);
    __syncwarp();
    for (int kk = 0; kk < KT; kk += KS) {
      const int key = KS == 1 ? kk : kk + (lane >> 4);
      const float4 w4 = *reinterpret_cast<const float4*>(pt + key * MT + warp * 4);
      const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        const int d = KS == 1 ? (lane + 32 * j) * 4 : (lane & 15) * 4;
        const int byte = d * ES;
        const float4 v = load4<BF16>(vs + piece(key, byte >> 4) + (byte & 15));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!masked || !(w[i] < 0.0f)) {
            o[i][j].x = fmaf(w[i], v.x, o[i][j].x);
            o[i][j].y = fmaf(w[i], v.y, o[i][j].y);
            o[i][j].z = fmaf(w[i], v.z, o[i][j].z);
            o[i][j].w = fmaf(w[i], v.w, o[i][j].w);
          }
      }
    }
    __syncwarp();
  }

  // (m, l, O) of every row to shared memory: O [WK][MT][DP], m and l [WK][MT].
  __device__ void dump(float* so, float* sm, float* sl) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = l[i];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) sm[warp * 4 + i] = m[i], sl[warp * 4 + i] = sum;
#pragma unroll
      for (int j = 0; j < NQ; ++j) {
        float4 v = o[i][j];
        if (KS == 2) {
          v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
          v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
          v.z += __shfl_xor_sync(0xffffffffu, v.z, 16);
          v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
        }
        const int d = KS == 1 ? (lane + 32 * j) * 4 : (lane & 15) * 4;
        if (KS == 1 || lane < 16) *reinterpret_cast<float4*>(so + (warp * 4 + i) * DP + d) = v;
      }
    }
  }
};

// ---------------------------------------------------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------------------------------------------------

// Sizes that follow from an engine's.  Dynamic shared memory holds the ring (reused for O at the end of a unit), the
// engine's own, the keys' offsets and validity, and the rows' m, l and weights at the end of a unit.
template <class E>
struct Lay {
  static constexpr int kPart = E::MT * (E::kDP + 2) + 4;  // floats of a part: O, m, l, status
  static constexpr int kFinish = E::WK * E::MT * E::kDP * 4;
  static constexpr int kRing = E::STAGES * E::STAGE > kFinish ? E::STAGES * E::STAGE : kFinish;
  static constexpr int kSmem = kRing + E::EXTRA + (E::STAGES + 1) * (E::KT * 8 + 16) + E::WK * E::MT * 3 * 4;
};

template <bool BF16>
__device__ __forceinline__ void store4(char* p, float4 v) {
  if (BF16) {
    uint2 u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(v.y), "f"(v.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(v.w), "f"(v.z));
    *reinterpret_cast<uint2*>(p) = u;
  } else {
    *reinterpret_cast<float4*>(p) = v;
  }
}

// One query row's quad of columns, normalised, and its lse.
template <class E>
__device__ __forceinline__ void write_row(const AttnParams& p, const AttnRequest& r, int hkv, int row, int d, float4 o,
                                          float m, float l) {
  if (row >= r.n * p.group) return;
  const int64_t grow = r.row0 + row / p.group;
  const int head = hkv * p.group + row % p.group;
  const bool none = m == -kInfF;  // nothing seen, or only scores of -inf
  const float inv = none ? 0.0f : 1.0f / l;
  if (d < p.c.head_dim) {
    o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    store4<E::kBf16>(p.out + (grow * p.o_row + head * p.o_head + d) * (E::kBf16 ? 2 : 4), o);
  }
  if (d == 0 && p.lse) p.lse[grow * p.heads + head] = none ? -kInfF : fmaf(m, kLn2, logf(l));
}

template <class E>
__global__ void __launch_bounds__(E::THREADS) k_attention(AttnParams p) {
  constexpr int T = E::THREADS, KT = E::KT, MT = E::MT, S = E::STAGES, DP = E::kDP, WK = E::WK;
  constexpr int RING = S + 1;
  constexpr int ES = E::kBf16 ? 2 : 4;
  constexpr int PIECES = DP * ES / 16;  // 16-byte pieces of a staged row
  constexpr int QUADS = DP / 4;
  extern __shared__ __align__(128) char smem[];
  char* ring = smem;
  char* extra = ring + Lay<E>::kRing;
  int64_t* s_off = reinterpret_cast<int64_t*>(extra + E::EXTRA);              // [RING][KT]
  uint32_t* s_valid = reinterpret_cast<uint32_t*>(s_off + RING * KT);         // [RING][4]
  float* s_m = reinterpret_cast<float*>(s_valid + RING * 4);                  // [WK][MT]
  float* s_l = s_m + WK * MT;
  float* s_w = s_l + WK * MT;
  __shared__ int64_t s_sum[T / 32];
  __shared__ int64_t s_find[2];
  __shared__ int s_last;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int block = blockIdx.x;

  grid_dependency_wait();
  allow_dependents();

  // The line of tiles: its length, and the request this block starts in.
  auto tiles_of = [&](const AttnRequest& r) -> int64_t {
    if (r.n == 0) return 0;
    const int64_t row_tiles = (static_cast<int64_t>(r.n) * p.group + MT - 1) / MT;
    return p.c.heads * row_tiles * ((r.len + r.n + KT - 1) / KT);
  };
  int64_t mine = 0;
  for (int b = t; b < p.batch; b += T) mine += tiles_of(attn_request(p, b));
  int64_t sum = mine;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_sum[warp] = sum;
  if (t == 0) s_find[0] = -1;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < T / 32; ++w) total += s_sum[w];
  __syncthreads();
  const int64_t g = total < gridDim.x ? (total > 0 ? total : 1) : gridDim.x;  // blocks that have work
  // Requests without rows have no tiles: their status is written here.
  for (int b = block * T + t; b < p.batch; b += gridDim.x * T) {
    const AttnRequest r = attn_request(p, b);
    if (r.n == 0) p.status[b] = r.status;
  }
  if (block >= g || total == 0) return;
  const int64_t start = block * total / g, end = (block + 1) * total / g;
  int64_t before = 0;  // tiles of the requests before the chunk
  for (int b0 = 0; b0 < p.batch; b0 += T) {
    const int b = b0 + t;
    int64_t own = b < p.batch ? tiles_of(attn_request(p, b)) : 0;
    int64_t inc = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    int64_t base = before, chunk = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) base += s_sum[w];
      chunk += s_sum[w];
    }
    if (own > 0 && base + inc - own <= start && start < base + inc) {
      s_find[0] = b;
      s_find[1] = base + inc - own;
    }
    __syncthreads();
    before += chunk;
    if (s_find[0] >= 0) break;
  }
  int b = static_cast<int>(s_find[0]);
  int64_t first = s_find[1];  // first tile of request b

  for (int64_t pos = start; pos < end;) {
    AttnRequest r = attn_request(p, b);
    const int64_t have = tiles_of(r);
    if (pos >= first + have) {  // next request
      first += have;
      ++b;
      continue;
    }
    const int nt = (r.len + r.n + KT - 1) / KT;
    const int row_tiles = (r.n * p.group + MT - 1) / MT;
    const int unit = static_cast<int>((pos - first) / nt);
    const int t0 = static_cast<int>((pos - first) - static_cast<int64_t>(unit) * nt);
    const int rt = unit % row_tiles, hkv = unit / row_tiles;
    const int cnt = static_cast<int>(min(static_cast<int64_t>(nt - t0), end - pos));
    const int keys = r.len + r.n;
    uint32_t bad = 0u;  // this thread placed a key outside the cache

    E eng;
    // Offsets of a tile's keys: fetched as raw words two tiles before they are needed.
    int64_t word = -1;
    auto fetch = [&](int tile) {
      if (t < KT) word = tile < t0 + cnt ? key_word(p, r, b, tile * KT + t) : -1;
    };
    auto place = [&](int tile) {
      if (t < KT) {
        const int x = tile * KT + t;
        const int64_t off = tile < t0 + cnt ? key_offset(p, r, x, word) : -1;
        const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
        if (tile < t0 + cnt && x < keys && off < 0) bad |= kStSlotRange;
        s_off[(tile % RING) * KT + t] = off;
        if (lane == 0) s_valid[(tile % RING) * 4 + warp] = ok;
      }
    };
    auto load = [&](int tile) {
      if (tile < t0 + cnt) {
        const uint32_t dst = smem_addr(ring + (tile % S) * E::STAGE);
        for (int x = t; x < KT * PIECES; x += T) {
          const int key = x / PIECES, c = x % PIECES;
          const int64_t off = s_off[(tile % RING) * KT + key];
          const bool ok = off >= 0 && c * 16 < p.c.head_dim * ES;
          const int64_t byte = ok ? (off + hkv * p.c.head_stride) * ES + c * 16 : 0;
          cp_async16(dst + E::piece(key, c), p.c.k + byte, ok);
          cp_async16(dst + KT * E::ROW + E::piece(key, c), p.c.v + byte, ok);
        }
      }
      cp_async_commit();
    };
    for (int i = 0; i < S; ++i) {
      fetch(t0 + i);
      place(t0 + i);
    }
    fetch(t0 + S);
    __syncthreads();
    for (int i = 0; i < S - 1; ++i) load(t0 + i);
    eng.init(p, r, hkv, rt, extra);
    for (int tile = t0; tile < t0 + cnt; ++tile) {
      cp_async_wait<S - 2>();
      __syncthreads();
      load(tile + S - 1);
      place(tile + S);
      fetch(tile + S + 1);
      eng.tile(p, r, b, rt, tile * KT, ring + (tile % S) * E::STAGE, s_valid + (tile % RING) * 4);
    }
    cp_async_wait<0>();
    bad = (__syncthreads_or(static_cast<int>(bad)) ? kStSlotRange : 0u) | r.status;

    // Finish: the key groups' parts, joined in group order.
    float* s_o = reinterpret_cast<float*>(ring);
    eng.dump(s_o, s_m, s_l);
    __syncthreads();
    if (t < MT) {
      float M = -kInfF;
#pragma unroll
      for (int k = 0; k < WK; ++k) M = fmax_nan(M, s_m[k * MT + t]);
      float L = 0.0f;
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float w = M == -kInfF ? 0.0f : ex2_fast(s_m[k * MT + t] - M);
        s_w[k * MT + t] = w;
        L = fmaf(w, s_l[k * MT + t], L);
      }
      s_m[t] = M;
      s_l[t] = L;
    }
    __syncthreads();
    auto joined = [&](int row, int d) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float w = s_w[k * MT + row];
        const float4 v = *reinterpret_cast<const float4*>(s_o + (k * MT + row) * DP + d);
        a.x = fmaf(w, v.x, a.x), a.y = fmaf(w, v.y, a.y), a.z = fmaf(w, v.z, a.z), a.w = fmaf(w, v.w, a.w);
      }
      return a;
    };
    const bool whole = cnt == nt;
    const bool reports = hkv == 0 && rt == row_tiles - 1;  // this unit's keys are all of the request's
    if (whole) {
      for (int x = t; x < MT * QUADS; x += T) {
        const int row = x / QUADS, d = (x % QUADS) * 4;
        write_row<E>(p, r, hkv, rt * MT + row, d, joined(row, d), s_m[row], s_l[row]);
      }
      if (reports && t == 0) p.status[b] = bad;
    } else {
      // A part: slot 0 for the block's first tiles, 1 for a unit that begins inside the block.
      float* part = p.parts + (static_cast<int64_t>(block) * 2 + (pos == start ? 0 : 1)) * Lay<E>::kPart;
      for (int x = t; x < MT * QUADS; x += T) {
        const int row = x / QUADS, d = (x % QUADS) * 4;
        *reinterpret_cast<float4*>(part + row * DP + d) = joined(row, d);
      }
      if (t < MT) part[MT * DP + t] = s_m[t], part[MT * DP + MT + t] = s_l[t];
      if (t == 0) part[MT * (DP + 2)] = __uint_as_float(bad);
      __syncthreads();
      // The unit's blocks: those that own its first and its last tile.
      const int64_t u0 = first + static_cast<int64_t>(unit) * nt, u1 = u0 + nt - 1;
      const int c0 = static_cast<int>(((u0 + 1) * g - 1) / total), c1 = static_cast<int>(((u1 + 1) * g - 1) / total);
      if (t == 0) {
        const bool last = ticket_add(&p.tickets[c0], 1u) == static_cast<unsigned>(c1 - c0);
        if (last) p.tickets[c0] = 0u;
        s_last = last ? 1 : 0;
      }
      __syncthreads();
      if (s_last) {
        const int64_t begin0 = c0 * total / g;
        auto part_of = [&](int c) {
          return p.parts + (static_cast<int64_t>(c) * 2 + (c == c0 && begin0 != u0 ? 1 : 0)) * Lay<E>::kPart;
        };
        uint32_t any = 0u;
        if (t < MT) {
          float M = -kInfF, L = 0.0f;
          for (int c = c0; c <= c1; ++c) M = fmax_nan(M, __ldcg(part_of(c) + MT * DP + t));
          if (M > -kInfF || M != M)
            for (int c = c0; c <= c1; ++c)
              L = fmaf(ex2_fast(__ldcg(part_of(c) + MT * DP + t) - M), __ldcg(part_of(c) + MT * DP + MT + t), L);
          s_m[t] = M;
          s_l[t] = L;
        }
        if (t == 0)
          for (int c = c0; c <= c1; ++c) any |= __float_as_uint(__ldcg(part_of(c) + MT * (DP + 2)));
        __syncthreads();
        for (int x = t; x < MT * QUADS; x += T) {
          const int row = x / QUADS, d = (x % QUADS) * 4;
          const float M = s_m[row];
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          if (M != -kInfF) {
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
              const float* q = part_of(c);
              const float w = ex2_fast(__ldcg(q + MT * DP + row) - M);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(q + row * DP + d));
              a.x = fmaf(w, v.x, a.x), a.y = fmaf(w, v.y, a.y), a.z = fmaf(w, v.z, a.z), a.w = fmaf(w, v.w, a.w);
            }
          }
          write_row<E>(p, r, hkv, rt * MT + row, d, a, M, s_l[row]);
        }
        if (reports && t == 0) p.status[b] = any;
      }
    }
    __syncthreads();  // the ring and the offsets are free again
    pos += cnt;
  }
}

// The shared memory opt-in and the resident blocks of an SM, once for each device.
template <class E>
cudaError_t blocks_per_sm(int* n) {
  static std::mutex mu;
  static int have[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (have[dev] == 0) {
    e = cudaFuncSetAttribute(k_attention<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<E>::kSmem);
    if (e != cudaSuccess) return e;
    int fit = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, k_attention<E>, E::THREADS, Lay<E>::kSmem);
    if (e != cudaSuccess) return e;
    have[dev] = fit < 1 ? 1 : fit;
  }
  *n = have[dev];
  return cudaSuccess;
}

template <class E>
cudaError_t launch(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  int per_sm = 1;
  const cudaError_t e = blocks_per_sm<E>(&per_sm);
  if (e != cudaSuccess) return e;
  int grid = dev.sms * per_sm;
  if (grid > kAttnMaxBlocks) grid = kAttnMaxBlocks;
  return launch_pdl(k_attention<E>, dim3(static_cast<unsigned>(grid)), dim3(E::THREADS), Lay<E>::kSmem, stream, p);
}

template <bool BF16>
cudaError_t launch_dim(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  if (p.c.head_dim <= 64) return launch<SimtEngine<BF16, 64>>(p, dev, stream);
  if (p.c.head_dim <= 128) return launch<SimtEngine<BF16, 128>>(p, dev, stream);
  return launch<SimtEngine<BF16, 256>>(p, dev, stream);
}

// Floats of one part: the largest row tile any engine has for this head size.
size_t part_bytes(int32_t head_dim) {
  const size_t dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  return (64 * (dp + 2) + 4) * sizeof(float);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_verify_attention_workspace_bytes(int32_t /*batch*/, int32_t /*max_len*/, int32_t /*num_heads*/,
                                             int32_t /*kv_heads*/, int32_t head_dim) {
  return align_up(kAttnCounterBytes + 2 * static_cast<size_t>(kAttnMaxBlocks) * part_bytes(head_dim), 256);
}

sv_status_t spec_verify_paged_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t num_heads,
                                        const sv_kv_cache_t* cache, int32_t layer, int32_t batch, int64_t total_rows,
                                        int32_t max_len, const int32_t* cu_seqlens, const int64_t* seq_lens,
                                        const int64_t* row_slots, const uint8_t* mask, float scale, void* out,
                                        int64_t out_row_stride, int64_t out_head_stride, float* lse,
                                        uint32_t* dev_status, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (batch < 0 || batch > 65535 || max_len < 1 || total_rows < 0 || total_rows > INT32_MAX) return SV_ERR_BAD_SHAPE;
  KvView c{};
  const sv_status_t s = check_cache(cache, &c);
  if (s != SV_OK) return s;
  if (layer < 0 || layer >= c.layers || num_heads < 1 || num_heads % c.heads != 0 || !std::isfinite(scale))
    return SV_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(max_len) * num_heads > (1 << 24)) return SV_ERR_BAD_SHAPE;
  if (!cu_seqlens && total_rows < static_cast<int64_t>(batch) * max_len) return SV_ERR_BAD_SHAPE;
  if (q_row_stride < 0 || q_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0) return SV_ERR_BAD_SHAPE;
  if (batch == 0) return SV_OK;
  if (!q || !out || !seq_lens || !dev_status) return SV_ERR_NULL_ARG;
  if (!aligned16(q) || !aligned16(out) || (q_row_stride * c.es) % 16 != 0 || (q_head_stride * c.es) % 16 != 0 ||
      (out_row_stride * c.es) % 16 != 0 || (out_head_stride * c.es) % 16 != 0)
    return SV_ERR_MISALIGNED;
  if (!ws || ws_bytes < spec_verify_attention_workspace_bytes(batch, max_len, num_heads, c.heads, c.head_dim) ||
      (reinterpret_cast<uintptr_t>(ws) & 255) != 0)
    return SV_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  c.k += layer * c.layer_stride * c.es;
  c.v += layer * c.layer_stride * c.es;
  char* base = static_cast<char*>(ws);
  const AttnParams p{static_cast<const char*>(q),
                     q_row_stride, q_head_stride, static_cast<char*>(out), out_row_stride, out_head_stride, lse, c,
                     cu_seqlens, seq_lens, row_slots, mask, dev_status, batch, max_len, num_heads,
                     num_heads / c.heads, total_rows, scale * 1.44269504088896340736f,
                     reinterpret_cast<uint32_t*>(base), reinterpret_cast<float*>(base + kAttnCounterBytes)};
  e = c.es == 2 ? launch_dim<true>(p, dev, stream) : launch_dim<false>(p, dev, stream);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

}  // extern "C"
