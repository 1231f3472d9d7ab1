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

#include "sv_attention_ring.cuh"

namespace sv {
namespace {

// ---------------------------------------------------------------------------------------------------------------------
// Engine: plain fp32 arithmetic.  Four warps of four rows each; a lane scores one key of the tile, then gathers columns.
// ---------------------------------------------------------------------------------------------------------------------

__device__ __forceinline__ float4 load4(const char* p) { return *reinterpret_cast<const float4*>(p); }

template <int DP>
struct SimtEngine {
  static constexpr bool kBf16 = false;
  static constexpr int kDP = DP;
  static constexpr int MT = 16, KT = 32, WK = 1, THREADS = 128;
  static constexpr int ES = 4;
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
        f = load4(p.q + at * ES);
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
      const float4 k = load4(kp);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = *reinterpret_cast<const float4*>(q + (warp * 4 + i) * DP + c * 4);
        s[i] = fmaf(a.x, k.x, s[i]);
        s[i] = fmaf(a.y, k.y, s[i]);
        s[i] = fmaf(a.z, k.z, s[i]);
        s[i] = fmaf(a.w, k.w, s[i]);
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
        const float4 v = load4(vs + piece(key, byte >> 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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
  static constexpr int kFinish = E::WK * E::MT * E::kDP * 4;
  static constexpr int kRing = E::STAGES * E::STAGE > kFinish ? E::STAGES * E::STAGE : kFinish;
  static constexpr int kSmem = kRing + E::EXTRA + (E::STAGES + 1) * (E::KT * 8 + 16) + E::WK * E::MT * 3 * 4;
};

// What a unit costs beside its key tiles (loading Q, the join of the key groups, the first tiles' latency), in tiles.
constexpr int kUnitPlaces = 2;

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
  __shared__ int64_t s_sum[2 * T / 32];
  __shared__ int64_t s_find[2];
  __shared__ int s_last;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  auto sync = [] { __syncthreads(); };

  grid_dependency_wait();
  allow_dependents();
  const AttnSpan span = attn_span<MT, KT, kUnitPlaces, T>(p, t, s_sum, s_find, sync);
  AttnWalk<MT, KT, kUnitPlaces> walk(p, span);
  AttnSegment s;
  while (walk.next(s)) {
    const AttnRequest& r = s.r;
    const int end = s.t0 + s.cnt;
    const int keys = r.len + r.n;
    uint32_t bad = 0u;   // this thread placed a key outside the cache
    bool found = false;  // it took values that are not finite out of V

    E eng;
    // Offsets of a tile's keys: fetched as raw words two tiles before they are needed.
    int64_t word = -1;
    auto fetch = [&](int tile) {
      if (t < KT) word = tile < end ? key_word(p, r, s.b, tile * KT + t) : -1;
    };
    auto place = [&](int tile) {
      if (t < KT) {
        const int x = tile * KT + t;
        const int64_t off = tile < end ? key_offset(p, r, x, word) : -1;
        const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
        if (tile < end && x < keys && off < 0) bad |= kStSlotRange;
        s_off[(tile % RING) * KT + t] = off;
        if (lane == 0) s_valid[(tile % RING) * 4 + warp] = ok;
      }
    };
    auto load = [&](int tile) {
      if (tile < end) {
        const uint32_t dst = smem_addr(ring + (tile % S) * E::STAGE);
        for (int x = t; x < KT * PIECES; x += T) {
          const int key = x / PIECES, c = x % PIECES;
          const int64_t off = s_off[(tile % RING) * KT + key];
          const bool ok = off >= 0 && c * 16 < p.c.head_dim * ES;
          const int64_t byte = ok ? (off + s.hkv * p.c.head_stride) * ES + c * 16 : 0;
          cp_async16(dst + E::piece(key, c), p.c.k + byte, ok);
          cp_async16(dst + KT * E::ROW + E::piece(key, c), p.c.v + byte, ok);
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) {
      fetch(s.t0 + i);
      place(s.t0 + i);
    }
    fetch(s.t0 + S);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < S - 1; ++i) load(s.t0 + i);
    eng.init(p, r, s.hkv, s.rt, extra);
#pragma unroll 1
    for (int tile = s.t0; tile < end; ++tile) {
      cp_async_wait<S - 2>();
      __syncthreads();
      load(tile + S - 1);
      place(tile + S);
      fetch(tile + S + 1);
      if (r.n > 1 && (tile + 1) * KT > r.len) {
        char* v = ring + (tile % S) * E::STAGE + KT * E::ROW;
#pragma unroll 1
        for (int x = max(r.len - tile * KT, 0) * PIECES + t; x < KT * PIECES; x += T)
          if (make_finite<E::kBf16>(reinterpret_cast<uint4*>(v + E::piece(x / PIECES, x % PIECES)))) found = true;
        __syncthreads();
      }
      eng.tile(p, r, s.b, s.rt, tile * KT, ring + (tile % S) * E::STAGE, s_valid + (tile % RING) * 4);
    }
    cp_async_wait<0>();
    bad = (__syncthreads_or(static_cast<int>(bad)) ? kStSlotRange : 0u) | r.status;
    const bool careful = __syncthreads_or(found ? 1 : 0) != 0;

    // Finish: the key groups' parts, joined in group order.
    float* s_o = reinterpret_cast<float*>(ring);
    eng.dump(s_o, s_m, s_l);
    __syncthreads();
    for (int row = t; row < MT; row += T) {
      float M = -kInfF;
#pragma unroll
      for (int k = 0; k < WK; ++k) M = fmax_nan(M, s_m[k * MT + row]);
      float L = 0.0f;
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float w = M == -kInfF ? 0.0f : ex2_fast(s_m[k * MT + row] - M);
        s_w[k * MT + row] = w;
        L = fmaf(w, s_l[k * MT + row], L);
      }
      s_m[row] = M;
      s_l[row] = L;
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
      if (careful && s.rt * MT + row < r.n * p.group) {
        const AttnSegment copy = s;
        const float4 f = nonfinite_seen<E::kBf16, KT>(p, copy, (s.rt * MT + row) / p.group, d);
        a.x += f.x, a.y += f.y, a.z += f.z, a.w += f.w;
      }
      return a;
    };
    if (s.cnt == s.nt) {
#pragma unroll 1
      for (int x = t; x < MT * QUADS; x += T) {
        const int row = x / QUADS, d = (x % QUADS) * 4, grow = s.rt * MT + row;
        if (grow < r.n * p.group) {
          const int i = grow / p.group;
          write_row<E::kBf16>(p, r.row0 + i, s.hkv * p.group + grow - i * p.group, d, joined(row, d), s_m[row], s_l[row]);
        }
      }
      if (s.reports && t == 0) p.status[s.b] = bad;
    } else {
      using P = AttnPart<MT, DP>;
      float* part = attn_part<MT, DP>(p, blockIdx.x, s.t0 == 0);
#pragma unroll 1
      for (int x = t; x < MT * QUADS; x += T) {
        const int row = x % MT, quad = x / MT;
        *reinterpret_cast<float4*>(part + x * 4) = joined(row, quad * 4);
      }
      for (int row = t; row < MT; row += T) part[P::kM + row] = s_m[row], part[P::kL + row] = s_l[row];
      if (t == 0) part[P::kStatus] = __uint_as_float(bad);
      attn_join<E::kBf16, MT, DP, T>(p, span, s, t, &s_last);
    }
    __syncthreads();  // the ring and the offsets are free again
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

cudaError_t launch_attention(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int dim = p.c.head_dim;
  const int64_t rows = static_cast<int64_t>(p.max_len) * p.group;
  if (p.c.es == 2) return rows <= 16 ? launch_attention_few(p, dev, stream) : launch_attention_wide(p, dev, stream);
  return dim <= 64 ? launch<SimtEngine<64>>(p, dev, stream)
                   : dim <= 128 ? launch<SimtEngine<128>>(p, dev, stream) : launch<SimtEngine<256>>(p, dev, stream);
}

// Floats of one part: the largest row tile any engine has for this head size.
size_t part_bytes(int32_t head_dim) {
  const size_t dp = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
  return (64 * (dp + 2) + 16) * sizeof(float);
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

}  // namespace

// Boxes need pages of a multiple of eight rows (the swizzle's period); a layout the driver takes no map of has none.
KvMaps kv_maps(const KvView& c) {
  KvMaps m{};
  int rows = kKeys;
  while (rows >= 8 && c.page_size % rows != 0) rows /= 2;
  const EncodeTiledFn encode = encode_tiled();
  if (rows < 8 || !encode) return m;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.pages)};
  // an axis of one entry may come without a step
  auto step = [&](int64_t s) { return static_cast<cuuint64_t>(s > 0 ? s * c.es : (c.head_dim * c.es + 15) / 16 * 16); };
  const cuuint64_t strides[3] = {step(c.head_stride), step(c.slot_stride), step(c.page_stride)};
  const cuuint32_t box[4] = {128u / c.es, 1, static_cast<cuuint32_t>(rows), 1}, ones[4] = {1, 1, 1, 1};
  char* const base[2] = {c.k, c.v};
  CUtensorMap* const map[2] = {&m.k, &m.v};
  for (int i = 0; i < 2; ++i)
    if (encode(map[i], c.es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base[i], dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return m;
  m.rows = rows;
  return m;
}

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
                     reinterpret_cast<uint32_t*>(base), reinterpret_cast<uint32_t*>(base) + kAttnMaxBlocks,
                     reinterpret_cast<float*>(base + kAttnCounterBytes)};
  e = launch_attention(p, dev, stream);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

}  // extern "C"
