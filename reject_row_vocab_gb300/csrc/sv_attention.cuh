// What the attention kernels share: the call's parameters, a request's
// layout, the division of the work over blocks, and the join of its parts.
//
// A unit is one request, one cache head and one tile of MT query rows (a
// request's new rows times the query heads that share the cache head).  Its
// keys are the request's committed positions followed by its new rows, cut
// into tiles of KT keys.  All units' tiles form one line, each unit's preceded
// by U places that stand for what a unit costs beside its tiles; block c of g
// has places [c T / g, (c + 1) T / g) of it.  The line goes through the cache
// heads one by one, and through the requests within a head: so blocks side by
// side in time read the heads of the same positions, which lie side by side in
// memory (one token of 128 requests, 8 heads of 96: 275 us when both were
// measured, with a request's heads one after the other 352; of 128: 317 and 327;
// blocks of 16 rows of 64 requests: 101 and 104).  So every block gets the same work whatever the
// requests' lengths are, a long history is split over many blocks and a short
// one is not split at all.  A unit that lies in one block is finished there;
// otherwise each block leaves its part (m, l, O), and the parts are joined in
// block order, by the unit's last block to arrive or by a second kernel.
#pragma once

#include <cstdint>

#include "sv_kv.cuh"

namespace sv {

constexpr int kAttnMaxBlocks = 512;     // upper bound on the grid (the workspace is laid out for it)
constexpr int kAttnCounterBytes = sizeof(uint32_t) * kAttnMaxBlocks + 256;  // tickets, then the error word

struct AttnParams {
  const char* q;
  int64_t q_row, q_head;  // strides in elements
  char* out;
  int64_t o_row, o_head;
  float* lse;
  KvView c;  // k and v at the call's layer
  const int32_t* cu;
  const int64_t* seq_lens;
  const int64_t* row_slots;
  const uint8_t* mask;
  uint32_t* status;
  int32_t batch, max_len, heads, group;
  int64_t total_rows;
  float scale_log2;  // scale * log2(e)
  uint32_t* tickets;  // [kAttnMaxBlocks], zero between calls
  uint32_t* err;      // a wait gave up: reported by every call until the workspace is zero-filled
  float* parts;       // [grid, 2, part_floats]
};

__device__ __forceinline__ uint32_t attn_timeout(const AttnParams& p) { return __ldcg(p.err) ? kStTimeout : 0u; }

struct AttnRequest {
  int64_t row0;
  int32_t n;      // new rows; 0 when the row range is invalid
  int32_t len;    // committed positions
  uint32_t status;
};

__device__ __forceinline__ AttnRequest attn_request(const AttnParams& p, int b) {
  AttnRequest r{static_cast<int64_t>(b) * p.max_len, p.max_len, 0, 0u};
  if (p.cu) {
    const int64_t lo = p.cu[b], hi = p.cu[b + 1];
    r.row0 = lo;
    r.n = static_cast<int32_t>(hi - lo);
    if (lo < 0 || hi <= lo || hi - lo > p.max_len || hi > p.total_rows) {
      r.n = 0;
      r.status = kStBadLayout;
      return r;
    }
  }
  const int64_t len = p.seq_lens[b], most = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
  if (len < 0) {
    r.status = kStBadLayout;
  } else if (len > most) {
    r.status = kStSlotRange;
    r.len = static_cast<int32_t>(most);
  } else {
    r.len = static_cast<int32_t>(len);
  }
  return r;
}

// The raw word that places key x of a request (a page id or a slot), and what becomes of it.  Fetched a tile ahead
// of its use, so that the dependent loads of the K/V rows do not wait for it.
__device__ __forceinline__ int64_t key_word(const AttnParams& p, const AttnRequest& r, int b, int x) {
  if (x < 0 || x >= r.len + r.n) return -1;
  if (x >= r.len && p.row_slots) return p.row_slots[r.row0 + (x - r.len)];
  const uint32_t page = divide(static_cast<uint32_t>(x), p.c.div_mul, p.c.div_shift);
  if (page >= static_cast<uint32_t>(p.c.max_pages)) return -1;
  return p.c.table[b * p.c.ld_table + page];
}
__device__ __forceinline__ int64_t key_offset(const AttnParams& p, const AttnRequest& r, int x, int64_t word) {
  if (x < 0 || x >= r.len + r.n) return -1;
  if (x >= r.len && p.row_slots) return kv_slot_offset(p.c, word);
  if (word < 0 || word > INT32_MAX) return -1;
  const uint32_t page = divide(static_cast<uint32_t>(x), p.c.div_mul, p.c.div_shift);
  return kv_page_offset(p.c, static_cast<int32_t>(word), static_cast<uint32_t>(x) - page * p.c.page_size);
}

// 16-byte asynchronous copy global -> shared; zero-fills when !valid (the source is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Matrix instructions' fragments: four 8 x 8 blocks of 16-bit values, and the product of 16 x 16 by 16 x 8 on top of c.
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether new row i sees new row j of the same request.
__device__ __forceinline__ bool row_sees(const AttnParams& p, int b, int i, int j) {
  if (!p.mask) return j <= i;
  return p.mask[(static_cast<int64_t>(b) * p.max_len + i) * p.max_len + j] != 0;
}

constexpr float kLn2 = 0.693147180559945309417f;

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

// Which of keys x0 .. x0 + 31 new row i of a request sees, among those of `valid`.
__device__ __forceinline__ uint32_t row_sees_of(const AttnParams& p, const AttnRequest& r, int b, int i, int x0,
                                                uint32_t valid) {
  if (i >= r.n) return 0u;
  const int hist = r.len - x0;  // keys of the history among them
  if (hist >= 32) return valid;
  uint32_t see = hist <= 0 ? 0u : (1u << hist) - 1u;
  if (!p.mask) {
    const int upto = hist + i + 1;
    see = upto <= 0 ? 0u : upto >= 32 ? 0xffffffffu : (1u << upto) - 1u;
  } else {
    const uint8_t* m = p.mask + (static_cast<int64_t>(b) * p.max_len + i) * p.max_len - hist;
#pragma unroll 4
    for (int k = max(hist, 0); k < min(32, hist + r.n); ++k)
      if (m[k]) see |= 1u << k;
  }
  return see & valid;
}

// A query row's quad of columns, normalised, and (with the first quad) its lse.
template <bool BF16>
__device__ __forceinline__ void write_row(const AttnParams& p, int64_t row, int head, int d, float4 o, float m, float l) {
  const bool none = m == -kInfF;  // nothing seen, or only scores of -inf
  const float inv = none ? 0.0f : 1.0f / l;
  if (d < p.c.head_dim) {
    o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    store4<BF16>(p.out + (row * p.o_row + head * p.o_head + d) * (BF16 ? 2 : 4), o);
  }
  if (d == 0 && p.lse) p.lse[row * p.heads + head] = none ? -kInfF : fmaf(m, kLn2, logf(l));
}

// ---------------------------------------------------------------------------------------------------------------------
// The line of tiles
// ---------------------------------------------------------------------------------------------------------------------

// Places of a request within a cache head: its units there times (U + key tiles).
template <int MT, int KT, int U>
__device__ __forceinline__ int64_t attn_places(const AttnParams& p, const AttnRequest& r) {
  if (r.n == 0) return 0;
  const int64_t row_tiles = (static_cast<int64_t>(r.n) * p.group + MT - 1) / MT;
  return row_tiles * ((r.len + r.n + KT - 1) / KT + U);
}

// A block's stretch of the line, and the request it starts in.
struct AttnSpan {
  int64_t total, g;     // all places; blocks that have work
  int64_t start, end;   // this block's places (start == end: none)
  int32_t b, head;      // request and cache head of the first one
  int64_t first;        // that request's first place
};

// a b / c for b c < 2^63, by 32-bit division where the numbers are small.
__device__ __forceinline__ int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  const int64_t n = a * b;
  if (n <= UINT32_MAX && c <= UINT32_MAX) return static_cast<uint32_t>(n) / static_cast<uint32_t>(c);
  return n / c;
}

// Computed by every block for itself, by T threads of which this is thread t; sync() is a barrier among them.  One
// scan over the first T requests gives the total and finds the start; only larger batches are gone through again.
// s_sum [2 T / 32] (32 at most) and s_find [2] are shared.
template <int MT, int KT, int U, int T, class Sync>
__device__ __forceinline__ AttnSpan attn_span(const AttnParams& p, int t, int64_t* s_sum, int64_t* s_find, Sync sync) {
  constexpr int W = T / 32;
  static_assert(W <= 16, "s_sum");
  const int lane = t & 31, warp = t >> 5;
  AttnSpan sp{};
  int64_t own = 0, rest = 0;
  for (int b = t; b < p.batch; b += T) {
    const AttnRequest r = attn_request(p, b);
    const int64_t places = attn_places<MT, KT, U>(p, r);
    if (b == t)
      own = places;
    else
      rest += places;
    // a request without rows has no places: its status is written here
    if (r.n == 0 && b % gridDim.x == blockIdx.x) p.status[b] = r.status;
  }
  auto scan = [&](int64_t x) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += o;
    }
    return x;
  };
  int64_t inc = scan(own);
  if (p.batch > T) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, off);
  }
  if (lane == 31) s_sum[warp] = inc, s_sum[W + warp] = rest;
  if (t == 0) s_find[0] = -1;
  sync();
  int64_t base = 0, chunk = 0;  // places before this warp, and of this chunk of requests
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) base += s_sum[w];
    chunk += s_sum[w];
    sp.total += s_sum[w] + s_sum[W + w];
  }
  const int64_t per_head = sp.total;
  sp.total *= p.c.heads;
  const int64_t blocks = gridDim.x;
  sp.g = sp.total < blocks ? (sp.total > 0 ? sp.total : 1) : blocks;
  if (blockIdx.x >= sp.g || sp.total == 0) return sp;
  sp.start = mul_div(blockIdx.x, sp.total, sp.g);
  sp.end = mul_div(blockIdx.x + 1, sp.total, sp.g);
  sp.head = static_cast<int32_t>(mul_div(sp.start, 1, per_head));
  const int64_t start = sp.start - sp.head * per_head;  // within the head
  int64_t before = 0;
  for (int b0 = 0;;) {
    const int64_t at = before + base + inc - own;
    if (own > 0 && at <= start && start < at + own) {
      s_find[0] = b0 + t;
      s_find[1] = at;
    }
    sync();
    before += chunk;
    b0 += T;
    if (s_find[0] >= 0 || b0 >= p.batch) break;
    own = b0 + t < p.batch ? attn_places<MT, KT, U>(p, attn_request(p, b0 + t)) : 0;
    inc = scan(own);
    if (lane == 31) s_sum[warp] = inc;
    sync();
    base = chunk = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) base += s_sum[w];
      chunk += s_sum[w];
    }
  }
  sp.b = static_cast<int32_t>(s_find[0]);
  sp.first = sp.head * per_head + s_find[1];
  return sp;
}

// The block's next segment: consecutive key tiles of one unit.
struct AttnSegment {
  AttnRequest r;
  int32_t b, hkv, rt;
  int32_t t0, cnt, nt;  // its key tiles [t0, t0 + cnt) of nt
  int64_t u0;           // the place of the unit's first tile
  bool reports;         // its unit sees all of the request's keys: it carries the request's status
};

template <int MT, int KT, int U>
struct AttnWalk {
  const AttnParams& p;
  AttnSpan sp;
  int64_t pos;

  __device__ AttnWalk(const AttnParams& params, const AttnSpan& s) : p(params), sp(s), pos(s.start) {}

  __device__ bool next(AttnSegment& s) {
    while (pos < sp.end) {
      s.r = attn_request(p, sp.b);
      const int64_t have = attn_places<MT, KT, U>(p, s.r);
      if (pos >= sp.first + have) {
        sp.first += have;
        if (++sp.b == p.batch) sp.b = 0, ++sp.head;
        continue;
      }
      s.b = sp.b;
      s.nt = (s.r.len + s.r.n + KT - 1) / KT;
      const int row_tiles = (s.r.n * p.group + MT - 1) / MT;
      const int64_t in = pos - sp.first;
      const int unit = in <= INT32_MAX ? static_cast<int>(static_cast<uint32_t>(in) / static_cast<uint32_t>(s.nt + U))
                                       : static_cast<int>(in / (s.nt + U));
      s.u0 = sp.first + static_cast<int64_t>(unit) * (s.nt + U) + U;
      s.t0 = static_cast<int>(max(pos - s.u0, static_cast<int64_t>(0)));
      s.cnt = static_cast<int>(min(static_cast<int64_t>(s.nt), sp.end - s.u0)) - s.t0;
      pos = s.u0 + s.nt;
      if (s.cnt <= 0) continue;  // the block's places end before the unit's first tile
      s.rt = unit;
      s.hkv = sp.head;
      s.reports = s.hkv == 0 && s.rt == row_tiles - 1;
      return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------------------------------------------------------------
// NaN and infinities in V.  A weight of 0 does not silence them, and only new rows can be seen by some rows of a tile and
// not by others: there they are taken out of the products, and added at the end to the rows that see them.
// ---------------------------------------------------------------------------------------------------------------------

// Whether a row of the request may not see one of its new rows.  (A single row sees itself, unless a mask says otherwise.)
__device__ __forceinline__ bool new_rows_differ(const AttnParams& p, const AttnRequest& r) { return r.n > 1 || p.mask; }

__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {  // two bf16
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
}

// Takes the values that are not finite out of 16 bytes of V; whether there were any.
template <bool BF16>
__device__ __forceinline__ bool make_finite(uint4* at) {
  const uint4 u = *at;
  uint4 f;
  if (BF16)
    f = make_uint4(finite_pair(u.x), finite_pair(u.y), finite_pair(u.z), finite_pair(u.w));
  else
    f = make_uint4((u.x & 0x7f800000u) == 0x7f800000u ? 0u : u.x, (u.y & 0x7f800000u) == 0x7f800000u ? 0u : u.y,
                   (u.z & 0x7f800000u) == 0x7f800000u ? 0u : u.z, (u.w & 0x7f800000u) == 0x7f800000u ? 0u : u.w);
  if (f.x == u.x && f.y == u.y && f.z == u.z && f.w == u.w) return false;
  *at = f;
  return true;
}

// The sum of the NaN and infinite values that new row i sees of columns d .. d + 3 of the segment's new rows' V.
template <bool BF16, int KT>
__device__ __noinline__ float4 nonfinite_seen(const AttnParams& p, const AttnSegment& s, int i, int d) {
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < s.r.n; ++j) {
    const int x = s.r.len + j;
    if (x < s.t0 * KT || x >= (s.t0 + s.cnt) * KT || !row_sees(p, s.b, i, j)) continue;
    const int64_t off = key_offset(p, s.r, x, key_word(p, s.r, s.b, x));
    if (off < 0) continue;
    const int64_t at = off + s.hkv * p.c.head_stride + d;
    for (int k = 0; k < 4 && d + k < p.c.head_dim; ++k) {
      const float v = BF16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.c.v)[at + k]) << 16)
                           : reinterpret_cast<const float*>(p.c.v)[at + k];
      if (!(fabsf(v) < kInfF)) f[k] += v;
    }
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}

// ---------------------------------------------------------------------------------------------------------------------
// Parts of a unit that several blocks share
// ---------------------------------------------------------------------------------------------------------------------

// Floats of a part: O as [DP / 4][MT] quads of columns, m [MT], l [MT], status, and an AttnSplit (see there).
template <int MT, int DP>
struct AttnPart {
  static constexpr int kM = MT * DP, kL = kM + MT, kStatus = kL + MT, kSplit = kStatus + 4, kFloats = kSplit + 12;
};

// What the join kernel needs of a unit that begins in a block and goes on behind it.
struct AttnSplit {
  int64_t row0;
  int32_t n, b, hkv, rt;
  int32_t last;     // the unit's last block; 0: the block left no such unit
  int32_t reports;
  int32_t pad[4];
};
static_assert(sizeof(AttnSplit) == 48, "AttnSplit layout");

// A block leaves at most two parts: of a unit that began before it, and of one that goes on behind it.
template <int MT, int DP>
__device__ __forceinline__ float* attn_part(const AttnParams& p, int block, bool begins) {
  return p.parts + (static_cast<int64_t>(block) * 2 + (begins ? 1 : 0)) * AttnPart<MT, DP>::kFloats;
}

// The block that owns a place.
__device__ __forceinline__ int attn_owner(const AttnSpan& sp, int64_t place) {
  const int64_t n = (place + 1) * sp.g - 1;
  if (n <= UINT32_MAX && sp.total <= UINT32_MAX) return static_cast<int>(static_cast<uint32_t>(n) / static_cast<uint32_t>(sp.total));
  return static_cast<int>(n / sp.total);
}

// Joins parts c0 .. c1 of a unit and writes its rows: E quads of columns a thread, PARTS parts in flight; a part's m, l
// and O are fetched together, and the running maximum moves as they come.
template <bool BF16, int MT, int DP, int T, int E, int PARTS>
__device__ __forceinline__ void attn_join_rows(const AttnParams& p, const AttnSegment& s, int c0, int c1, int live,
                                               int t) {
  using P = AttnPart<MT, DP>;
  const float* first = attn_part<MT, DP>(p, c0, true);
  const float* rest = attn_part<MT, DP>(p, 0, false);
  auto part_of = [&](int c) { return c == c0 ? first : rest + static_cast<int64_t>(c) * 2 * P::kFloats; };
  int wide = 1;  // threads side by side on the rows: a power of two
  while (wide < live) wide *= 2;
  const int row = t & (wide - 1), step = T / wide;
  const int grow = s.rt * MT + row, i = grow / p.group;
  const int head = s.hkv * p.group + grow - i * p.group;
  for (int q0 = t / wide; q0 < DP / 4 && row < live; q0 += step * E) {
    float4 a[E];
    float M = -kInfF, L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = c0; cb <= c1; cb += PARTS) {
      float m[PARTS], l[PARTS];
      float4 v[PARTS][E];
#pragma unroll
      for (int j = 0; j < PARTS; ++j) {
        m[j] = -kInfF, l[j] = 0.0f;
        if (cb + j <= c1) {
          const float* q = part_of(cb + j);
          m[j] = __ldcg(q + P::kM + row), l[j] = __ldcg(q + P::kL + row);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            v[j][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q0 + e * step < DP / 4)
              v[j][e] = __ldcg(reinterpret_cast<const float4*>(q) + (q0 + e * step) * MT + row);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < PARTS; ++j) {
        if (cb + j > c1) break;
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
    for (int e = 0; e < E; ++e) write_row<BF16>(p, s.r.row0 + i, head, (q0 + e * step) * 4, a[e], M, L);
  }
}

// At the end of a block of T threads: the units that it has left parts of.  Each has a ticket; the last of its blocks to come
// joins the parts, in block order, and writes the rows.  Two quads of columns a thread and eight parts at a time: a single
// request of 100000 leaves about 19 parts of a unit, and what their join waits for is the memory, part after part.
// segments [count], s_last: shared.
template <bool BF16, int MT, int DP, int T>
__device__ __forceinline__ void attn_join(const AttnParams& p, const AttnSpan& sp, const AttnSegment* segments, int count,
                                          int* s_last) {
  const int t = threadIdx.x;
#pragma unroll 1
  for (int x = 0; x < count; ++x) {
    const AttnSegment& s = segments[x];
    // the unit's blocks are those that own its first and its last tile
    const int c0 = attn_owner(sp, s.u0), c1 = attn_owner(sp, s.u0 + s.nt - 1);
    if (t == 0) {
      __threadfence();  // the block's parts, written before its last barrier
      const bool last = ticket_add(&p.tickets[c0], 1u) == static_cast<unsigned>(c1 - c0);
      if (last) p.tickets[c0] = 0u;
      *s_last = last ? 1 : 0;
    }
    __syncthreads();
    if (*s_last) {
      attn_join_rows<BF16, MT, DP, T, 2, 8>(p, s, c0, c1, min(MT, s.r.n * p.group - s.rt * MT), t);
      if (s.reports && t == 0) {
        uint32_t any = 0u;
        for (int c = c0; c <= c1; ++c)
          any |= __float_as_uint(__ldcg(attn_part<MT, DP>(p, c, c == c0) + AttnPart<MT, DP>::kStatus));
        p.status[s.b] = any | attn_timeout(p);
      }
    }
    __syncthreads();  // s_last is free again
  }
}

// bf16 with up to 16 rows a unit, bf16 with any number of rows on tensor memory, fp32.
cudaError_t launch_attention_few(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_attention_wide(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_attention_f32(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace sv
