// New rows go into the paged cache with their keys rotated on the way, and
// their queries are rotated beside them ([E2D] §2.4: a draft tree's position
// ids come from the depth, its places from where the rows are staged).
//
//   a = position * inv_freq[i]
//   (x, y) -> magnitude (x cos a - y sin a, y cos a + x sin a)
//
// A warp takes one row (a part of its heads where there are few rows), a lane
// eight columns of a head: a pair's other half is in the lane itself or one
// shuffle away, and the row's sines and cosines are computed once, by the
// warp, and kept in registers for all heads.  The angle is reduced to a part of
// a turn in more than a float's bits: to 2^-25 of a radian up to position 2^22, to
// 2^-43 beyond.
//
// The 4-bit cache: 16 columns are two lanes, one shuffle gives their largest
// magnitude.  Which scale and which code is nearest hangs on which side of a
// border a value lies, and a rotation in fp32 gets that wrong for one value in a
// million.  So its keys are turned in pairs of floats: angles to 2^-43 of a radian at
// any position, sines and cosines to 2^-37, products and their sum to 2^-46.  The sum is
// rounded to odd, which keeps it on its side of every border that the exact one is
// further than 2^-37 (|x| + |y|) from.
//
// Bound by the rows' bytes: 8192 rows of 32 + 8 + 8 heads of 128 in bf16, 40 us
// (5.2 TB/s); over 4 bits by steps that wait for one another, twenty warps a
// multiprocessor not being enough to hide them (52 % of the issue slots are used, the
// ALU 37 %): 51.5 us, 45.4 with keys turned in fp32.  Five blocks of four warps and
// four passes in flight are the best of both (two passes: 47 and 57.6 us; four blocks:
// 45 and 57).  A row's heads go to as many warps as give every multiprocessor
// sixteen: one token takes 8 us of the GPU.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cmath>
#include <type_traits>
#include <cstdint>

#include "sv_rows.cuh"

namespace sv {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kMaxPairs = 128;
constexpr int kUnroll = 4;

enum Pairing { kNeighbours = 0, kHalves = 1, kHalvesOdd = 2 };  // halves: of a multiple of eight pairs, of any number

struct HeadRows {
  const char* p;
  int64_t row, head;  // strides in elements
};

struct AppendParams {
  RowsView r;
  const int64_t* positions;
  const float* inv_freq;
  int32_t pairs;
  float magnitude;
  HeadRows q, k, v;
  char* q_out;
  int64_t o_row, o_head;
  int32_t q_heads, kv_heads, dim;
  uint32_t* status;
  int32_t passes, chunks, per;  // a row's passes over its heads, dealt out to `chunks` warps
};

// Sums and products of floats as pairs of floats (Dekker, Knuth): the rounded result in x, what it lacks in y.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v)));
}
__device__ __forceinline__ float2 two_product(float a, float b) {
  const float p = __fmul_rn(a, b);
  return make_float2(p, __fmaf_rn(a, b, -p));
}

// Part of a turn, hi + lo, of position * f.  Positions below 2^22 in pairs of floats: f / 2 pi to 2^-49 of itself, the product
// exactly, whole turns taken off.  (The 64-bit unit does two lanes a clock: 8192 rows took 8 us of it.)
__device__ __forceinline__ float2 part_of_turn(float position, float f) {
  constexpr float kHi = 0.15915494f;                                                      // 1 / 2 pi
  constexpr float kLo = static_cast<float>(0.15915494309189533577 - static_cast<double>(kHi));  // and what it lacks
  const float h = f * kHi, l = fmaf(f, kLo, fmaf(f, kHi, -h));
  const float x = h * position, low = fmaf(l, position, fmaf(h, position, -x));
  const float part = x - rintf(x), t = part + low;
  return make_float2(t, low - (t - part));
}
// The same to 2^-47 of a radian: f / 2 pi to 2^-70 of itself in three floats, its products with the position exactly as far as that
// counts, and their sum in a pair.  (Above, what one float holds beside the first product is rounded to 2^-48 of all turns: 2^-31
// of a radian at 100 000, 2^-25 at 2^22.)
__device__ __forceinline__ float2 part_of_turn_in_pairs(float position, float f) {
  constexpr double kTurn = 0.15915494309189535, kTurnLack = -9.839338337591243e-18;  // 1 / 2 pi
  constexpr float kHi = static_cast<float>(kTurn);
  constexpr float kMid = static_cast<float>(kTurn - static_cast<double>(kHi));
  constexpr float kLo = static_cast<float>(kTurn - static_cast<double>(kHi) - static_cast<double>(kMid) + kTurnLack);
  const float h = __fmul_rn(f, kHi);
  const float2 m = two_product(f, kMid), l = two_sum(__fmaf_rn(f, kHi, -h), m.x);
  const float rest = __fadd_rn(l.y, __fmaf_rn(f, kLo, m.y));
  const float2 x = two_product(h, position), y = two_product(l.x, position), low = two_sum(x.y, y.x);
  const float2 t = two_sum(__fsub_rn(x.x, rintf(x.x)), low.x);
  return make_float2(t.x, __fadd_rn(t.y, __fadd_rn(low.y, __fmaf_rn(rest, position, y.y))));
}
// Of any position, in pairs of doubles: f / 2 pi to 2^-104 of itself, a position's upper and lower 32 bits by themselves (2^63
// has 2^60 whole turns).
__device__ __noinline__ float2 part_of_turn_far(int64_t position, float f) {
  constexpr double kHi = 0.15915494309189535;     // 1 / 2 pi
  constexpr double kLo = -9.839338337591243e-18;  // and what it lacks
  const double w = static_cast<double>(f), h = w * kHi, l = fma(w, kLo, fma(w, kHi, -h));
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double p = i ? static_cast<double>(static_cast<uint32_t>(position)) : static_cast<double>(position >> 32) * 4294967296.0;
    const double x = h * p, low = fma(l, p, fma(h, p, -x));
    t += (x - rint(x)) + (low - rint(low));
  }
  t = t - rint(t);
  const float hi = static_cast<float>(t);
  return make_float2(hi, static_cast<float>(t - hi));
}
// Cosine and sine.
__device__ __forceinline__ float2 turn_of(float2 t) {
  float s, c;
  sincospif(2.0f * t.x, &s, &c);
  const float lo = t.y * 6.28318531f;
  return make_float2(fmaf(-lo, s, c), fmaf(lo, c, s));
}

// Cosine and sine of k / 64 of a turn, in pairs of floats.
struct TurnTable {
  float4 v[64];
};
constexpr double taylor(double x, int first) {  // of the sine (1) or the cosine (0), |x| <= pi / 4
  double term = first ? x : 1.0, sum = term;
  for (int i = first + 1; i < 24; i += 2) term *= -x * x / (i * (i + 1.0)), sum += term;
  return sum;
}
constexpr TurnTable turn_table() {
  TurnTable t{};
  for (int k = 0; k < 64; ++k) {
    const int quarter = (k + 8) / 16, i = k - quarter * 16;  // the nearest quarter of a turn, and the rest
    const double x = i * (6.28318530717958647693 / 64.0), c0 = taylor(x, 0), s0 = taylor(x, 1);
    const int q = quarter % 4;
    const double c = q == 0 ? c0 : q == 1 ? -s0 : q == 2 ? -c0 : s0, s = q == 0 ? s0 : q == 1 ? c0 : q == 2 ? -s0 : -c0;
    const float ch = static_cast<float>(c), sh = static_cast<float>(s);
    t.v[k] = float4{ch, static_cast<float>(c - ch), sh, static_cast<float>(s - sh)};
  }
  return t;
}
__device__ const TurnTable kTurnTable = turn_table();

// Cosine (x, y) and sine (z, w) in pairs of floats: those of the nearest 64th of a turn, turned by the rest a, |a| < 0.05:
// sin a = a - a^3 / 6 + a^5 / 120 - .., cos a - 1 = - a^2 / 2 + a^4 / 24 - ..
__device__ __forceinline__ float4 turn_in_pairs(float2 t) {
  const float k = rintf(t.x * 64.0f), r = __fmaf_rn(k, -1.0f / 64.0f, t.x);
  const float4 at = kTurnTable.v[static_cast<int>(k) & 63];
  constexpr float kHi = 6.2831855f;  // 2 pi
  constexpr float kLo = static_cast<float>(6.28318530717958647693 - static_cast<double>(kHi));
  float2 a = two_product(r, kHi);
  a.y = __fmaf_rn(t.y, kHi, __fmaf_rn(r, kLo, a.y));
  const float2 z = two_product(a.x, a.x);
  const float sin_lo = __fmaf_rn(__fmul_rn(a.x, z.x), __fmaf_rn(z.x, __fmaf_rn(z.x, -1.0f / 5040.0f, 1.0f / 120.0f), -1.0f / 6.0f),
                                 __fmaf_rn(a.y, __fmul_rn(-0.5f, z.x), a.y));
  const float cos_hi = __fmul_rn(-0.5f, z.x);  // (cos a) - 1
  const float cos_lo = __fmaf_rn(__fmul_rn(z.x, z.x), __fmaf_rn(z.x, -1.0f / 720.0f, 1.0f / 24.0f),
                                 __fmaf_rn(-0.5f, z.y, __fmul_rn(-a.x, a.y)));
  // (own + own_lo) cos a + (other + other_lo) sin a
  auto add = [&](float own, float own_lo, float other, float other_lo) {
    const float2 u = two_product(other, a.x), w = two_product(own, cos_hi);
    const float2 x = two_sum(u.x, w.x), y = two_sum(own, x.x);
    float low = __fmaf_rn(other, sin_lo, __fmul_rn(own, cos_lo));
    low = __fmaf_rn(other_lo, a.x, __fmaf_rn(own_lo, cos_hi, low));
    low = __fadd_rn(__fadd_rn(own_lo, low), __fadd_rn(__fadd_rn(u.y, w.y), __fadd_rn(x.y, y.y)));
    const float hi = __fadd_rn(y.x, low);
    return make_float2(hi, __fsub_rn(low, __fsub_rn(hi, y.x)));
  };
  const float2 c = add(at.x, at.y, -at.z, -at.w), s = add(at.z, at.w, at.x, at.y);
  return make_float4(c.x, c.y, s.x, s.y);
}

// Eight values of a row as they lie, and as pairs of floats.
template <int ES>
struct Eight {
  uint32_t w[ES * 2];
};
struct Pairs {
  uint64_t v[4];
};

__device__ __forceinline__ uint64_t add_pair_rz(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// x c + y s with c and s in pairs of floats (c_lo, s_lo what they lack), rounded to odd: towards 0, and, where that lost
// something, to an odd last bit.  What has at most 23 bits lies on the same side of the result as of the exact sum.
__device__ __forceinline__ uint64_t turn_to_odd(uint64_t x, uint64_t c, uint64_t c_lo, uint64_t y, uint64_t s, uint64_t s_lo) {
  const uint64_t minus = pair(-1.0f, -1.0f);
  // The products, their sum, and what each lacks (Dekker, Knuth).  The sum is one of two floats: where they cancel, a product added
  // without rounding leaves bits below both, and what such a sum lacks is not found by the steps for two floats.
  const uint64_t p = mul_pair(x, c), p_lo = fma_pair(x, c, mul_pair(p, minus));
  const uint64_t q = mul_pair(y, s), q_lo = fma_pair(y, s, mul_pair(q, minus));
  const uint64_t sum = add_pair(p, q), v = sub_pair(sum, p);
  const uint64_t lost = add_pair(sub_pair(p, sub_pair(sum, v)), sub_pair(q, v));
  const uint64_t low = add_pair(lost, fma_pair(y, s_lo, fma_pair(x, c_lo, add_pair(p_lo, q_lo))));
  const uint64_t cut = add_pair_rz(sum, low), rest = sub_pair(low, sub_pair(cut, sum));
  float w[2], r[2], n[2];
  unpair(cut, w[0], w[1]), unpair(rest, r[0], r[1]), unpair(sum, n[0], n[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __uint_as_float(__float_as_uint(w[i]) | (r[i] != 0.0f ? 1u : 0u));
    if (!(fabsf(n[i]) < 1e30f)) w[i] = n[i];  // (not a number, or a product on the way to none)
  }
  return pair(w[0], w[1]);
}

template <int ES>
__device__ __forceinline__ Pairs pairs_of(const Eight<ES>& e) {
  Pairs p;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p.v[i] = ES == 4 ? pair(__uint_as_float(e.w[ES * i / 2]), __uint_as_float(e.w[ES * i / 2 + 1])) : pair(bf16_lo(e.w[i]), bf16_hi(e.w[i]));
  return p;
}

template <int ES>
__device__ __forceinline__ void load8(Eight<ES>& e, const char* p, bool first, bool second) {
  uint4 a = make_uint4(0u, 0u, 0u, 0u);
  if (first) a = *reinterpret_cast<const uint4*>(p);
  e.w[0] = a.x, e.w[1] = a.y, e.w[2] = a.z, e.w[3] = a.w;
  if (ES == 4) {
    a = make_uint4(0u, 0u, 0u, 0u);
    if (second) a = *reinterpret_cast<const uint4*>(p + 16);
    e.w[ES * 2 - 4] = a.x, e.w[ES * 2 - 3] = a.y, e.w[ES * 2 - 2] = a.z, e.w[ES * 2 - 1] = a.w;
  }
}

template <int ES>
__device__ __forceinline__ void store8(char* p, const Eight<ES>& e, bool second) {
  *reinterpret_cast<uint4*>(p) = make_uint4(e.w[0], e.w[1], e.w[2], e.w[3]);
  if (ES == 4 && second)
    *reinterpret_cast<uint4*>(p + 16) = make_uint4(e.w[ES * 2 - 4], e.w[ES * 2 - 3], e.w[ES * 2 - 2], e.w[ES * 2 - 1]);
}

template <int ES>
__device__ __forceinline__ Eight<ES> round8(const Pairs& x) {
  Eight<ES> e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpair(x.v[i], lo, hi);
    if (ES == 4)
      e.w[ES * i / 2] = __float_as_uint(lo), e.w[ES * i / 2 + 1] = __float_as_uint(hi);
    else
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(e.w[i]) : "f"(hi), "f"(lo));
  }
  return e;
}

// Eight values (of a head's lanes, a multiple of four, all of them) into the 4-bit cache: codes, scale; whether all are finite.
__device__ __forceinline__ bool quantize8(const Pairs& x, uint32_t* codes, uint32_t* byte) {
  float v[8], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(x.v[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmax_nan(top, fabsf(v[e]));
  const bool fine = top < kInfF;
  if (!fine) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] == v[e] ? v[e] : 0.0f;
  }
  if (!(top <= 61440.0f)) {
    top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(v[e], -61440.0f), 61440.0f), top = fmaxf(top, fabsf(v[e]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  *byte = scale_byte(top);
  const float scale = scale_value(*byte), inv = *byte ? __frcp_rn(scale) : 0.0f;
  // Quotients: v times the rounded 1 / scale, whose remainder is exact and corrects it (Markstein's division), so that a value half
  // way between two codes is seen to be there.  (0 for a scale of 0.)
  const uint64_t s2 = pair(-scale, -scale), i2 = pair(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t y = pair(v[2 * i], v[2 * i + 1]), a = mul_pair(y, i2);
    unpair(fma_pair(fma_pair(a, s2, y), i2, a), v[2 * i], v[2 * i + 1]);
  }
  *codes = pack_codes(v);
  return fine;
}

enum Part { kQuery, kKey, kValue };

template <int ES, class C, Pairing PAIRING>
__global__ void __launch_bounds__(32 * kAppendWarps, 5) k_kv_append(const AppendParams p, const C c) {
  constexpr bool kPacked = std::is_same<C, PackedView>::value;
  __shared__ float2 s_turn[kAppendWarps][kMaxPairs];
  // Of the 4-bit cache: what s_turn lacks, and then what a column's cosine and (signed) sine lack.
  __shared__ float2 s_lack[kPacked ? kAppendWarps : 1][kPacked ? kMaxPairs : 1];
  __shared__ float4 s_low[kPacked ? kAppendWarps : 1][2][kPacked ? 2 * kMaxPairs / 4 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = (p.dim + 7) / 8, heads = 32 / lanes;  // lanes of a head, heads of a pass
  const int of = lane / lanes, d0 = (lane - of * lanes) * 8;
  const bool wide = ES == 2 || d0 + 4 < p.dim;  // the lane's second 16 bytes exist
  const int n = p.pairs;
  const bool turned = d0 < 2 * n;                                         // some of the lane's columns are rotated
  const int partner = (d0 < n ? lane + n / 8 : turned ? lane - n / 8 : lane) & 31;  // lane of the pairs' other halves
  const int q_passes = (p.q_heads + heads - 1) / heads, kv_passes = (p.kv_heads + heads - 1) / heads;
  grid_dependency_wait();
  allow_dependents();
  const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  flag_requests(p.r, p.status, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, threads);
  const int64_t items = rows_count(p.r) * p.chunks;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp; item < items; item += threads / 32) {
    const int64_t row = p.chunks == 1 ? item : item / p.chunks;
    const int chunk = static_cast<int>(item - row * p.chunks);
    const int first = chunk * p.per, last = min(first + p.per, p.passes);
    const bool turns = n > 0 && first < q_passes + kv_passes;
    float freq[kMaxPairs / 32];  // (on their way while the row's place is looked up)
#pragma unroll
    for (int i = 0; i < kMaxPairs / 32; ++i) freq[i] = turns && i * 32 + lane < n ? p.inv_freq[i * 32 + lane] : 0.0f;
    int j;
    const int b = row_request(p.r, row, lane, &j);
    if (b < 0) continue;
    const int64_t len = p.r.seq_lens ? p.r.seq_lens[b] : 0;
    if (len < 0) continue;
    const Place place = p.r.row_slots ? slot_place(c, p.r.row_slots[row]) : position_place(c, b, len + j);
    if (place.page < 0 && chunk == 0 && lane == 0) atomicOr(p.status + b, kStSlotRange);
    Pairs co, si;
    if (turns) {
      const int64_t pos = p.positions ? p.positions[row] : len + j;
      const bool far = pos <= -(1 << 22) || pos >= 1 << 22;
#pragma unroll
      for (int i = 0; i < kMaxPairs / 32; ++i)
        if (i * 32 + lane < n) {
          const float2 t = far       ? part_of_turn_far(pos, freq[i])
                           : kPacked ? part_of_turn_in_pairs(static_cast<float>(pos), freq[i])
                                     : part_of_turn(static_cast<float>(pos), freq[i]);
          if constexpr (kPacked) {
            const float4 u = turn_in_pairs(t);
            s_turn[warp][i * 32 + lane] = make_float2(u.x, u.z), s_lack[warp][i * 32 + lane] = make_float2(u.y, u.w);
          } else {
            s_turn[warp][i * 32 + lane] = turn_of(t);
          }
        }
      __syncwarp();
      if (turned) {
        float low_c[8], low_s[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float c[2], s[2];
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int d = d0 + e + f;
            const bool high = PAIRING == kNeighbours ? f : d >= n;  // the pair's second column
            int i = PAIRING == kNeighbours ? d / 2 : high ? d - n : d;
            if (i >= n) i = 0;  // (a column that is left as it is)
            const float2 t = s_turn[warp][i];
            const float sign = high ? p.magnitude : -p.magnitude;
            c[f] = t.x * p.magnitude, s[f] = t.y * sign;
            if constexpr (kPacked) {
              const float2 l = s_lack[warp][i];
              low_c[e + f] = fmaf(l.x, p.magnitude, fmaf(t.x, p.magnitude, -c[f]));
              low_s[e + f] = fmaf(l.y, sign, fmaf(t.y, sign, -s[f]));
            }
          }
          co.v[e / 2] = pair(c[0], c[1]), si.v[e / 2] = pair(s[0], s[1]);
        }
        if (kPacked && of == 0) {
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            s_low[warp][0][(d0 + e) / 4] = make_float4(low_c[e], low_c[e + 1], low_c[e + 2], low_c[e + 3]);
            s_low[warp][1][(d0 + e) / 4] = make_float4(low_s[e], low_s[e + 1], low_s[e + 2], low_s[e + 3]);
          }
        }
      }
      __syncwarp();
    }
    bool odd = false;  // a value that is not finite went into the 4-bit cache
    // Passes [lo, hi) over the heads of one part, `steps` bytes of a source's pass and of its destination's apart.
    auto part = [&](auto which, int lo, int hi, const HeadRows& from, int total) {
      constexpr Part kPart = decltype(which)::value;
      constexpr bool kInto = kPart != kQuery;  // into the cache
      lo = max(lo, 0);
      if (lo >= hi || (kInto && place.page < 0)) return;
      const int head0 = lo * heads + of;
      const char* src = from.p + (row * from.row + head0 * from.head + d0) * ES;
      const int64_t src_step = heads * from.head * ES;
      char* dst;
      int64_t dst_step;
      int scale_at = 0;
      if constexpr (!kInto) {
        dst = p.q_out + (row * p.o_row + head0 * p.o_head + d0) * ES, dst_step = heads * p.o_head * ES;
      } else if constexpr (!kPacked) {
        dst = (kPart == kValue ? c.v : c.k) +
              (place.page * c.page_stride + place.in * c.slot_stride + head0 * c.head_stride + d0) * ES;
        dst_step = heads * c.head_stride * ES;
      } else {
        const int codes = (kPart == kValue ? packed_v_codes(c.page_size, c.head_dim) : 0) + place.in * (c.head_dim / 2) + d0 / 2;
        scale_at = (kPart == kValue ? packed_v_scales(c.page_size, c.head_dim) : packed_k_scales(c.page_size, c.head_dim)) +
                   place.in * (c.head_dim / 16) + d0 / 16 - codes;
        dst = c.data + place.page * c.page_stride + head0 * c.head_stride + codes, dst_step = heads * c.head_stride;
      }
      const int live = of < heads ? (total - of + heads - 1) / heads : 0;  // passes in which this lane has a head
      for (int pass0 = lo; pass0 < hi; pass0 += kUnroll) {
        Eight<ES> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const bool have = pass0 + u < min(hi, live);
          load8<ES>(raw[u], src + u * src_step, have, have && wide);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (pass0 + u >= hi) break;
          const bool have = pass0 + u < live;
          Eight<ES> out = raw[u];
          Pairs x;
          if (kPart != kValue || (kPacked && kInto)) x = pairs_of(raw[u]);
          if (kPart != kValue && n > 0) {
            Pairs y = x;
            if (PAIRING == kHalves) {
              Eight<ES> other;
#pragma unroll
              for (int i = 0; i < ES * 2; ++i) other.w[i] = __shfl_sync(0xffffffffu, raw[u].w[i], partner);
              y = pairs_of(other);
            } else if (PAIRING == kNeighbours) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float lo_, hi_;
                unpair(x.v[i], lo_, hi_);
                y.v[i] = pair(hi_, lo_);
              }
            } else {
              if (turned && have) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int d = d0 + e;
                  f[e] = 0.0f;
                  if (d < 2 * n) {
                    const char* o = src + u * src_step + (d < n ? n + e : e - n) * ES;
                    f[e] = ES == 4 ? *reinterpret_cast<const float*>(o)
                                   : __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(o)) << 16);
                  }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) y.v[i] = pair(f[2 * i], f[2 * i + 1]);
              }
              __syncwarp();  // (q_out may be q: other lanes' reads of the head come first)
            }
            if (turned) {
              const Pairs was = x;
              if constexpr (kPacked && kPart == kKey) {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                  const float4 c = s_low[warp][0][d0 / 4 + i / 2], s = s_low[warp][1][d0 / 4 + i / 2];
                  x.v[i] = turn_to_odd(x.v[i], co.v[i], pair(c.x, c.y), y.v[i], si.v[i], pair(s.x, s.y));
                  x.v[i + 1] = turn_to_odd(x.v[i + 1], co.v[i + 1], pair(c.z, c.w), y.v[i + 1], si.v[i + 1], pair(s.z, s.w));
                }
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) x.v[i] = fma_pair(x.v[i], co.v[i], mul_pair(y.v[i], si.v[i]));
              }
              if (2 * n - d0 < 8) {  // columns behind the last pair are left as they are
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float a0, a1, b0, b1;
                  unpair(x.v[i], a0, a1), unpair(was.v[i], b0, b1);
                  x.v[i] = pair(d0 + 2 * i < 2 * n ? a0 : b0, d0 + 2 * i + 1 < 2 * n ? a1 : b1);
                }
              }
              if (!kPacked || !kInto) out = round8<ES>(x);
            }
          }
          if constexpr (kPacked && kInto) {
            uint32_t codes, byte;
            odd = !quantize8(x, &codes, &byte) && have || odd;
            if (have) {
              *reinterpret_cast<uint32_t*>(dst + u * dst_step) = codes;
              if ((lane & 1) == 0) dst[u * dst_step + scale_at] = static_cast<char>(byte);
            }
          } else {
            if (have) store8<ES>(dst + u * dst_step, out, wide);
          }
        }
        src += kUnroll * src_step, dst += kUnroll * dst_step;
      }
    };
    part(std::integral_constant<Part, kQuery>{}, first, min(last, q_passes), p.q, p.q_heads);
    part(std::integral_constant<Part, kKey>{}, first - q_passes, min(last - q_passes, kv_passes), p.k, p.kv_heads);
    part(std::integral_constant<Part, kValue>{}, first - q_passes - kv_passes, min(last - q_passes - kv_passes, kv_passes), p.v, p.kv_heads);
    if (kPacked && __any_sync(0xffffffffu, odd) && lane == 0) atomicOr(p.status + b, kStNonFinite);
  }
}

// ---------------------------------------------------------------------------
// Host checks
// ---------------------------------------------------------------------------

// A [rows, heads, dim] array in bytes.
struct Span {
  const char* p;
  int64_t row, rows, head, heads, bytes;  // steps and counts; bytes of a head's row
  int64_t end() const { return (rows > 0 ? (rows - 1) * row : 0) + (heads - 1) * head + bytes; }
};

// Whether two arrays have no byte in common, as far as that shows: ranges that do not meet, or parts of the rows (or of the
// heads) of one larger array.
bool apart(const Span& a, const Span& b) {
  if (a.p + a.end() <= b.p || b.p + b.end() <= a.p) return true;
  for (int i = 0; i < 2; ++i) {
    const int64_t step = i ? a.head : a.row, other = i ? b.head : b.row;
    const int64_t in_a = i ? (a.rows - 1) * a.row + a.bytes : (a.heads - 1) * a.head + a.bytes;
    const int64_t in_b = i ? (b.rows - 1) * b.row + b.bytes : (b.heads - 1) * b.head + b.bytes;
    if (step <= 0 || step != other) continue;
    int64_t d = (b.p - a.p) % step;
    if (d < 0) d += step;
    if (in_a <= d && d + in_b <= step) return true;
  }
  return false;
}

bool meets_range(const Span& a, const char* lo, int64_t bytes) { return a.p < lo + bytes && lo < a.p + a.end(); }

sv_status_t check_array(const void* p, int64_t row, int64_t head, int es) {
  if (row < 0 || head < 0) return SV_ERR_BAD_SHAPE;
  if (!p) return SV_ERR_NULL_ARG;
  return aligned16(p) && (row * es) % 16 == 0 && (head * es) % 16 == 0 ? SV_OK : SV_ERR_MISALIGNED;
}

// The caches' memory as ranges, and whether their entries lie apart.
struct Memory {
  const char* at[2];
  int64_t bytes[2];
};
bool memory_of(const KvView& c, Memory* m) {
  StepAxis axes[4] = {{c.head_stride * c.es, c.heads}, {c.slot_stride * c.es, c.page_size},
                      {c.page_stride * c.es, c.pages}, {c.layer_stride * c.es, c.layers}};
  int64_t span = 0;
  if (!entries_apart(c) || !steps_nested(axes, 4, static_cast<int64_t>(c.head_dim) * c.es, &span)) return false;
  *m = Memory{{c.k, c.v}, {span, span}};
  return true;
}
bool memory_of(const PackedView& c, Memory* m) {
  StepAxis axes[3] = {{c.head_stride, c.heads}, {c.page_stride, c.pages}, {c.layer_stride, c.layers}};
  int64_t span = 0;
  if (!steps_nested(axes, 3, packed_block_bytes(c.page_size, c.head_dim), &span)) return false;
  *m = Memory{{c.data, c.data}, {span, span}};
  return true;
}

void to_layer(KvView* c, int layer) {
  c->k += layer * c->layer_stride * c->es;
  c->v += layer * c->layer_stride * c->es;
}
void to_layer(PackedView* c, int layer) { c->data += layer * c->layer_stride; }

template <int ES, class C>
cudaError_t launch_append(const AppendParams& p, const C& c, Pairing pairing, unsigned grid, cudaStream_t stream) {
  auto kernel = pairing == kNeighbours ? k_kv_append<ES, C, kNeighbours>
                : pairing == kHalves   ? k_kv_append<ES, C, kHalves>
                                       : k_kv_append<ES, C, kHalvesOdd>;
  return launch_pdl(kernel, dim3(grid), dim3(32 * kAppendWarps), 0, stream, p, c);
}

template <class C>
sv_status_t append_entry(C c, int es, int32_t layer, const sv_rows_t* rows, const int64_t* positions,
                         const sv_rotation_t* rotation, const HeadRows& k, const HeadRows& v, const HeadRows& q,
                         int32_t num_heads, void* q_out, int64_t o_row, int64_t o_head, uint32_t* dev_status,
                         cudaStream_t stream) {
  RowsView r{};
  sv_status_t s = check_rows(rows, &r);
  if (s != SV_OK) return s;
  if (layer < 0 || layer >= c.layers) return SV_ERR_BAD_SHAPE;
  if (q.p && (num_heads < 1 || num_heads > (1 << 20))) return SV_ERR_BAD_SHAPE;
  if (!q.p) num_heads = 0;
  if (rotation && (rotation->pairs < 0 || 2 * static_cast<int64_t>(rotation->pairs) > c.head_dim ||
                   !std::isfinite(rotation->magnitude)))
    return SV_ERR_BAD_SHAPE;
  if (r.batch == 0 || rows_count(r) == 0) return SV_OK;
  if (!dev_status || (rotation && rotation->pairs > 0 && !rotation->inv_freq)) return SV_ERR_NULL_ARG;
  if (!r.seq_lens && (!r.row_slots || (rotation && !positions))) return SV_ERR_NULL_ARG;
  if ((s = check_array(k.p, k.row, k.head, es)) != SV_OK || (s = check_array(v.p, v.row, v.head, es)) != SV_OK) return s;
  if (q.p && ((s = check_array(q.p, q.row, q.head, es)) != SV_OK || (s = check_array(q_out, o_row, o_head, es)) != SV_OK)) return s;
  const int64_t bytes = static_cast<int64_t>(c.head_dim) * es;
  const Span sk{k.p, k.row * es, r.total, k.head * es, c.heads, bytes}, sv{v.p, v.row * es, r.total, v.head * es, c.heads, bytes};
  Memory m{};
  if (!memory_of(c, &m)) return SV_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i)
    if (meets_range(sk, m.at[i], m.bytes[i]) || meets_range(sv, m.at[i], m.bytes[i])) return SV_ERR_UNSUPPORTED;
  if (q.p) {
    const Span sq{q.p, q.row * es, r.total, q.head * es, num_heads, bytes};
    const Span so{static_cast<const char*>(q_out), o_row * es, r.total, o_head * es, num_heads, bytes};
    StepAxis axes[2] = {{so.row, so.rows}, {so.head, so.heads}};
    int64_t span;
    if (!steps_nested(axes, 2, bytes, &span)) return SV_ERR_UNSUPPORTED;
    const bool same = sq.p == so.p && (r.total < 2 || sq.row == so.row) && (num_heads < 2 || sq.head == so.head);
    if ((!same && !apart(so, sq)) || !apart(so, sk) || !apart(so, sv)) return SV_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i)
      if (meets_range(so, m.at[i], m.bytes[i]) || meets_range(sq, m.at[i], m.bytes[i])) return SV_ERR_UNSUPPORTED;
  }
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  to_layer(&c, layer);
  const int lanes = (c.head_dim + 7) / 8, heads = 32 / lanes;
  const int64_t passes = (num_heads + heads - 1) / heads + 2 * static_cast<int64_t>((c.heads + heads - 1) / heads);
  // As many warps a row as it takes to give every multiprocessor sixteen.
  const int64_t count = rows_count(r), want = 16 * static_cast<int64_t>(dev.sms);
  int64_t chunks = (want + count - 1) / count;
  chunks = chunks > passes ? passes : chunks;
  const int64_t per = (passes + chunks - 1) / chunks;
  chunks = (passes + per - 1) / per;
  const int n = rotation ? rotation->pairs : 0;
  const AppendParams p{r, positions, rotation ? rotation->inv_freq : nullptr, n, rotation ? rotation->magnitude : 1.0f, q, k, v,
                       static_cast<char*>(q_out), o_row, o_head, num_heads, c.heads, c.head_dim, dev_status,
                       static_cast<int32_t>(passes), static_cast<int32_t>(chunks), static_cast<int32_t>(per)};
  const int64_t blocks = (count * chunks + kAppendWarps - 1) / kAppendWarps, most = 64 * static_cast<int64_t>(dev.sms);
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  const Pairing pairing = n == 0 || rotation->interleaved ? kNeighbours : n % 8 == 0 ? kHalves : kHalvesOdd;
  e = es == 2 ? launch_append<2>(p, c, pairing, grid, stream) : launch_append<4>(p, c, pairing, grid, stream);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

sv_status_t spec_verify_kv_append(const sv_kv_cache_t* cache, int32_t layer, const sv_rows_t* rows,
                                  const int64_t* positions, const sv_rotation_t* rotation, const void* k,
                                  int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
                                  int64_t v_head_stride, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                  int32_t num_heads, void* q_out, int64_t out_row_stride, int64_t out_head_stride,
                                  uint32_t* dev_status, cudaStream_t stream) {
  KvView c{};
  const sv_status_t s = check_cache(cache, &c);
  if (s != SV_OK) return s;
  return append_entry(c, c.es, layer, rows, positions, rotation,
                      HeadRows{static_cast<const char*>(k), k_row_stride, k_head_stride},
                      HeadRows{static_cast<const char*>(v), v_row_stride, v_head_stride},
                      HeadRows{static_cast<const char*>(q), q_row_stride, q_head_stride}, num_heads, q_out,
                      out_row_stride, out_head_stride, dev_status, stream);
}

sv_status_t spec_verify_packed_kv_append(const sv_packed_kv_cache_t* cache, int32_t layer, const sv_rows_t* rows,
                                         const int64_t* positions, const sv_rotation_t* rotation, const void* k,
                                         int64_t k_row_stride, int64_t k_head_stride, const void* v,
                                         int64_t v_row_stride, int64_t v_head_stride, const void* q,
                                         int64_t q_row_stride, int64_t q_head_stride, int32_t num_heads, void* q_out,
                                         int64_t out_row_stride, int64_t out_head_stride, uint32_t* dev_status,
                                         cudaStream_t stream) {
  PackedView c{};
  const sv_status_t s = check_packed_cache(cache, &c);
  if (s != SV_OK) return s;
  return append_entry(c, c.dtype == SV_BF16 ? 2 : 4, layer, rows, positions, rotation,
                      HeadRows{static_cast<const char*>(k), k_row_stride, k_head_stride},
                      HeadRows{static_cast<const char*>(v), v_row_stride, v_head_stride},
                      HeadRows{static_cast<const char*>(q), q_row_stride, q_head_stride}, num_heads, q_out,
                      out_row_stride, out_head_stride, dev_status, stream);
}

}  // extern "C"
