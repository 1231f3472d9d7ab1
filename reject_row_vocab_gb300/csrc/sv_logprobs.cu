// Log probabilities of given tokens, with entropy and top alternatives, and
// their gradient by the logits ([E2D] §6.2: the target is softmax(l / T)).
//
// Forward, k_token_logprobs.  With k = log2(e) / T and M the row maximum,
//   Z = sum 2^((l - M) k),  W = sum (l - M) 2^((l - M) k)
//   logprob(id) = (l_id - M) / T - ln Z,   H = ln Z - (W / Z) / T.
// One pass: each thread keeps a running (m, s, w) of the elements it has read
// and rescales it when its maximum grows; a block joins its threads' triples,
// and the last block of a row joins the blocks' in block order, so results do
// not depend on the order the blocks finish in.  An element costs an exponential
// and about three and a half other issues, a batch of vectors is asked for only
// when the one before is used up: issue slots and DRAM are each about half
// used, and most waits are for memory.  Measured: 1024 rows of 151936 bf16, 20
// alternatives: 65 us, 4.8 TB/s; without alternatives 57 us; 5 rows of 32000
// fp32, 5 alternatives: 13 us, latency.
//
// Top alternatives from the same pass: a thread's running maximum is the
// largest of its own elements, so the top_k-th largest of the block's thread
// maxima is a lower bound on the block's top_k-th element.  Only batches whose
// largest logit reaches the bound (about top_k of some thousands; their maxima
// are put down as they pass) can hold a top element, and only they are read
// again: all elements of the threads that reach it, 8 percent of the row, cost
// as much as a fifth of the pass.  Elements
// are ordered by a 64-bit key - value, then the lower index - so the selection
// is unique whatever the order of the candidates.
//
// Backward, k_token_logprobs_bwd.  With t = (l - M) k - log2 Z and p = 2^t,
//   dl = p (A + B t) + (the row's given tokens)/T,
//   A = -(G + gH H)/T,  B = -gH ln 2 / T:
// two multiply-adds and an exponential an element between a read and a write.
// Bound by the bytes.  Measured: 1024 rows of 151936 bf16 with an entropy term:
// 98 us, 6.4 TB/s; 80 rows of 32003 fp32: 11 us.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cfloat>
#include <cstdint>
#include <mutex>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kLpThreads = 128;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 64;
constexpr int kMaxGiven = 1024;
constexpr int kMaxBlocks = 1280;    // of the forward kernel (the workspace is laid out for them)
constexpr int kMinVectors = 1024;   // 16-byte vectors that a block takes at least
constexpr int kCandCap = 1024;  // candidates a block sorts in shared memory
constexpr int kBatch = 4;       // vectors that a thread reads at once
constexpr int kPeaks = 40;      // groups of batches whose largest logits are kept
constexpr float kLn2 = 0.693147180559945309417f;

// A logits vector: 16 bytes as floats.
template <bool BF16>
struct Vec;
template <>
struct Vec<true> {
  static constexpr int N = 8;
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = bf16_lo(u.x), f[1] = bf16_hi(u.x), f[2] = bf16_lo(u.y), f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z), f[5] = bf16_hi(u.z), f[6] = bf16_lo(u.w), f[7] = bf16_hi(u.w);
  }
};
template <>
struct Vec<false> {
  static constexpr int N = 4;
  __device__ static void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
};

// The largest of a vector's logits that are numbers.
template <bool BF16>
__device__ __forceinline__ float largest(const uint4& u) {
  if (BF16) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(u.x), "r"(u.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u.z), "r"(u.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return fmaxf(bf16_lo(a), bf16_hi(a));
  }
  return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}

// Order-preserving whole number of a float (-0 as 0); 0 stands for "no element" (-inf and unusable logits).
__device__ __forceinline__ uint32_t ordered(float x) {
  if (!usable_logit(x) || x == -kInfF) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ uint64_t top_key(float x, int32_t idx) {
  const uint32_t o = ordered(x);
  return o == 0u ? 0ull : (static_cast<uint64_t>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}

// Running sums of a thread, block or row against a reference m, with t = (l - m) k: s = sum 2^t, w = sum t 2^t.
struct Run {
  float m, s, w;
};

__device__ __forceinline__ void run_merge(Run& a, const Run& b, float k) {
  if (b.m == -kInfF) return;
  if (a.m == -kInfF) {
    a = b;
    return;
  }
  const float M = fmaxf(a.m, b.m);
  const float da = (a.m - M) * k, db = (b.m - M) * k;
  const float ea = ex2_fast(da), eb = ex2_fast(db);
  // a term that vanished has sums that vanish with it (0 times a large distance is 0, not a stray product)
  a.w = (ea > 0.0f ? ea * fmaf(a.s, da, a.w) : 0.0f) + (eb > 0.0f ? eb * fmaf(b.s, db, b.w) : 0.0f);
  a.s = ea * a.s + eb * b.s;
  a.m = M;
}

// The lanes' triples, in order (both sides of an exchange join the lower lane's first): the same in every lane.  Rolled, as
// what runs once a row is: its instructions are fetched anew each time.
__device__ __forceinline__ Run run_join(Run r, float k) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int off = 1; off < 32; off <<= 1) {
    Run o{__shfl_xor_sync(0xffffffffu, r.m, off), __shfl_xor_sync(0xffffffffu, r.s, off),
          __shfl_xor_sync(0xffffffffu, r.w, off)};
    if (lane & off) {
      const Run mine = r;
      r = o;
      o = mine;
    }
    run_merge(r, o, k);
  }
  return r;
}

// log2(e) / T, of the unscaled distribution for a greedy temperature.  Held at 1e-30 at least: there every finite logit of
// ordinary size has the same weight, and a masked entry's distance still has to end in a weight of zero.
__device__ __forceinline__ float logprob_temperature(const float* row_temp, int64_t i) {
  const float T = row_temp ? row_temp[i] : 1.0f;
  return sampling_temperature(T) ? T : 1.0f;
}
__device__ __forceinline__ float logprob_k(float T) { return fmaxf(temperature_k(T), 1e-30f); }

struct LogprobParams {
  LogitsView lg;
  int64_t n;
  const int32_t* row_index;
  const int32_t* ids;
  int32_t num_ids;
  int64_t ldi;
  const float* row_temp;
  int32_t top_k;
  float* logprob;
  float* entropy;
  float* row_max;
  float* log_z;
  int32_t* top_ids;
  float* top_logprob;
  uint32_t* flags;
  uint32_t* tickets;  // [kMaxBlocks], zero between calls
  Run* part;          // [kMaxBlocks][2]
  uint32_t* part_flags;
  uint64_t* part_top;  // [kMaxBlocks][2][top_k]
  int64_t min_vectors;  // that a block takes
};

template <bool BF16>
__device__ __forceinline__ float logit_at(const LogitsView& lg, int64_t row, int64_t col) {
  const int64_t i = row * lg.ld + col;
  if (BF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(lg.base) + i)) << 16);
  return __ldg(static_cast<const float*>(lg.base) + i);
}

// One element joins a running triple (the ragged end of a row, and vectors that hold NaN or +inf).
__device__ __forceinline__ void run_add(Run& r, float x, float k, uint32_t& flags) {
  if (!usable_logit(x)) {
    flags |= kStNonFinite;
    return;
  }
  if (x == -kInfF) return;
  run_merge(r, Run{x, 1.0f, 0.0f}, k);
}

// A thread's running sums while it streams, against a reference: weights are 2^(l k - c) with c = ref k as rounded, one
// multiply-add an element; settle() makes up for the rounding, which is the same for all of them.  That needs a rounding
// within the exponent's range: it is past it from |ref| k = 2^31 on, as in a row masked with -1e10 or at temperatures below
// 1e-8.  A reference that is `far` is therefore subtracted before the product, an operation a pair of elements more (all
// rows done that way: 66.7 us for 1024 of 151936, where this took 64.4).  The reference is the largest logit of the
// warp's first vectors, and moves only when a logit passes it by 64 log2 units (2^64 times a row's length is far from fp32's
// end): moving it at every new maximum made up two thirds of the instructions.  Logits below `low` are read as `low`, which
// has a weight of 0 just as well: their exponent stays finite, and 0 times it is 0.
template <bool BF16>
struct Stream {
  Run r{-kInfF, 0.0f, 0.0f};  // what has been settled
  float ref = -kInfF, c = 0.0f, low = -kInfF, limit = -kInfF;  // the same in all lanes of a warp
  uint32_t low2 = 0xff80ff80u;
  bool far = false;
  bool packed = true;  // false: no number below the reference has a finite exponent: element by element
  float2 s2{0.0f, 0.0f}, w2{0.0f, 0.0f};

  __device__ __forceinline__ void settle(float k) {
    if (ref == -kInfF || !packed) return;
    const float off = far ? 0.0f : fmaf(ref, -k, c);  // c - ref k, exactly: 2^(l k - c) 2^off = 2^t and t = (l k - c) + off
    const float e = ex2_fast(off), s = s2.x + s2.y, w = w2.x + w2.y;
    run_merge(r, Run{ref, e * s, e * fmaf(s, off, w)}, k);
    s2 = w2 = make_float2(0.0f, 0.0f);
  }
  // A larger reference; unit: 1 / k.  Both ends are rounded down: where 300 or 64 units are less than the reference's last
  // place, `low` is the number below it, and `limit` the reference itself.
  __device__ __forceinline__ void rise(float to, float k, float unit) {
    settle(k);
    ref = to;
    c = ref * k;
    far = !(fabsf(c) < 0x1p24f);  // the rounding of c is one half at most
    low = __fmaf_rd(-300.0f, unit, ref);
    limit = __fmaf_rd(64.0f, unit, ref);
    if (BF16) {
      uint32_t b = __float_as_uint(low);
      if (low < 0.0f && (b & 0xffffu)) b += 0x10000u;
      b >>= 16;
      low2 = b | b << 16;
      low = bf16_hi(low2);
    }
    packed = (ref - low) * k < 1e37f;
  }
  // A vector's elements (two at a time), all of them numbers, to sums of the batch: a row in one block gives a thread some
  // 600 elements for each half, and beside a likely token's weight the last bits of the many small ones would be lost.
  template <bool FAR>
  __device__ __forceinline__ void add(uint4 u, float k, float2& bs, float2& bw) const {
    constexpr int N = Vec<BF16>::N;
    const float2 kk = make_float2(k, k), cc = make_float2(-c, -c), from = make_float2(-ref, -ref);
    if (BF16) {
      u.x = bmax2_nan(u.x, low2), u.y = bmax2_nan(u.y, low2);
      u.z = bmax2_nan(u.z, low2), u.w = bmax2_nan(u.w, low2);
    }
    float f[N];
    Vec<BF16>::unpack(u, f);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      float2 x = make_float2(f[e], f[e + 1]);
      if (!BF16) x = make_float2(fmaxf(x.x, low), fmaxf(x.y, low));
      const float2 y = FAR ? __fmul2_rn(__fadd2_rn(x, from), kk) : __ffma2_rn(x, kk, cc);
      const float2 z = make_float2(ex2_fast(y.x), ex2_fast(y.y));
      bs = __fadd2_rn(bs, z);
      bw = __ffma2_rn(y, z, bw);
    }
  }
};

// The top_k largest of the n keys in `cand` (unique, in any order), sorted into `out` (top_k entries, 0 = none).
__device__ __forceinline__ void rank_top(const uint64_t* cand, int n, int top_k, uint64_t* out) {
  for (int i = threadIdx.x; i < top_k; i += kLpThreads) out[i] = 0ull;
  __syncthreads();
  for (int c = threadIdx.x; c < n; c += kLpThreads) {
    const uint64_t key = cand[c];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += cand[j] > key ? 1 : 0;
    if (key != 0ull && rank < top_k) out[rank] = key;
  }
  __syncthreads();
}

// Shared memory of a block.
struct LogprobShared {
  Run run[kLpWarps];
  float max[kLpWarps];
  uint64_t cand[kCandCap];
  uint64_t top[kMaxTop];
  uint64_t key[kLpWarps];
  alignas(16) uint16_t level[kLpThreads];
  uint16_t peak[kPeaks][kLpThreads];  // the largest logit of each thread's groups of batches, as 16-bit bounds
  uint16_t who[kCandCap];             // groups that may hold a top element: thread + kLpThreads group
  int64_t sums[kLpWarps];
  int64_t find[2];
  uint32_t flags, found, last, owners, bound;
};

// The top_k keys of vectors [lo, hi) of a row (and of its ragged end, tails elements from tail0) into sh.top, given each
// thread's largest logit of its own vectors lo + t, lo + t + kLpThreads, ... (and the end), and sh.peak, where a group is
// `batches` batches of kBatch of them.
template <bool BF16>
__device__ __noinline__ void select_top(const LogprobParams& p, LogprobShared& sh, int64_t row, int lo, int hi, int tail0,
                                        int tails, float mine_max, int batches) {
  constexpr int N = Vec<BF16>::N;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint4* vec = reinterpret_cast<const uint4*>(static_cast<const char*>(p.lg.base) + row * p.lg.ld * (BF16 ? 2 : 4));
  // The largest 16-bit bound that top_k threads' maxima reach, found bit by bit by one warp.
  const uint32_t mine = ordered(mine_max) >> 16;
  sh.level[t] = static_cast<uint16_t>(mine);
  if (t == 0) sh.found = 0u, sh.owners = 0u;
  __syncthreads();
  if (warp == 0) {
    uint32_t v[kLpWarps], most = 0u, least = 0xffffu;
#pragma unroll
    for (int e = 0; e < kLpWarps; ++e) v[e] = sh.level[lane + 32 * e], most = max(most, v[e]), least = min(least, v[e]);
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    const int differ = (32 - __clz(most ^ least) + 1) & ~1;  // bits below the leading ones that all have
    uint32_t thr = most >> differ << differ;
    const uint32_t k = static_cast<uint32_t>(p.top_k);
#pragma unroll 1
    for (int bit = differ - 2; bit >= 0; bit -= 2) {  // three candidates a step, their threads counted in ten bits each
      uint32_t n = 0u;
#pragma unroll
      for (int e = 0; e < kLpWarps; ++e) {
        const uint32_t d = v[e] >> bit, to = thr >> bit;
        n += (d >= (to | 1u) ? 1u : 0u) + (d >= (to | 2u) ? 1u << 10 : 0u) + (d >= (to | 3u) ? 1u << 20 : 0u);
      }
      n = __reduce_add_sync(0xffffffffu, n);
      thr |= ((n >> 20) >= k ? 3u : (n >> 10 & 0x3ffu) >= k ? 2u : (n & 0x3ffu) >= k ? 1u : 0u) << bit;
    }
    if (lane == 0) sh.bound = max(thr, 1u);  // 0 stands for no element
  }
  __syncthreads();
  const uint32_t bound = sh.bound;
  // no element below it counts (bounds up to that of the lowest number let everything pass)
  const float least = bound > 0x80u ? from_ordered(bound << 16) : -kInfF;
  const int span = kLpThreads * kBatch * batches;  // vectors of the line between a thread's groups
  if (mine >= bound)
#pragma unroll 4
    for (int group = 0; lo + group * span < hi; ++group)
      if (sh.peak[group][t] >= bound) {
        const uint32_t at = atomicAdd(&sh.owners, 1u);
        if (at < kCandCap) sh.who[at] = static_cast<uint16_t>(t + kLpThreads * group);
      }
  auto offer = [&](float f, int idx) {
    if ((ordered(f) >> 16) >= bound) {
      const uint32_t at = atomicAdd(&sh.found, 1u);
      if (at < kCandCap) sh.cand[at] = top_key(f, idx);
    }
  };
  if (t < tails && mine >= bound) offer(logit_at<BF16>(p.lg, row, tail0 + t), tail0 + t);
  __syncthreads();
  const int who = static_cast<int>(sh.owners);
  const int per = kBatch * batches;  // vectors of a group
  if (who <= kCandCap) {             // those groups' vectors again
    for (int y = t; y < who * per; y += kLpThreads) {
      const int item = y / per, w = sh.who[item];
      const int x = lo + w / kLpThreads * span + w % kLpThreads + (y - item * per) * kLpThreads;
      if (x >= hi) continue;
      uint4 u = ld_stream16(vec + x);
      if (largest<BF16>(u) < least) continue;
#pragma unroll 1
      for (int e = 0; e < N; e += N / 4) {  // word by word
        offer(BF16 ? bf16_lo(u.x) : __uint_as_float(u.x), x * N + e);
        if (BF16) offer(bf16_hi(u.x), x * N + e + 1);
        u.x = u.y, u.y = u.z, u.z = u.w;
      }
    }
  } else if (t == 0) {
    sh.found = kCandCap + 1;
  }
  __syncthreads();
  const uint32_t found = sh.found;
  if (found <= kCandCap) {
    rank_top(sh.cand, static_cast<int>(found), p.top_k, sh.top);
    return;
  }
  // More candidates than the sort holds (long runs of equal logits): one block-wide search an alternative.
  uint64_t last = ~0ull;
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0ull;
    for (int x = lo + t; x < hi; x += kLpThreads) {
      float f[N];
      Vec<BF16>::unpack(ld_stream16(vec + x), f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint64_t key = top_key(f[e], x * N + e);
        if (key < last && key > best) best = key;
      }
    }
    if (t < tails) {
      const uint64_t key = top_key(logit_at<BF16>(p.lg, row, tail0 + t), tail0 + t);
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
    if (lane == 0) sh.key[warp] = best;
    __syncthreads();
    best = 0ull;
    for (int w = 0; w < kLpWarps; ++w) best = max(best, sh.key[w]);
    if (t == 0) sh.top[j] = best;
    last = best == 0ull ? 1ull : best;  // nothing left: no key is below 1
    __syncthreads();
  }
}

// Joins the parts of a row, left by blocks c0 .. c1, into sh.run[0], sh.flags and sh.top.
__device__ __noinline__ void join_parts(const LogprobParams& p, LogprobShared& sh, int c0, int c1, float k) {
  const int t = threadIdx.x;
  auto slot = [&](int c) { return c * 2 + (c == c0 ? 1 : 0); };  // a block's first row began before it, but for the first
  if (t < 32) {  // a lane a part (and the 32nd after it), then the lanes in order
    Run r{-kInfF, 0.0f, 0.0f};
    uint32_t f = 0u;
    for (int c = c0 + t; c <= c1; c += 32) {
      const Run* q = p.part + slot(c);
      const Run o{__ldcg(&q->m), __ldcg(&q->s), __ldcg(&q->w)};
      f |= __ldcg(&p.part_flags[slot(c)]);
      run_merge(r, o, k);
    }
    r = run_join(r, k);
    f = __reduce_or_sync(0xffffffffu, f);
    if (t == 0) {
      sh.run[0] = r;
      sh.flags = f;
      sh.found = 0u;
      sh.key[0] = 0ull;
    }
  }
  __syncthreads();
  if (p.top_k == 0) return;
  // A part's last key is a lower bound on the row's top_k-th: the largest of them leaves about top_k keys.
  for (int c = c0 + t; c <= c1; c += kLpThreads)
    atomicMax(reinterpret_cast<unsigned long long*>(&sh.key[0]),
              static_cast<unsigned long long>(__ldcg(&p.part_top[static_cast<int64_t>(slot(c)) * p.top_k + p.top_k - 1])));
  __syncthreads();
  const uint64_t bound = sh.key[0];
  for (int x = t; x < (c1 - c0 + 1) * p.top_k; x += kLpThreads) {
    const uint64_t key = __ldcg(&p.part_top[static_cast<int64_t>(slot(c0 + x / p.top_k)) * p.top_k + x % p.top_k]);
    if (key != 0ull && key >= bound) {
      const uint32_t at = atomicAdd(&sh.found, 1u);
      if (at < kCandCap) sh.cand[at] = key;
    }
  }
  __syncthreads();
  rank_top(sh.cand, min(static_cast<int>(sh.found), kCandCap), p.top_k, sh.top);
}

// The outputs of row i from sh.run[0], sh.flags and sh.top.
template <bool BF16>
__device__ __noinline__ void write_outputs(const LogprobParams& p, LogprobShared& sh, int64_t i, int64_t row, float T) {
  const int t = threadIdx.x;
  const Run r = sh.run[0];
  const bool empty = r.m == -kInfF;
  const float lz = empty ? -kInfF : logf(r.s);
  bool range = false;
  for (int j = t; j < p.num_ids; j += kLpThreads) {
    const int32_t id = p.ids[i * p.ldi + j];
    float lp = 0.0f;
    if (id != -1) {
      lp = -kInfF;
      if (id >= 0 && id < p.lg.vocab) {
        const float l = logit_at<BF16>(p.lg, row, id);
        if (usable_logit(l) && l != -kInfF) lp = __fdiv_rn(l - r.m, T) - lz;
      } else {
        range = true;
      }
    }
    p.logprob[i * p.num_ids + j] = lp;
  }
  for (int j = t; j < p.top_k; j += kLpThreads) {
    const uint64_t key = sh.top[j];
    p.top_ids[i * p.top_k + j] = key ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    p.top_logprob[i * p.top_k + j] =
        key ? __fdiv_rn(from_ordered(static_cast<uint32_t>(key >> 32)) - r.m, T) - lz : -kInfF;
  }
  const int outside = __syncthreads_or(range ? 1 : 0);
  if (t == 0) {
    // the entropy of a distribution is not negative; rounding may leave a value just below 0
    const float h = fmaf(__fdiv_rn(r.w, r.s), -kLn2, lz);
    if (p.entropy) p.entropy[i] = empty || h < 0.0f ? 0.0f : h;
    if (p.row_max) p.row_max[i] = r.m;
    if (p.log_z) p.log_z[i] = lz;
    if (p.flags) p.flags[i] = sh.flags | (outside ? kStTokenRange : 0u) | (empty ? kStNonFinite : 0u);
  }
}

__device__ __forceinline__ void write_padding(const LogprobParams& p, int64_t i, uint32_t flags) {
  for (int j = 0; j < p.num_ids; ++j) p.logprob[i * p.num_ids + j] = 0.0f;
  for (int j = 0; j < p.top_k; ++j) p.top_ids[i * p.top_k + j] = -1, p.top_logprob[i * p.top_k + j] = -kInfF;
  if (p.entropy) p.entropy[i] = 0.0f;
  if (p.row_max) p.row_max[i] = -kInfF;
  if (p.log_z) p.log_z[i] = 0.0f;
  if (p.flags) p.flags[i] = flags;
}

// The vectors of all rows form one line; block c of g takes vectors [c total / g, (c + 1) total / g) of it, so that every
// block reads as much, however many rows there are and whichever of them are padding.  A row that lies in one block is
// finished there; of one that several share each leaves its part, and the last to arrive joins them in block order.
template <bool BF16>
__global__ void __launch_bounds__(kLpThreads, 7) k_token_logprobs(LogprobParams p) {
  constexpr int N = Vec<BF16>::N;
  constexpr int U = kBatch;
  __shared__ LogprobShared sh;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  grid_dependency_wait();
  allow_dependents();
  const int nvec = p.lg.vocab / N, tail0 = nvec * N;
  const int per_row = nvec > 0 ? nvec : 1;  // (a row of less than a vector has its ragged end only)

  // Rows that there are, and the padding.
  auto padding = [&](int64_t i) {
    const int64_t r = p.row_index[i];
    return r < 0 || r >= p.lg.rows;
  };
  int64_t rows = p.n;
  if (p.row_index) {
    int64_t mine = 0;
    for (int64_t i = t; i < p.n; i += kLpThreads) mine += padding(i) ? 0 : 1;
    for (int64_t i = blockIdx.x * kLpThreads + t; i < p.n; i += static_cast<int64_t>(gridDim.x) * kLpThreads)
      if (padding(i)) write_padding(p, i, p.row_index[i] == -1 ? 0u : kStBadLayout);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
    if (lane == 0) sh.sums[warp] = mine;
    __syncthreads();
    rows = 0;
#pragma unroll
    for (int w = 0; w < kLpWarps; ++w) rows += sh.sums[w];
    __syncthreads();
  }
  const int64_t total = rows * per_row;
  int64_t g = total / p.min_vectors;
  if (g > gridDim.x) g = gridDim.x;
  if (g < 1) g = 1;
  // a whole number of blocks a row, where that leaves few of them idle: then no block has parts of two
  if (rows > 0 && rows <= g && g / rows * rows * 5 >= g * 4) g = g / rows * rows;
  // ... or of rows a block
  const int64_t each = rows > g ? (rows + g - 1) / g : 1;
  if (each > 1 && rows % each == 0 && rows / each * 5 >= g * 4) g = rows / each;
  if (blockIdx.x >= g || total == 0) return;
  const int64_t start = blockIdx.x * total / g, end = (blockIdx.x + 1) * total / g;
  int64_t ord = start / per_row;  // rows before this block's first one
  int64_t i = ord;                // its output
  if (p.row_index) {              // the ord-th output that is not padding
    int64_t before = 0;
    for (int64_t i0 = 0; i0 < p.n; i0 += kLpThreads) {
      const bool is = i0 + t < p.n && !padding(i0 + t);
      const uint32_t b = __ballot_sync(0xffffffffu, is);
      if (lane == 0) sh.sums[warp] = __popc(b);
      __syncthreads();
      int64_t at = before;
#pragma unroll
      for (int w = 0; w < kLpWarps; ++w) {
        if (w == warp && is && at + __popc(b & ((1u << lane) - 1u)) == ord) sh.find[0] = i0 + t;
        at += sh.sums[w];
      }
      before = at;
      __syncthreads();
      if (before > ord) break;
    }
    i = sh.find[0];
  }

  for (int64_t pos = start; pos < end; ++i) {
    if (p.row_index && padding(i)) continue;
    const int64_t row = p.row_index ? p.row_index[i] : i;
    const int64_t row0 = ord * per_row;  // the row's first place in the line
    const int lo = static_cast<int>(pos - row0);
    const int hi = static_cast<int>(min(static_cast<int64_t>(per_row), end - row0));
    const int vhi = min(hi, nvec);
    const bool whole = lo == 0 && hi == per_row;
    const int tails = hi == per_row ? p.lg.vocab - tail0 : 0;  // the ragged end belongs to the row's last block
    pos = row0 + hi;
    ++ord;
    const float T = logprob_temperature(p.row_temp, i);
    const float k = logprob_k(T), unit = __frcp_rn(k);
    const uint4* vec = reinterpret_cast<const uint4*>(static_cast<const char*>(p.lg.base) + row * p.lg.ld * (BF16 ? 2 : 4));

    Stream<BF16> st;
    uint32_t flags = 0u;
    float top = -kInfF;  // the thread's largest usable logit
    // batches of a group, so that the groups fit sh.peak; the current one's largest, its batches so far, its number
    const int batches = ((vhi - lo + kLpThreads * U - 1) / (kLpThreads * U) + kPeaks - 1) / kPeaks;
    float peak = -kInfF;
    int had = 0, group = 0;
    auto batch_done = [&](float m) {
      top = fmaxf(top, m);
      if (p.top_k == 0) return;
      peak = fmaxf(peak, m);
      if (++had == batches) {
        sh.peak[group++][t] = static_cast<uint16_t>(ordered(peak) >> 16);
        peak = -kInfF;
        had = 0;
      }
    };
    for (int v0 = lo + warp * 32; v0 < vhi; v0 += kLpThreads * U) {
      uint4 u[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int x = v0 + lane + j * kLpThreads;
        // beyond the part: all -inf (bf16 pairs 0xff80, fp32 0xff800000)
        u[j] = x < vhi ? ld_stream16(vec + x)
                       : (BF16 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                               : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u));
      }
      float vm;
      if (BF16) {
        uint32_t a = 0xff80ff80u;
#pragma unroll
        for (int j = 0; j < U; ++j)
          a = bmax2_nan(a, bmax2_nan(bmax2_nan(u[j].x, u[j].y), bmax2_nan(u[j].z, u[j].w)));
        vm = fmax_nan(bf16_lo(a), bf16_hi(a));
      } else {
        vm = -kInfF;
#pragma unroll
        for (int j = 0; j < U; ++j)
          vm = fmax_nan(vm, fmax_nan(fmax_nan(__uint_as_float(u[j].x), __uint_as_float(u[j].y)),
                                     fmax_nan(__uint_as_float(u[j].z), __uint_as_float(u[j].w))));
      }
      const bool odd = !usable_logit(vm);  // a NaN or +inf among them
      if (__any_sync(0xffffffffu, odd || vm > st.limit)) {
        float to = odd ? -kInfF : vm;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, off));
        if (to > st.limit) st.rise(to, k, unit);
      }
      if (odd || !st.packed) {  // element by element
        float most = -kInfF;
#pragma unroll 1
        for (int j = 0; j < U; ++j) {
          float f[N];
          Vec<BF16>::unpack(j == 0 ? u[0] : j == 1 ? u[1] : j == 2 ? u[2] : u[U - 1], f);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            run_add(st.r, f[e], k, flags);
            if (usable_logit(f[e])) most = fmaxf(most, f[e]);
          }
        }
        batch_done(most);
        continue;
      }
      batch_done(vm);
      if (st.ref == -kInfF) continue;  // nothing above -inf yet
      float2 s2 = make_float2(0.0f, 0.0f), w2 = make_float2(0.0f, 0.0f);
      if (st.far) {
#pragma unroll 1
        for (int j = 0; j < U; ++j)
          st.template add<true>(j == 0 ? u[0] : j == 1 ? u[1] : j == 2 ? u[2] : u[U - 1], k, s2, w2);
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j) st.template add<false>(u[j], k, s2, w2);
      }
      st.s2 = __fadd2_rn(st.s2, s2);
      st.w2 = __fadd2_rn(st.w2, w2);
    }
    st.settle(k);
    if (had > 0) sh.peak[group][t] = static_cast<uint16_t>(ordered(peak) >> 16);
    Run r = st.r;
    if (t < tails) {
      const float l = logit_at<BF16>(p.lg, row, tail0 + t);
      run_add(r, l, k, flags);
      if (usable_logit(l)) top = fmaxf(top, l);
    }
    if (t == 0) sh.flags = 0u;
    __syncthreads();
    if (p.top_k > 0) select_top<BF16>(p, sh, row, lo, vhi, tail0, tails, top, batches);

    // Join the threads' sums.
    r = run_join(r, k);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0) {
      sh.run[warp] = r;
      sh.max[warp] = top;
      if (flags) atomicOr(&sh.flags, flags);
    }
    __syncthreads();
    if (t == 0) {
      r = sh.run[0];
#pragma unroll 1
      for (int w = 1; w < kLpWarps; ++w) run_merge(r, sh.run[w], k), top = fmaxf(top, sh.max[w]);
      // from here on against the row's (or part's) largest logit
      if (top > -kInfF) {
        const float d = (r.m - top) * k;
        const float e = ex2_fast(d);
        r = Run{top, e * r.s, e * fmaf(r.s, d, r.w)};
      }
      sh.run[0] = r;
    }
    if (!whole) {
      const int64_t at = static_cast<int64_t>(blockIdx.x) * 2 + (lo == 0 ? 1 : 0);
      for (int j = t; j < p.top_k; j += kLpThreads) p.part_top[at * p.top_k + j] = sh.top[j];
      if (t == 0) {
        p.part[at] = r;
        p.part_flags[at] = sh.flags;
      }
      const int c0 = static_cast<int>(((row0 + 1) * g - 1) / total), c1 = static_cast<int>(((row0 + per_row) * g - 1) / total);
      __threadfence();  // each thread's own writes, before the barrier that lets thread 0 take the ticket for all
      __syncthreads();
      if (t == 0) {
        sh.last = ticket_add(&p.tickets[c0], 1u) == static_cast<unsigned>(c1 - c0) ? 1u : 0u;
        if (sh.last) p.tickets[c0] = 0u;
      }
      __syncthreads();
      if (!sh.last) continue;
      join_parts(p, sh, c0, c1, k);
    }
    __syncthreads();
    write_outputs<BF16>(p, sh, i, row, T);
    __syncthreads();
  }
}

struct LogprobWs {
  size_t part, flags, top, total;
};

// The same offsets whatever the number of rows, so that the tickets of one call never lie where another wrote its parts.
LogprobWs logprob_ws(int32_t top_k) {
  LogprobWs L{};
  size_t off = sizeof(uint32_t) * kMaxBlocks;
  L.part = off;
  off = align_up(off + sizeof(Run) * 2 * kMaxBlocks, 256);
  L.flags = off;
  off = align_up(off + sizeof(uint32_t) * 2 * kMaxBlocks, 256);
  L.top = off;
  off = align_up(off + sizeof(uint64_t) * 2 * kMaxBlocks * static_cast<size_t>(top_k > 0 ? top_k : 0), 256);
  L.total = off;
  return L;
}

// Resident blocks of a multiprocessor, once for each device.
template <bool BF16>
cudaError_t logprob_blocks(int* n) {
  static std::mutex mu;
  static int have[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (have[dev] == 0) {
    int fit = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, k_token_logprobs<BF16>, kLpThreads, 0);
    if (e != cudaSuccess) return e;
    have[dev] = fit < 1 ? 1 : fit;
  }
  *n = have[dev];
  return cudaSuccess;
}

// ---------------------------------------------------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------------------------------------------------

struct LogprobBwdParams {
  LogitsView lg;
  const int32_t* ids;
  int32_t num_ids;
  int64_t ldi;
  const float* row_temp;
  const float* row_max;
  const float* log_z;
  const float* entropy;
  const int32_t* top_ids;
  int32_t top_k;
  const float* g_logprob;
  const float* g_entropy;
  const float* g_top;
  void* dlogits;
  int64_t ldd;
  int32_t splits;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Blocks take a part of a row each; about 32 a multiprocessor (six of them resident), so that the ends of some lie under
// the streams of others.
constexpr int kBwdThreads = 256;

template <bool BF16>
__global__ void __launch_bounds__(kBwdThreads, 6) k_token_logprobs_bwd(LogprobBwdParams p) {
  constexpr int N = Vec<BF16>::N;
  constexpr int U = 4;
  __shared__ int32_t s_id[kMaxGiven + kMaxTop];  // -1: no part in the gradient
  __shared__ float s_g[kMaxGiven + kMaxTop];
  __shared__ float s_sum[(kBwdThreads / 32)];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t row = blockIdx.x / p.splits;
  const int split = static_cast<int>(blockIdx.x - row * p.splits);
  grid_dependency_wait();
  allow_dependents();
  const float M = p.row_max[row], lz = p.log_z[row];
  const bool empty = !(M > -kInfF);
  const float T = logprob_temperature(p.row_temp, row);
  const float k = logprob_k(T), invT = __frcp_rn(T);
  const int given = p.num_ids + p.top_k;
  float G = 0.0f;
  for (int j = t; j < given; j += kBwdThreads) {
    const bool top = j >= p.num_ids;
    int32_t id = top ? p.top_ids[row * p.top_k + j - p.num_ids] : p.ids[row * p.ldi + j];
    const float g = top ? p.g_top[row * p.top_k + j - p.num_ids] : p.g_logprob[row * p.num_ids + j];
    if (id < 0 || id >= p.lg.vocab || empty || !usable_logit(logit_at<BF16>(p.lg, row, id))) id = -1;
    s_id[j] = id;
    s_g[j] = g;
    if (id >= 0) G += g;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) G += __shfl_xor_sync(0xffffffffu, G, off);
  if (lane == 0) s_sum[warp] = G;
  __syncthreads();
  G = 0.0f;
#pragma unroll
  for (int w = 0; w < (kBwdThreads / 32); ++w) G += s_sum[w];

  const float gH = p.g_entropy ? p.g_entropy[row] : 0.0f;
  // Exponents are held kLift higher, and the factors 2^kLift lower: a probability under 2^-126, where the exponential is
  // flushed to 0, may still have a factor of some thousands (1/T, its logarithm and the entropy).
  constexpr float kLift = 16.0f, kLower = 0x1p-16f;
  const float B = -gH * kLn2 * invT;
  const float A = fmaf(-kLift, B, -(G + (p.g_entropy ? gH * p.entropy[row] : 0.0f)) * invT) * kLower;
  const float Bl = B * kLower;
  const float lz2 = fmaf(lz, 1.44269504088896340736f, -kLift);
  // p (A + B t) for one logit; 0 for one that is not a usable, finite logit
  auto grad = [&](float l) {
    const float d = (l - M) * k - lz2;
    const float x = fmaxf(d, -200.0f);  // 2^-200 is 0 in fp32, and keeps 0 * t from becoming NaN
    const float y = ex2_fast(x) * fmaf(Bl, x, A);
    return (usable_logit(l) && !empty) ? y : 0.0f;
  };
  const int nvec = p.lg.vocab / N;
  const int lo = static_cast<int>(static_cast<int64_t>(nvec) * split / p.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(nvec) * (split + 1) / p.splits);
  const uint4* vec = reinterpret_cast<const uint4*>(static_cast<const char*>(p.lg.base) + row * p.lg.ld * (BF16 ? 2 : 4));
  char* out = static_cast<char*>(p.dlogits) + row * p.ldd * (BF16 ? 2 : 4);
  uint4* ovec = reinterpret_cast<uint4*>(out);
  for (int v = lo + t; v < hi; v += kBwdThreads * U) {
    uint4 u[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (v + j * kBwdThreads < hi) u[j] = ld_stream16(vec + v + j * kBwdThreads);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (v + j * kBwdThreads < hi) {
        float f[N];
        Vec<BF16>::unpack(u[j], f);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = grad(f[e]);
        uint4 o;
        if (BF16)
          o = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[N - 4], f[N - 3]),
                         pack_bf16(f[N - 2], f[N - 1]));
        else
          o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        __stcs(ovec + v + j * kBwdThreads, o);
      }
  }
  auto store = [&](int64_t col, float x) {
    if (BF16)
      reinterpret_cast<unsigned short*>(out)[col] = static_cast<unsigned short>(pack_bf16(x, 0.0f) & 0xffffu);
    else
      reinterpret_cast<float*>(out)[col] = x;
  };
  const bool last = split == p.splits - 1;
  const int c0 = lo * N, c1 = last ? p.lg.vocab : hi * N;
  if (last && nvec * N + t < p.lg.vocab) store(nvec * N + t, grad(logit_at<BF16>(p.lg, row, nvec * N + t)));
  __syncthreads();
  // The given tokens of this part: written over, whole, and rounded once.
  for (int j = t; j < given; j += kBwdThreads) {
    const int32_t id = s_id[j];
    if (id < c0 || id >= c1) continue;
    float g = 0.0f;
    bool first = true;
    for (int x = 0; x < given; ++x)
      if (s_id[x] == id) {
        if (x < j) first = false;
        g += s_g[x];
      }
    if (first) store(id, fmaf(g, invT, grad(logit_at<BF16>(p.lg, row, id))));
  }
}

sv_status_t check_rows(const void* logits, sv_dtype_t dt, int64_t ld, int64_t rows, int32_t vocab) {
  if (!logits) return SV_ERR_NULL_ARG;
  if (dt != SV_F32 && dt != SV_BF16) return SV_ERR_BAD_DTYPE;
  if (vocab < 1 || rows < 0 || rows > INT32_MAX || ld < vocab) return SV_ERR_BAD_SHAPE;
  const int64_t es = dt == SV_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(logits) & 15) != 0 || (ld * es) % 16 != 0) return SV_ERR_MISALIGNED;
  return SV_OK;
}

// Blocks a row's gradient is split over: enough that about `want` blocks run, each with at least 1024 vectors.
int32_t row_splits(int64_t n, int32_t vocab, bool bf16, int32_t want) {
  const int64_t nvec = vocab / (bf16 ? 8 : 4);
  int64_t s = (want + n - 1) / n;
  if (s > nvec / 1024) s = nvec / 1024;
  if (s > 32) s = 32;
  return static_cast<int32_t>(s < 1 ? 1 : s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_verify_logprobs_workspace_bytes(int64_t /*n*/, int32_t /*vocab*/, int32_t top_k) {
  return logprob_ws(top_k).total;
}

sv_status_t spec_verify_token_logprobs(const void* logits, sv_dtype_t dtype, int64_t ld, int64_t rows, int32_t vocab,
                                       int64_t n, const int32_t* row_index, const int32_t* ids, int32_t num_ids,
                                       int64_t ldi, const float* row_temp, int32_t top_k, float* logprob,
                                       float* entropy, float* row_max, float* log_z, int32_t* top_ids,
                                       float* top_logprob, uint32_t* flags, void* ws, size_t ws_bytes,
                                       cudaStream_t stream) {
  if (n == 0 && rows >= 0) return SV_OK;  // an empty batch has no arrays to check
  const sv_status_t c = check_rows(logits, dtype, ld, rows, vocab);
  if (c != SV_OK) return c;
  if (n < 0 || n > INT32_MAX || (!row_index && n > rows)) return SV_ERR_BAD_SHAPE;
  if (num_ids < 0 || num_ids > kMaxGiven || top_k < 0 || top_k > kMaxTop || ldi < num_ids) return SV_ERR_BAD_SHAPE;
  if (num_ids > 0 && (!ids || !logprob)) return SV_ERR_NULL_ARG;
  if (top_k > 0 && (!top_ids || !top_logprob)) return SV_ERR_NULL_ARG;
  const LogprobWs L = logprob_ws(top_k);
  if (!ws || ws_bytes < L.total || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return SV_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  char* base = static_cast<char*>(ws);
  const bool bf16 = dtype == SV_BF16;
  int per_sm = 1;
  e = bf16 ? logprob_blocks<true>(&per_sm) : logprob_blocks<false>(&per_sm);
  if (e != cudaSuccess) return cuda_failure(e);
  // one resident wave, less where the rows are not worth it
  const int64_t vectors = n * (vocab / (bf16 ? 8 : 4));
  int64_t blocks = static_cast<int64_t>(dev.sms) * per_sm;
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  // ... and no more parts of a row than the join of the top alternatives holds
  int64_t least = kMinVectors;
  if (top_k > 0) {
    const int64_t parts = kCandCap / top_k - 2, nvec = vocab / (bf16 ? 8 : 4);
    if (least < (nvec + parts - 1) / parts) least = (nvec + parts - 1) / parts;
  }
  if (blocks > vectors / least) blocks = vectors / least;
  if (blocks < 1) blocks = 1;
  const LogprobParams p{LogitsView{logits, dtype, ld, rows, vocab},
                        n, row_index, ids, num_ids, ldi, row_temp, top_k, logprob, entropy, row_max, log_z, top_ids,
                        top_logprob, flags, reinterpret_cast<uint32_t*>(base), reinterpret_cast<Run*>(base + L.part),
                        reinterpret_cast<uint32_t*>(base + L.flags), reinterpret_cast<uint64_t*>(base + L.top), least};
  const dim3 grid(static_cast<unsigned>(blocks));
  e = bf16 ? launch_pdl(k_token_logprobs<true>, grid, dim3(kLpThreads), 0, stream, p)
           : launch_pdl(k_token_logprobs<false>, grid, dim3(kLpThreads), 0, stream, p);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

sv_status_t spec_verify_token_logprobs_backward(const void* logits, sv_dtype_t dtype, int64_t ld, int64_t rows,
                                                int32_t vocab, const int32_t* ids, int32_t num_ids, int64_t ldi,
                                                const float* row_temp, const float* row_max, const float* log_z,
                                                const float* entropy, const int32_t* top_ids, int32_t top_k,
                                                const float* g_logprob, const float* g_entropy, const float* g_top,
                                                void* dlogits, int64_t ldd, cudaStream_t stream) {
  if (rows == 0) return SV_OK;  // an empty batch has no arrays to check
  sv_status_t c = check_rows(logits, dtype, ld, rows, vocab);
  if (c != SV_OK) return c;
  c = check_rows(dlogits, dtype, ldd, rows, vocab);
  if (c != SV_OK) return c;
  if (num_ids < 0 || num_ids > kMaxGiven || top_k < 0 || top_k > kMaxTop || ldi < num_ids ||
      rows > INT32_MAX / 32)
    return SV_ERR_BAD_SHAPE;
  if (!row_max || !log_z) return SV_ERR_NULL_ARG;
  if (num_ids > 0 && (!ids || !g_logprob)) return SV_ERR_NULL_ARG;
  if (top_k > 0 && (!top_ids || !g_top)) return SV_ERR_NULL_ARG;
  if (g_entropy && !entropy) return SV_ERR_NULL_ARG;
  const bool bf16 = dtype == SV_BF16;
  const uintptr_t a = reinterpret_cast<uintptr_t>(logits), d = reinterpret_cast<uintptr_t>(dlogits);
  const uintptr_t es = bf16 ? 2 : 4;
  const uintptr_t an = (static_cast<uintptr_t>(rows - 1) * ld + vocab) * es;
  const uintptr_t dn = (static_cast<uintptr_t>(rows - 1) * ldd + vocab) * es;
  if (a < d + dn && d < a + an) return SV_ERR_UNSUPPORTED;  // blocks read each other's logits
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  const LogprobBwdParams p{LogitsView{logits, dtype, ld, rows, vocab},
                           ids, num_ids, ldi, row_temp, row_max, log_z, entropy, top_ids, top_k, g_logprob,
                           g_entropy, g_top, dlogits, ldd, row_splits(rows, vocab, bf16, 32 * dev.sms)};
  const dim3 grid(static_cast<unsigned>(rows * p.splits));
  e = bf16 ? launch_pdl(k_token_logprobs_bwd<true>, grid, dim3(kBwdThreads), 0, stream, p)
           : launch_pdl(k_token_logprobs_bwd<false>, grid, dim3(kBwdThreads), 0, stream, p);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

}  // extern "C"
