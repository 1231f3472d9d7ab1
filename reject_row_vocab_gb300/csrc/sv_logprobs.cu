// Log probabilities of given tokens, with entropy and top alternatives, and
// their gradient by the logits ([E2D] §6.2: the target is softmax(l / T)).
//
// Forward, k_token_logprobs.  With k = log2(e) / T and M the row maximum,
//   Z = sum 2^((l - M) k),  W = sum (l - M) 2^((l - M) k)
//   logprob(id) = (l_id - M) / T - ln Z,   H = ln Z - (W / Z) / T.
// One pass: each thread keeps a running (m, s, w) of the elements it has read
// and rescales it when its maximum grows; a block joins its threads' triples,
// and the last block of a row joins the blocks' in block order, so results do
// not depend on the order the blocks finish in.
//
// Top alternatives from the same pass: a thread's running maximum is the
// largest of its own elements, so the top_k-th largest of the block's thread
// maxima is a lower bound on the block's top_k-th element.  Only threads whose
// maximum reaches the bound (about top_k of 256) can hold a top element, and
// only their elements are looked at again (from L2), by whole warps.  Elements
// are ordered by a 64-bit key - value, then the lower index - so the selection
// is unique whatever the order of the candidates.
//
// Backward, k_token_logprobs_bwd.  With t = (l - M) k - log2 Z and p = 2^t,
//   dl = p (A + B t) + (the row's given tokens)/T,
//   A = -(G + gH H)/T,  B = -gH ln 2 / T:
// two multiply-adds and an exponential an element between a read and a write.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cfloat>
#include <cstdint>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 64;
constexpr int kMaxGiven = 1024;
constexpr int kMaxSplits = 32;
constexpr int kMaxSplitRows = 1024;           // rows are split only below this many (see row_splits)
constexpr int kMaxParts = 2 * kMaxSplitRows;  // parts of a call with split rows
constexpr int kCandCap = 1024;  // candidates a block sorts in shared memory
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

// Running sums of a thread, block or row: s = sum 2^((l - m) k), w = sum (l - m) 2^((l - m) k).
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
  const float da = a.m - M, db = b.m - M;
  const float ea = ex2_fast(da * k), eb = ex2_fast(db * k);
  // a term that vanished has sums that vanish with it (0 * a large distance is 0, not a stray product)
  a.w = (ea > 0.0f ? ea * (a.w + a.s * da) : 0.0f) + (eb > 0.0f ? eb * (b.w + b.s * db) : 0.0f);
  a.s = ea * a.s + eb * b.s;
  a.m = M;
}

// log2(e) / T; the unscaled distribution for a greedy temperature.  Held at 1e-30 at least: below that every finite
// logit of ordinary size has the same weight, and a masked entry's distance still has to end in a weight of zero.
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
  int32_t splits;
  uint32_t* tickets;  // [n], zero between calls
  Run* part;          // [n, splits]
  uint32_t* part_flags;
  uint64_t* part_top;  // [n, splits, top_k]
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

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads) k_token_logprobs(LogprobParams p) {
  constexpr int N = Vec<BF16>::N;
  constexpr int U = 4;  // vectors in flight a thread
  __shared__ Run s_run[kLpWarps];
  __shared__ uint32_t s_flags, s_count, s_last;
  __shared__ uint64_t s_cand[kCandCap];
  __shared__ uint64_t s_top[kMaxTop];
  __shared__ uint64_t s_key[kLpWarps];
  __shared__ uint16_t s_who[kLpThreads];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t i = blockIdx.x / p.splits;
  const int split = static_cast<int>(blockIdx.x - i * p.splits);
  grid_dependency_wait();
  allow_dependents();
  int64_t row = p.row_index ? p.row_index[i] : i;
  if (row < 0 || row >= p.lg.rows) {  // padding
    if (split != 0) return;
    for (int j = t; j < p.num_ids; j += kLpThreads) p.logprob[i * p.num_ids + j] = 0.0f;
    for (int j = t; j < p.top_k; j += kLpThreads) {
      p.top_ids[i * p.top_k + j] = -1;
      p.top_logprob[i * p.top_k + j] = -kInfF;
    }
    if (t == 0) {
      if (p.entropy) p.entropy[i] = 0.0f;
      if (p.row_max) p.row_max[i] = -kInfF;
      if (p.log_z) p.log_z[i] = 0.0f;
      if (p.flags) p.flags[i] = row == -1 ? 0u : kStBadLayout;
    }
    return;
  }
  const float T = logprob_temperature(p.row_temp, i);
  const float k = logprob_k(T);
  const int nvec = p.lg.vocab / N;
  const int lo = static_cast<int>(static_cast<int64_t>(nvec) * split / p.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(nvec) * (split + 1) / p.splits);
  const char* base = static_cast<const char*>(p.lg.base) + row * p.lg.ld * (BF16 ? 2 : 4);
  const uint4* vec = reinterpret_cast<const uint4*>(base);
  const int tail0 = nvec * N;  // the ragged end belongs to the last block of the row
  const int tails = split == p.splits - 1 ? p.lg.vocab - tail0 : 0;

  if (t == 0) s_flags = 0u, s_count = 0u;
  __syncthreads();
  Run r{-kInfF, 0.0f, 0.0f};
  uint32_t flags = 0u;
  for (int v = lo + t; v < hi; v += kLpThreads * U) {
    uint4 u[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int x = v + j * kLpThreads;
      // beyond the part: all -inf (bf16 pairs 0xff80, fp32 0xff800000)
      u[j] = x < hi ? ld_stream16(vec + x)
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
    if (!(vm <= r.m)) {
      if (!usable_logit(vm)) {  // a NaN or +inf among them: element by element
#pragma unroll
        for (int j = 0; j < U; ++j) {
          float f[N];
          Vec<BF16>::unpack(u[j], f);
#pragma unroll
          for (int e = 0; e < N; ++e) run_add(r, f[e], k, flags);
        }
        continue;
      }
      run_merge(r, Run{vm, 0.0f, 0.0f}, k);  // the new reference
    }
    if (r.m > -kInfF) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        float f[N];
        Vec<BF16>::unpack(u[j], f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float d = fmaxf(f[e] - r.m, -FLT_MAX);  // -inf entries: weight 0, and 0 * d = 0
          const float x = ex2_fast(d * k);
          r.s += x;
          r.w = fmaf(x, d, r.w);
        }
      }
    }
  }
  if (t < tails) run_add(r, logit_at<BF16>(p.lg, row, tail0 + t), k, flags);

  // Top alternatives of the part.
  if (p.top_k > 0) {
    const uint32_t mine = ordered(r.m) >> 16;
    uint32_t thr = 0u;  // the largest 16-bit bound that top_k threads' maxima reach
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t cand = thr | (1u << bit);
      if (__syncthreads_count(mine >= cand) >= p.top_k) thr = cand;
    }
    const uint32_t bound = max(thr, 1u);  // 0 stands for no element
    if (mine >= bound) s_who[atomicAdd(&s_count, 1u)] = static_cast<uint16_t>(t);
    __syncthreads();
    const int who = static_cast<int>(s_count);
    __syncthreads();
    if (t == 0) s_count = 0u;
    __syncthreads();
    for (int c = warp; c < who; c += kLpWarps) {
      const int owner = s_who[c];
      for (int x = lo + owner + lane * kLpThreads; x < hi; x += 32 * kLpThreads) {
        float f[N];
        Vec<BF16>::unpack(ld_stream16(vec + x), f);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if ((ordered(f[e]) >> 16) >= bound) {
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < kCandCap) s_cand[at] = top_key(f[e], x * N + e);
          }
      }
      if (owner < tails && lane == 0) {
        const float f = logit_at<BF16>(p.lg, row, tail0 + owner);
        if ((ordered(f) >> 16) >= bound) {
          const uint32_t at = atomicAdd(&s_count, 1u);
          if (at < kCandCap) s_cand[at] = top_key(f, tail0 + owner);
        }
      }
    }
    __syncthreads();
    const uint32_t found = s_count;
    if (found <= kCandCap) {
      rank_top(s_cand, static_cast<int>(found), p.top_k, s_top);
    } else {
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
        if (lane == 0) s_key[warp] = best;
        __syncthreads();
        best = 0ull;
        for (int w = 0; w < kLpWarps; ++w) best = max(best, s_key[w]);
        if (t == 0) s_top[j] = best;
        last = best == 0ull ? 1ull : best;  // nothing left: no key is below 1
        __syncthreads();
      }
    }
  }

  // Join the threads' sums.
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    Run o{__shfl_xor_sync(0xffffffffu, r.m, off), __shfl_xor_sync(0xffffffffu, r.s, off),
          __shfl_xor_sync(0xffffffffu, r.w, off)};
    // both sides of an exchange join in the same order, lower lane first
    if (lane & off) {
      const Run mine = r;
      r = o;
      o = mine;
    }
    run_merge(r, o, k);
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0) {
    s_run[warp] = r;
    if (flags) atomicOr(&s_flags, flags);
  }
  __syncthreads();
  if (t == 0) {
    r = s_run[0];
    for (int w = 1; w < kLpWarps; ++w) run_merge(r, s_run[w], k);
    s_run[0] = r;
  }

  if (p.splits > 1) {
    const int64_t at = i * p.splits + split;
    for (int j = t; j < p.top_k; j += kLpThreads) p.part_top[at * p.top_k + j] = s_top[j];
    if (t == 0) {
      p.part[at] = r;
      p.part_flags[at] = s_flags;
    }
    __threadfence();  // each thread's own writes, before the barrier that lets thread 0 take the ticket for all
    __syncthreads();
    if (t == 0) s_last = ticket_add(&p.tickets[i], 1u) == static_cast<unsigned>(p.splits - 1) ? 1u : 0u;
    __syncthreads();
    if (!s_last) return;
    // The last block of the row joins the parts in order.
    if (t == 0) {
      p.tickets[i] = 0u;
      r = Run{-kInfF, 0.0f, 0.0f};
      uint32_t f = 0u;
      for (int s = 0; s < p.splits; ++s) {
        const Run* q = p.part + i * p.splits + s;
        run_merge(r, Run{__ldcg(&q->m), __ldcg(&q->s), __ldcg(&q->w)}, k);
        f |= __ldcg(&p.part_flags[i * p.splits + s]);
      }
      s_run[0] = r;
      s_flags = f;
      s_count = 0u;
    }
    if (p.top_k > 0) {
      // A part's last key is a lower bound on the row's top_k-th: the largest of them leaves about top_k keys.
      const uint64_t* keys = p.part_top + i * p.splits * p.top_k;
      if (warp == 0) {
        uint64_t b = lane < p.splits ? __ldcg(&keys[lane * p.top_k + p.top_k - 1]) : 0ull;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, off));
        if (lane == 0) s_key[0] = b;
      }
      __syncthreads();
      const uint64_t bound = s_key[0];
      for (int x = t; x < p.splits * p.top_k; x += kLpThreads) {
        const uint64_t key = __ldcg(&keys[x]);
        if (key != 0ull && key >= bound) {
          const uint32_t at = atomicAdd(&s_count, 1u);
          if (at < kCandCap) s_cand[at] = key;
        }
      }
      __syncthreads();
      rank_top(s_cand, min(static_cast<int>(s_count), kCandCap), p.top_k, s_top);
    }
  }
  __syncthreads();

  // Outputs of the row.
  r = s_run[0];
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
    const uint64_t key = s_top[j];
    p.top_ids[i * p.top_k + j] = key ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    p.top_logprob[i * p.top_k + j] =
        key ? __fdiv_rn(from_ordered(static_cast<uint32_t>(key >> 32)) - r.m, T) - lz : -kInfF;
  }
  const int outside = __syncthreads_or(range ? 1 : 0);
  if (t == 0) {
    // the entropy of a distribution is not negative; rounding may leave a value just below 0
    if (p.entropy) p.entropy[i] = empty ? 0.0f : fmaxf(lz - __fdiv_rn(__fdiv_rn(r.w, r.s), T), 0.0f);
    if (p.row_max) p.row_max[i] = r.m;
    if (p.log_z) p.log_z[i] = lz;
    if (p.flags) p.flags[i] = s_flags | (outside ? kStTokenRange : 0u) | (empty ? kStNonFinite : 0u);
  }
}

struct LogprobWs {
  size_t tickets, part, flags, top, total;
};

// The same offsets whatever the number of rows, so that the tickets of one call never lie where another wrote its parts.
LogprobWs logprob_ws(int32_t top_k) {
  LogprobWs L{};
  size_t off = sizeof(uint32_t) * kMaxSplitRows;
  L.part = off;
  off = align_up(off + sizeof(Run) * kMaxParts, 256);
  L.flags = off;
  off = align_up(off + sizeof(uint32_t) * kMaxParts, 256);
  L.top = off;
  off = align_up(off + sizeof(uint64_t) * kMaxParts * static_cast<size_t>(top_k > 0 ? top_k : 0), 256);
  L.total = off;
  return L;
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

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads) k_token_logprobs_bwd(LogprobBwdParams p) {
  constexpr int N = Vec<BF16>::N;
  constexpr int U = 4;
  __shared__ int32_t s_id[kMaxGiven + kMaxTop];  // -1: no part in the gradient
  __shared__ float s_g[kMaxGiven + kMaxTop];
  __shared__ float s_sum[kLpWarps];
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
  for (int j = t; j < given; j += kLpThreads) {
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
  for (int w = 0; w < kLpWarps; ++w) G += s_sum[w];

  const float gH = p.g_entropy ? p.g_entropy[row] : 0.0f;
  const float A = -(G + (p.g_entropy ? gH * p.entropy[row] : 0.0f)) * invT;
  const float B = -gH * kLn2 * invT;
  const float lz2 = lz * 1.44269504088896340736f;
  // p (A + B t) for one logit; 0 for one that is not a usable, finite logit
  auto grad = [&](float l) {
    const float d = (l - M) * k - lz2;
    const float x = fmaxf(d, -200.0f);  // 2^-200 is 0 in fp32, and keeps 0 * t from becoming NaN
    const float y = ex2_fast(x) * fmaf(B, x, A);
    return (usable_logit(l) && !empty) ? y : 0.0f;
  };
  const int nvec = p.lg.vocab / N;
  const int lo = static_cast<int>(static_cast<int64_t>(nvec) * split / p.splits);
  const int hi = static_cast<int>(static_cast<int64_t>(nvec) * (split + 1) / p.splits);
  const uint4* vec = reinterpret_cast<const uint4*>(static_cast<const char*>(p.lg.base) + row * p.lg.ld * (BF16 ? 2 : 4));
  char* out = static_cast<char*>(p.dlogits) + row * p.ldd * (BF16 ? 2 : 4);
  uint4* ovec = reinterpret_cast<uint4*>(out);
  for (int v = lo + t; v < hi; v += kLpThreads * U) {
    uint4 u[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (v + j * kLpThreads < hi) u[j] = ld_stream16(vec + v + j * kLpThreads);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (v + j * kLpThreads < hi) {
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
        __stcs(ovec + v + j * kLpThreads, o);
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
  for (int j = t; j < given; j += kLpThreads) {
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

// Blocks a row is split over: enough that about `want` blocks run, each with at least 1024 vectors, and no more parts
// than the join of the top alternatives holds.
int32_t row_splits(int64_t n, int32_t vocab, bool bf16, int32_t want, int32_t top_k) {
  if (want > kMaxSplitRows) want = kMaxSplitRows;
  const int64_t nvec = vocab / (bf16 ? 8 : 4);
  int64_t s = (want + n - 1) / n;
  if (s > nvec / 1024) s = nvec / 1024;
  if (s > kMaxSplits) s = kMaxSplits;
  if (top_k > 0 && s > kCandCap / top_k) s = kCandCap / top_k;
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
  if (n < 0 || n > INT32_MAX / kMaxSplits || (!row_index && n > rows)) return SV_ERR_BAD_SHAPE;
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
  LogprobParams p{LogitsView{logits, dtype, ld, rows, vocab},
                  n, row_index, ids, num_ids, ldi, row_temp, top_k, logprob, entropy, row_max, log_z, top_ids,
                  top_logprob, flags, row_splits(n, vocab, bf16, 4 * dev.sms, top_k),
                  reinterpret_cast<uint32_t*>(base + L.tickets), reinterpret_cast<Run*>(base + L.part),
                  reinterpret_cast<uint32_t*>(base + L.flags), reinterpret_cast<uint64_t*>(base + L.top)};
  const dim3 grid(static_cast<unsigned>(n * p.splits));
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
      rows > INT32_MAX / kMaxSplits)
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
                           g_entropy, g_top, dlogits, ldd, row_splits(rows, vocab, bf16, 4 * dev.sms, 0)};
  const dim3 grid(static_cast<unsigned>(rows * p.splits));
  e = bf16 ? launch_pdl(k_token_logprobs_bwd<true>, grid, dim3(kLpThreads), 0, stream, p)
           : launch_pdl(k_token_logprobs_bwd<false>, grid, dim3(kLpThreads), 0, stream, p);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

}  // extern "C"
