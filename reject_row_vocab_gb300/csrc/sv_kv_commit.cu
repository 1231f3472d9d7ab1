// The KV move of a verification's commit lists ([E2D] §5.6.6, §8.1): K and V
// of every committed entry, from its slot to its position, in every layer.
//
//   cache[l][dst(e)] <- cache[l][src(e)]   for e in [commit_cu[b], commit_cu[b+1])
//
// Bound by the bytes: each moved row is read once and written once.  The rows
// of one request may overlap (drafts staged in place move towards the front),
// so a block owns whole columns of one request's rows: it reads the 16-byte
// column pieces of all its entries into registers, meets, and only then writes
// them.  Columns, layers, and K and V are independent of one another, so a
// block finds its entries' places once and takes several layers in turn,
// reading one ahead: a block for each layer spent most of its time on the
// chain of loads that leads to the places (64 requests, 32 layers: 31 us).
//
// Measured: 384 rows of 2 KB of K and of V in 32 layers, 64 requests: 25 us, 4.0
// TB/s read and written (256 requests: 83 us, 4.8); 28 layers of one request: 6.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>

#include "sv_kv.cuh"

namespace sv {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveBlocks = 8;  // blocks for each multiprocessor that a large call is given

// REGS: 16-byte pieces of a layer that a thread holds between the reads and the writes.  Two leave room for eight blocks on
// a multiprocessor (64 requests, 32 layers: 25 us, with four 28, with eight 47); lists of over 512 entries need four.
template <int REGS>
__global__ void __launch_bounds__(kMoveThreads) k_kv_commit(KvView c, int32_t max_len, int64_t list_len,
                                                            const int32_t* cu, const int64_t* src_slot,
                                                            const int64_t* dst_pos, uint32_t* status, int per_block) {
  __shared__ int64_t s_src[kMaxNodes], s_dst[kMaxNodes];  // element offsets, -1 for an entry that is not moved
  __shared__ uint32_t s_status;
  const int b = blockIdx.x, t = threadIdx.x;
  // this block's caches: K and V of a layer are two
  const int first = blockIdx.y * per_block, last = min(first + per_block, 2 * c.layers);
  grid_dependency_wait();
  allow_dependents();
  if (t == 0) s_status = 0u;
  __syncthreads();
  const int64_t lo = cu[b];
  const int64_t n64 = static_cast<int64_t>(cu[b + 1]) - lo;
  const bool bad = lo < 0 || n64 < 0 || n64 > max_len || lo + n64 > list_len;
  const int n = bad ? 0 : static_cast<int>(n64);
  for (int e = t; e < n; e += kMoveThreads) {
    const int64_t pos = dst_pos[lo + e];
    const int64_t src = kv_slot_offset(c, src_slot[lo + e]);
    int64_t dst = -1;
    if (pos >= 0 && pos < static_cast<int64_t>(c.max_pages) * c.page_size) {
      const uint32_t p = divide(static_cast<uint32_t>(pos), c.div_mul, c.div_shift);
      dst = kv_page_offset(c, c.table[b * c.ld_table + p], static_cast<uint32_t>(pos) - p * c.page_size);
    }
    const bool ok = src >= 0 && dst >= 0;
    if (!ok) atomicOr(&s_status, kStSlotRange);
    s_src[e] = ok ? src : -1;
    s_dst[e] = ok && src != dst ? dst : -1;  // an entry already in place is not moved
  }
  __syncthreads();
  if (blockIdx.y == 0 && t == 0 && status) status[b] = bad ? kStBadLayout : s_status;
  if (n == 0) return;
  const int per_head = c.head_dim * c.es / 16;
  const int cols = c.heads * per_head;  // 16-byte pieces of one row
  // As many columns at a time as fit the registers of the block (one at least).
  const int width = min(cols, kMoveThreads * REGS / n);
  for (int c0 = 0; c0 < cols; c0 += width) {
    const int w = min(width, cols - c0);
    int64_t src[REGS], dst[REGS];  // bytes; dst -1: nothing to move
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      const int x = t + i * kMoveThreads;
      src[i] = 0, dst[i] = -1;
      if (x < w * n) {
        const int e = x / w, col = c0 + x - e * w, head = col / per_head;
        const int64_t at = head * c.head_stride * c.es + (col - head * per_head) * 16;
        src[i] = s_src[e] * c.es + at;
        if (s_dst[e] >= 0) dst[i] = s_dst[e] * c.es + at;
      }
    }
    auto cache = [&](int q) { return (q & 1 ? c.v : c.k) + (q >> 1) * c.layer_stride * c.es; };
    uint4 r[REGS], ahead[REGS];
    auto read = [&](int q, uint4 (&to)[REGS]) {
#pragma unroll
      for (int i = 0; i < REGS; ++i)
        if (dst[i] >= 0) to[i] = *reinterpret_cast<const uint4*>(cache(q) + src[i]);
    };
    read(first, r);
    for (int q = first; q < last; ++q) {
      if (q + 1 < last) read(q + 1, ahead);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < REGS; ++i) {
        if (dst[i] >= 0) *reinterpret_cast<uint4*>(cache(q) + dst[i]) = r[i];
        r[i] = ahead[i];
      }
    }
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status_t spec_verify_kv_commit(const sv_kv_cache_t* cache, int32_t batch, int32_t max_len,
                                             int64_t list_len, const int32_t* commit_cu,
                                             const int64_t* commit_src_slot, const int64_t* commit_dst_pos,
                                             uint32_t* dev_status, cudaStream_t stream) {
  if (batch < 0 || batch > 65535 || max_len < 1 || max_len > kMaxNodes || list_len < 0) return SV_ERR_BAD_SHAPE;
  KvView c{};
  const sv_status_t s = check_cache(cache, &c);
  if (s != SV_OK) return s;
  if (c.layers > 32767) return SV_ERR_BAD_SHAPE;
  if (batch == 0) return SV_OK;
  if (!commit_cu || (list_len > 0 && (!commit_src_slot || !commit_dst_pos))) return SV_ERR_NULL_ARG;
  if (!entries_apart(c)) return SV_ERR_UNSUPPORTED;  // a block would read what another has already moved
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  // caches a block takes: a few blocks for each multiprocessor are enough, a small call has one for each cache
  const int64_t caches = 2 * static_cast<int64_t>(c.layers);
  int64_t per = batch * caches / (kMoveBlocks * dev.sms);
  per = per < 1 ? 1 : per > caches ? caches : per;
  const dim3 grid(static_cast<unsigned>(batch), static_cast<unsigned>((caches + per - 1) / per));
  static_assert(kMoveThreads * 4 >= kMaxNodes, "a column of the longest list");
  e = launch_pdl(max_len <= 2 * kMoveThreads ? k_kv_commit<2> : k_kv_commit<4>, grid, dim3(kMoveThreads), 0, stream, c,
                 max_len, list_len, commit_cu, commit_src_slot, commit_dst_pos, dev_status, static_cast<int>(per));
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}
