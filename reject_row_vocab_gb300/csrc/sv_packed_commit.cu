// The KV move of a verification's commit lists ([E2D] §5.6.6, §8.1) in the
// 4-bit cache: an entry's codes and scales, of K and of V, from its slot to
// its position, in every layer.
//
// As in the cache of whole numbers a request's sources and destinations may
// overlap, so a block owns pieces of all its entries: it reads them into
// registers, meets, and only then writes.  A piece is 16 bytes of codes, or as
// much of an entry's scales of a head as its alignment allows (8 bytes of heads of
// 128).  Places are found once for the layers that a block goes through.
//
// Bound by the chain lists, places, rows, and by pieces of 64 and 8 bytes: 384 rows of
// 64 requests in 32 layers, 8 heads of 128, take 16.8 us (28 MB there and back; with
// the sectors that the pieces touch it is 57), the block's barrier for each layer among
// them.  Blocks of 512 threads and a quarter of the blocks take 21.5 us.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>

#include "sv_rows.cuh"

namespace sv {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveBlocks = 8;  // blocks for each multiprocessor that a large call is given

template <int REGS>
__global__ void __launch_bounds__(kMoveThreads) k_packed_commit(PackedView c, int32_t max_len, int64_t list_len,
                                                                const int32_t* cu, const int64_t* src_slot,
                                                                const int64_t* dst_pos, uint32_t* status, int per_block) {
  __shared__ Place s_src[kMaxNodes], s_dst[kMaxNodes];  // page -1: not moved
  __shared__ uint32_t s_status;
  const int b = blockIdx.x, t = threadIdx.x;
  const int first = blockIdx.y * per_block, last = min(first + per_block, c.layers);
  grid_dependency_wait();
  allow_dependents();
  if (t == 0) s_status = 0u;
  __syncthreads();
  const int64_t lo = cu[b];
  const int64_t n64 = static_cast<int64_t>(cu[b + 1]) - lo;
  const bool bad = lo < 0 || n64 < 0 || n64 > max_len || lo + n64 > list_len;
  const int n = bad ? 0 : static_cast<int>(n64);
  for (int e = t; e < n; e += kMoveThreads) {
    const Place src = slot_place(c, src_slot[lo + e]), dst = position_place(c, b, dst_pos[lo + e]);
    const bool ok = src.page >= 0 && dst.page >= 0;
    if (!ok) atomicOr(&s_status, kStSlotRange);
    s_src[e] = src;
    // an entry already in place is not moved
    s_dst[e] = ok && !(src.page == dst.page && src.in == dst.in) ? dst : Place{-1, 0};
  }
  __syncthreads();
  if (blockIdx.y == 0 && t == 0 && status) status[b] = bad ? kStBadLayout : s_status;
  if (n == 0) return;
  // A head's pieces: K's codes, V's codes, K's scales, V's scales.
  const int codes = c.head_dim / 32, scale_bytes = c.head_dim / 16, unit = scale_bytes & -scale_bytes;
  const int scales = scale_bytes / unit, per_head = 2 * (codes + scales), cols = c.heads * per_head;
  const int width = min(cols, kMoveThreads * REGS / n);  // pieces at a time
  for (int c0 = 0; c0 < cols; c0 += width) {
    const int w = min(width, cols - c0);
    int64_t src[REGS], dst[REGS];  // bytes; dst -1: nothing to move
    int size[REGS];
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      const int x = t + i * kMoveThreads;
      src[i] = 0, dst[i] = -1, size[i] = 16;
      if (x < w * n) {
        const int e = x / w, col = c0 + x - e * w, head = col / per_head, piece = col - head * per_head;
        int at, step;  // within the block of a head: where the piece of entry 0 lies, and how far the entries are apart
        if (piece < 2 * codes) {
          const bool is_v = piece >= codes;
          at = (is_v ? packed_v_codes(c.page_size, c.head_dim) : 0) + (is_v ? piece - codes : piece) * 16;
          step = c.head_dim / 2;
        } else {
          const int k = piece - 2 * codes;
          const bool is_v = k >= scales;
          at = (is_v ? packed_v_scales(c.page_size, c.head_dim) : packed_k_scales(c.page_size, c.head_dim)) +
               (is_v ? k - scales : k) * unit;
          step = scale_bytes, size[i] = unit;
        }
        const Place from = s_src[e], to = s_dst[e];
        if (to.page >= 0) {
          src[i] = from.page * c.page_stride + head * c.head_stride + at + static_cast<int64_t>(from.in) * step;
          dst[i] = to.page * c.page_stride + head * c.head_stride + at + static_cast<int64_t>(to.in) * step;
        }
      }
    }
    uint4 r[REGS], ahead[REGS];
    auto read = [&](int layer, uint4 (&to)[REGS]) {
      const char* from = c.data + layer * c.layer_stride;
#pragma unroll
      for (int i = 0; i < REGS; ++i)
        if (dst[i] >= 0) {
          const char* a = from + src[i];
          if (size[i] == 16)
            to[i] = *reinterpret_cast<const uint4*>(a);
          else if (size[i] == 8)
            to[i].x = reinterpret_cast<const uint2*>(a)->x, to[i].y = reinterpret_cast<const uint2*>(a)->y;
          else if (size[i] == 4)
            to[i].x = *reinterpret_cast<const uint32_t*>(a);
          else
            to[i].x = *reinterpret_cast<const uint16_t*>(a);
        }
    };
    read(first, r);
    for (int layer = first; layer < last; ++layer) {
      if (layer + 1 < last) read(layer + 1, ahead);
      __syncthreads();
      char* to = c.data + layer * c.layer_stride;
#pragma unroll
      for (int i = 0; i < REGS; ++i) {
        if (dst[i] >= 0) {
          char* a = to + dst[i];
          if (size[i] == 16)
            *reinterpret_cast<uint4*>(a) = r[i];
          else if (size[i] == 8)
            *reinterpret_cast<uint2*>(a) = make_uint2(r[i].x, r[i].y);
          else if (size[i] == 4)
            *reinterpret_cast<uint32_t*>(a) = r[i].x;
          else
            *reinterpret_cast<uint16_t*>(a) = static_cast<uint16_t>(r[i].x);
        }
        r[i] = ahead[i];
      }
    }
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status_t spec_verify_packed_kv_commit(const sv_packed_kv_cache_t* cache, int32_t batch, int32_t max_len,
                                                    int64_t list_len, const int32_t* commit_cu,
                                                    const int64_t* commit_src_slot, const int64_t* commit_dst_pos,
                                                    uint32_t* dev_status, cudaStream_t stream) {
  if (batch < 0 || batch > 65535 || max_len < 1 || max_len > kMaxNodes || list_len < 0) return SV_ERR_BAD_SHAPE;
  PackedView c{};
  const sv_status_t s = check_packed_cache(cache, &c);
  if (s != SV_OK) return s;
  if (batch == 0) return SV_OK;
  if (!commit_cu || (list_len > 0 && (!commit_src_slot || !commit_dst_pos))) return SV_ERR_NULL_ARG;
  if (!blocks_apart(c)) return SV_ERR_UNSUPPORTED;  // a block would read what another has already moved
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  int64_t per = batch * static_cast<int64_t>(c.layers) / (kMoveBlocks * dev.sms);
  per = per < 1 ? 1 : per > c.layers ? c.layers : per;
  const int64_t parts = (c.layers + per - 1) / per;
  if (parts > 65535) return SV_ERR_BAD_SHAPE;
  const dim3 grid(static_cast<unsigned>(batch), static_cast<unsigned>(parts));
  e = launch_pdl(max_len <= 2 * kMoveThreads ? k_packed_commit<2> : k_packed_commit<4>, grid, dim3(kMoveThreads), 0, stream, c,
                 max_len, list_len, commit_cu, commit_src_slot, commit_dst_pos, dev_status, static_cast<int>(per));
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}
