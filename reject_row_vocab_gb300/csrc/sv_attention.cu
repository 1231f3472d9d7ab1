// Attention of the verify rows over the paged cache ([E2D] §2.4: each node
// sees the committed history, its ancestors and itself): the entry point, and
// the choice among its kernels.
//
//   s_x = scale q.k_x,  m = max s,  l = sum e^(s_x - m),  o = sum e^(s_x - m) v_x / l
//
// kept as running (m, l, O) over tiles of keys, in base 2 (scale log2(e) is
// the factor of the scores), in fp32.  The division of the work and the join
// of its parts are described in sv_attention.cuh.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cmath>
#include <cstdint>

#include "sv_attention_ring.cuh"

namespace sv {
namespace {

// bf16: units of 16 rows on matrix instructions of a warp where a request's rows of a cache head fit them, else units of
// 128 on tensor memory.  (64 requests of 200 to 400, 8 cache heads of 128: 16 rows 39 us and 45, 32 rows 62 and 46; of up to
// 4000: 16 rows 103 and 100, 32 rows 183 and 101.)  fp32: plain arithmetic.
cudaError_t launch_attention(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  if (p.c.es == 4) return launch_attention_f32(p, dev, stream);
  const int64_t rows = static_cast<int64_t>(p.max_len) * p.group;
  return rows <= 16 ? launch_attention_few(p, dev, stream) : launch_attention_wide(p, dev, stream);
}

// Bytes of one part: two of 512 blocks with units of 64 rows (what 128 rows need on half the blocks is less).
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
  // entries that share their memory (an axis repeated without a step) have no map either
  if ((c.heads > 1 && c.head_stride == 0) || (c.page_size > 1 && c.slot_stride == 0) || (c.pages > 1 && c.page_stride == 0))
    return m;
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
  // rows or heads of the output that lay over one another would be written in no order: the larger of the two steps has to
  // be at least what the other axis spans
  const bool row_last = out_row_stride >= out_head_stride;
  const int64_t steps[2] = {row_last ? out_head_stride : out_row_stride, row_last ? out_row_stride : out_head_stride};
  const int64_t counts[2] = {row_last ? num_heads : total_rows, row_last ? total_rows : num_heads};
  int64_t span = c.head_dim;
  for (int i = 0; i < 2; ++i) {
    if (counts[i] < 2) continue;
    if (steps[i] < span || steps[i] > (INT64_MAX - span) / counts[i]) return SV_ERR_BAD_SHAPE;
    span += steps[i] * (counts[i] - 1);
  }
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
