// Attention of the verify rows over a KV cache held in 4 bits: the entry point, and the choice among its kernels.  The
// mathematics and the division of the work are those of sv_attention.cu.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include "sv_attention_packed.cuh"

using namespace sv;

extern "C" sv_status_t spec_verify_packed_attention(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, int32_t num_heads, const sv_packed_kv_cache_t* cache,
    int32_t layer, int32_t batch, int64_t total_rows, int32_t max_len, const int32_t* cu_seqlens, const int64_t* seq_lens,
    const int64_t* row_slots, const uint8_t* mask, float scale, void* out, int64_t out_row_stride, int64_t out_head_stride,
    float* lse, uint32_t* dev_status, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!attention_sizes(batch, max_len, total_rows)) return SV_ERR_BAD_SHAPE;
  PackedView c{};
  sv_status_t s = check_packed_cache(cache, &c);
  if (s != SV_OK) return s;
  if (c.dtype != SV_BF16) return SV_ERR_BAD_DTYPE;
  KvView pages{};  // the pages alone: the memory is c's
  pages.es = 2, pages.layers = c.layers, pages.pages = c.pages, pages.page_size = c.page_size, pages.heads = c.heads;
  pages.head_dim = c.head_dim, pages.table = c.table, pages.max_pages = c.max_pages, pages.ld_table = c.ld_table;
  pages.div_mul = c.div_mul, pages.div_shift = c.div_shift;
  AttnParams p{};
  DeviceInfo dev{};
  s = attention_params(q, q_row_stride, q_head_stride, num_heads, pages, layer, batch, total_rows, max_len, cu_seqlens, seq_lens,
                       row_slots, mask, scale, out, out_row_stride, out_head_stride, lse, dev_status, ws, ws_bytes, &p, &dev);
  if (s != SV_OK || batch == 0) return s;
  c.data += layer * c.layer_stride;
  const int64_t rows = static_cast<int64_t>(max_len) * p.group;
  const cudaError_t e = rows <= (c.head_dim <= 128 ? 16 : 8) ? launch_packed_attention_few(p, c, dev, stream)
                                                             : launch_packed_attention_wide(p, c, dev, stream);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}
