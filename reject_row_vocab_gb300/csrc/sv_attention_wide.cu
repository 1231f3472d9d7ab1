// Attention over the paged cache for many query rows, on the fifth-generation
// tensor cores: bf16, tiles of 128 rows and 128 keys.
//
//   S = Q K^T (128 x 128, tensor memory)     one warp issues the products
//   P = 2^(c (S - m)), l += sum P            one thread a row: no exchange
//   O += P V  (P from tensor memory)         accumulated in tensor memory
//
// Four softmax warps, four loading warps, one warp that issues the matrix
// instructions (a lane of it, with what they take in uniform registers: by one
// thread alone an instruction took 70 clocks to issue, about as long as to run), one that loads the next unit's Q and one that walks the line
// of tiles ahead of them all, connected by mbarriers.  The loading warps bring
// K and V through the page table into a ring of tiles in the 128-byte swizzle
// the matrix unit reads, and run ahead over the ends of units.  S has two
// buffers, so the next tile's scores are computed while this one's weights are
// taken; P overwrites its own S.  The reference m moves (and O is rescaled) only
// when a row's maximum has grown by more than 2^8: the weights stay below 2^8,
// the sums in fp32, and the result does not depend on the reference.
//
// The weights are rounded to bf16 for the product with V (its operands have one
// type); l sums the unrounded ones, in fp32.  That leaves an error of 0.0022 of
// the outputs' norm, where rounding the outputs alone leaves 0.0017.  Two bf16
// values a weight, as the kernel for few rows has, would give 0.0017 here too,
// but lengthen the softmax warps' chain: 64 requests of 16 rows took 131 us
// instead of 102, two long ones 70 instead of 64.
//
// Bound by the bytes of K and V where histories are long, by the chain from
// scores to weights to sums at each unit's ends where they are short.
// Measured: blocks of 16 rows of 64 requests of up to 4000, 32 heads of 128 on 8
// in the cache: 102 us, 5.6 TB/s; 32 requests, heads of 256: 107 us; 5 rows of
// two requests of 60000 to 100000: 64 us, 5.0 TB/s (18 of them outside the
// stream); trees of 17 nodes of 16 requests in pages of one slot: 22 us; a
// causal block of 1024 rows of one request: 72 us without history, 148 (513
// TFLOP/s) behind 4000, all key tiles gone through by every tile of rows.
//
// Units that several blocks share are joined by a second kernel, spread over
// the whole GPU.  (By the last of the unit's blocks alone, two long requests
// took 90 us instead of 63, a 64-request block 127 instead of 118.)
//
// Every wait is bounded; a wait that gives up raises SV_DEV_TIMEOUT, lets all
// warps leave, and the block frees its tensor memory.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include "sv_attention_wide.cuh"

namespace sv {

cudaError_t launch_attention_wide(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int dim = p.c.head_dim;
  const KvMaps maps = kv_maps(p.c);
  return dim <= 64 ? launch_wide<1, 1, RowSource>(p, maps, dev, stream) : dim <= 128 ? launch_wide<2, 1, RowSource>(p, maps, dev, stream) : launch_wide<2, 2, RowSource>(p, maps, dev, stream);
}

}  // namespace sv
