// The entries of given rows' places, of one or several layers, as dense rows:
// of the 4-bit cache the values that they stand for, which bf16 and fp32 hold
// exactly.  (What a request's handing over, a dense attention over a prefix, or
// a look at the cache needs; [E2D] §5.6.6: the committed slots.)
//
// Bound by the bytes of the output.  A warp takes one row, or a part of its
// heads and layers; a lane has eight columns of a head: 16 bytes of bf16, four
// bytes of codes.
//
//   [E2D] "从 EAGLE 到 DFlash 2：SGLang 与 SpecForge 的投机解码训练和推理"
#include <cstdint>
#include <type_traits>

#include "sv_rows.cuh"

namespace sv {
namespace {

constexpr int kReadWarps = 4;
constexpr int kReadUnroll = 4;

struct ReadParams {
  RowsView r;
  char *k, *v;
  int64_t o_layer, o_row, o_head;  // strides in elements
  int32_t layers, heads, dim;
  uint32_t* status;
  int32_t passes, chunks, per;
};

template <int ES, class C>
__global__ void __launch_bounds__(32 * kReadWarps) k_kv_read(const ReadParams p, const C c) {
  constexpr bool kPacked = std::is_same<C, PackedView>::value;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = (p.dim + 7) / 8, heads = 32 / lanes;
  const int of = lane / lanes, d0 = (lane - of * lanes) * 8;
  const bool wide = ES == 2 || d0 + 4 < p.dim;
  const int slots = p.layers * 2 * p.heads;
  grid_dependency_wait();
  allow_dependents();
  const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  flag_requests(p.r, p.status, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x, threads);
  const int64_t items = rows_count(p.r) * p.chunks;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kReadWarps + warp; item < items; item += threads / 32) {
    const int64_t row = p.chunks == 1 ? item : item / p.chunks;
    const int chunk = static_cast<int>(item - row * p.chunks);
    int j;
    const int b = row_request(p.r, row, lane, &j);
    if (b < 0) continue;
    const int64_t len = p.r.seq_lens ? p.r.seq_lens[b] : 0;
    if (len < 0) continue;
    const Place place = p.r.row_slots ? slot_place(c, p.r.row_slots[row]) : position_place(c, b, len + j);
    const bool there = place.page >= 0;
    if (!there && chunk == 0 && lane == 0) atomicOr(p.status + b, kStSlotRange);
    const int first = chunk * p.per, last = min(first + p.per, p.passes);
    for (int pass0 = first; pass0 < last; pass0 += kReadUnroll) {
      uint4 a[kReadUnroll], a2[kReadUnroll];
      uint32_t code[kReadUnroll], byte[kReadUnroll];
      char* to[kReadUnroll];
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u) {
        const int s = (pass0 + u) * heads + of;
        to[u] = nullptr;
        a[u] = a2[u] = make_uint4(0u, 0u, 0u, 0u);
        code[u] = byte[u] = 0u;
        if (of >= heads || pass0 + u >= last || s >= slots) continue;
        const int which = s / p.heads, head = s - which * p.heads, layer = which >> 1;
        const bool is_v = which & 1;
        to[u] = (is_v ? p.v : p.k) + (layer * p.o_layer + row * p.o_row + head * p.o_head + d0) * ES;
        if (!there) continue;
        if constexpr (kPacked) {
          const char* block = c.data + layer * c.layer_stride + place.page * c.page_stride + head * c.head_stride;
          code[u] = *reinterpret_cast<const uint32_t*>(block + (is_v ? packed_v_codes(c.page_size, c.head_dim) : 0) +
                                                       place.in * (c.head_dim / 2) + d0 / 2);
          byte[u] = static_cast<unsigned char>(
              block[(is_v ? packed_v_scales(c.page_size, c.head_dim) : packed_k_scales(c.page_size, c.head_dim)) +
                    place.in * (c.head_dim / 16) + d0 / 16]);
        } else {
          const char* at = (is_v ? c.v : c.k) +
                           (layer * c.layer_stride + place.page * c.page_stride + place.in * c.slot_stride +
                            head * c.head_stride + d0) * ES;
          a[u] = *reinterpret_cast<const uint4*>(at);
          if (ES == 4 && wide) a2[u] = *reinterpret_cast<const uint4*>(at + 16);
        }
      }
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u) {
        if (!to[u]) continue;
        if constexpr (kPacked) {
          uint32_t h[4];
          unpack_codes(code[u], h);
          const uint32_t s2 = scale_pair(byte[u] | byte[u] << 16);
          float x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = mul_half2(h[i], s2);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
          }
          uint32_t w[ES * 2];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (ES == 4)
              w[i] = __float_as_uint(x[i]);
            else if (i % 2 == 0)
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i / 2]) : "f"(x[i + 1]), "f"(x[i]));
          a[u] = make_uint4(w[0], w[1], w[2], w[3]);
          if (ES == 4) a2[u] = make_uint4(w[ES * 2 - 4], w[ES * 2 - 3], w[ES * 2 - 2], w[ES * 2 - 1]);
        }
        *reinterpret_cast<uint4*>(to[u]) = a[u];
        if (ES == 4 && wide) *reinterpret_cast<uint4*>(to[u] + 16) = a2[u];
      }
    }
  }
}

void span_of(const KvView& c, const char** at, int64_t* bytes) {
  const int64_t span = ((c.layers - 1) * c.layer_stride + (c.pages - 1) * c.page_stride + (c.page_size - 1) * c.slot_stride +
                        (c.heads - 1) * c.head_stride + c.head_dim) * c.es;
  at[0] = c.k, at[1] = c.v, bytes[0] = bytes[1] = span;
}
void span_of(const PackedView& c, const char** at, int64_t* bytes) {
  at[0] = at[1] = c.data;
  bytes[0] = bytes[1] = (c.layers - 1) * c.layer_stride + (c.pages - 1) * c.page_stride + (c.heads - 1) * c.head_stride +
                        packed_block_bytes(c.page_size, c.head_dim);
}
void to_layer(KvView* c, int layer) {
  c->k += layer * c->layer_stride * c->es;
  c->v += layer * c->layer_stride * c->es;
}
void to_layer(PackedView* c, int layer) { c->data += layer * c->layer_stride; }

template <class C>
sv_status_t read_entry(C c, int es, int32_t layer, int32_t num_layers, const sv_rows_t* rows, void* k, void* v,
                       int64_t o_layer, int64_t o_row, int64_t o_head, uint32_t* dev_status, cudaStream_t stream) {
  RowsView r{};
  const sv_status_t s = check_rows(rows, &r);
  if (s != SV_OK) return s;
  if (layer < 0 || num_layers < 0 || layer > c.layers - num_layers || o_layer < 0 || o_row < 0 || o_head < 0) return SV_ERR_BAD_SHAPE;
  if (static_cast<int64_t>(num_layers) * 2 * c.heads > (1 << 26)) return SV_ERR_BAD_SHAPE;
  if (r.batch == 0 || rows_count(r) == 0 || num_layers == 0) return SV_OK;
  if (!k || !v || !dev_status || (!r.seq_lens && !r.row_slots)) return SV_ERR_NULL_ARG;
  if (!aligned16(k) || !aligned16(v) || (o_layer * es) % 16 != 0 || (o_row * es) % 16 != 0 || (o_head * es) % 16 != 0)
    return SV_ERR_MISALIGNED;
  const int64_t row_bytes = static_cast<int64_t>(c.head_dim) * es;
  StepAxis axes[3] = {{o_layer * es, num_layers}, {o_row * es, r.total}, {o_head * es, c.heads}};
  int64_t span, bytes[2];
  if (!steps_nested(axes, 3, row_bytes, &span)) return SV_ERR_UNSUPPORTED;
  char *const kp = static_cast<char*>(k), *const vp = static_cast<char*>(v);
  const char* at[2];
  span_of(c, at, bytes);
  auto meet = [](const char* a, int64_t na, const char* b, int64_t nb) { return a < b + nb && b < a + na; };
  if (meet(kp, span, vp, span)) return SV_ERR_UNSUPPORTED;
  for (int i = 0; i < 2; ++i)
    if (meet(kp, span, at[i], bytes[i]) || meet(vp, span, at[i], bytes[i])) return SV_ERR_UNSUPPORTED;
  DeviceInfo dev{};
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return cuda_failure(e);
  to_layer(&c, layer);
  const int lanes = (c.head_dim + 7) / 8, heads = 32 / lanes;
  const int64_t passes = (static_cast<int64_t>(num_layers) * 2 * c.heads + heads - 1) / heads;
  const int64_t count = rows_count(r), want = 32 * static_cast<int64_t>(dev.sms);
  int64_t chunks = (want + count - 1) / count;
  chunks = chunks > passes ? passes : chunks;
  const int64_t per = (passes + chunks - 1) / chunks;
  chunks = (passes + per - 1) / per;
  const ReadParams p{r, kp, vp, o_layer, o_row, o_head, num_layers, c.heads, c.head_dim, dev_status,
                     static_cast<int32_t>(passes), static_cast<int32_t>(chunks), static_cast<int32_t>(per)};
  const int64_t blocks = (count * chunks + kReadWarps - 1) / kReadWarps, most = 64 * static_cast<int64_t>(dev.sms);
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most)), block(32 * kReadWarps);
  e = es == 2 ? launch_pdl(k_kv_read<2, C>, grid, block, 0, stream, p, c) : launch_pdl(k_kv_read<4, C>, grid, block, 0, stream, p, c);
  return e == cudaSuccess ? SV_OK : cuda_failure(e);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

sv_status_t spec_verify_kv_read(const sv_kv_cache_t* cache, int32_t layer, int32_t num_layers, const sv_rows_t* rows,
                                void* k, void* v, int64_t layer_stride, int64_t row_stride, int64_t head_stride,
                                uint32_t* dev_status, cudaStream_t stream) {
  KvView c{};
  const sv_status_t s = check_cache(cache, &c);
  if (s != SV_OK) return s;
  return read_entry(c, c.es, layer, num_layers, rows, k, v, layer_stride, row_stride, head_stride, dev_status, stream);
}

sv_status_t spec_verify_packed_kv_read(const sv_packed_kv_cache_t* cache, int32_t layer, int32_t num_layers,
                                       const sv_rows_t* rows, void* k, void* v, int64_t layer_stride,
                                       int64_t row_stride, int64_t head_stride, uint32_t* dev_status,
                                       cudaStream_t stream) {
  PackedView c{};
  const sv_status_t s = check_packed_cache(cache, &c);
  if (s != SV_OK) return s;
  return read_entry(c, c.dtype == SV_BF16 ? 2 : 4, layer, num_layers, rows, k, v, layer_stride, row_stride, head_stride,
                    dev_status, stream);
}

size_t spec_verify_packed_kv_block_bytes(int32_t page_size, int32_t head_dim) {
  return packed_shape(page_size, head_dim) ? static_cast<size_t>(packed_block_bytes(page_size, head_dim)) : 0;
}

}  // extern "C"
