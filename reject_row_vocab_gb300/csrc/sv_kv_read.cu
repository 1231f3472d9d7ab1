// The entries of given rows' places, of one or several layers, as dense rows:
// of the 4-bit cache the values that they stand for, which bf16 and fp32 hold
// exactly.  (What a request's handing over, a dense attention over a prefix, or
// a look at the cache needs; [E2D] §5.6.6: the committed slots.)
//
// Bound by the bytes of the output.  A warp takes one row, or a part of its
// heads and layers; a lane has eight columns of a head, or, of codes, a group of
// 16 with its scale.  8192 rows of 8 heads of 128 out of 4 bits: 15 us (43 MB: 2.9
// TB/s; the floor is 6.4), of which looking up a row's place and the start take
// half, and as long out of bf16 (67 MB, 4.5 TB/s); 384 rows of 32 layers out of 4 bits
// 21 us.  Four passes in flight: eight take 15.9 and 23.3 us, two 14.5 and 21.7 (and
// 16.5 out of bf16); twice the warps a row 16.6 and 20.7.
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

// Columns of a lane: of the 4-bit cache a group's (8 bytes of codes and its scale), else eight.
template <class C>
constexpr int kLaneCols = std::is_same<C, PackedView>::value ? 16 : 8;

template <int ES, class C>
__global__ void __launch_bounds__(32 * kReadWarps) k_kv_read(const ReadParams p, const C c) {
  constexpr bool kPacked = std::is_same<C, PackedView>::value;
  constexpr int kCols = kLaneCols<C>, kPieces = kCols * ES / 16;  // 16-byte pieces of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = (p.dim + kCols - 1) / kCols, heads = 32 / lanes;
  const int of = lane / lanes, d0 = (lane - of * lanes) * kCols;
  const int live = of < heads ? (p.heads - of + heads - 1) / heads : 0;  // passes over the heads in which this lane has one
  const int rounds = (p.heads + heads - 1) / heads;                      // passes over the heads
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
    // This lane's columns of head `of` of layer 0: in K's memory and V's, and in the outputs.
    const char *from[2] = {nullptr, nullptr}, *scale[2] = {nullptr, nullptr};
    int64_t layer_step, head_step;
    if constexpr (kPacked) {
      const char* block = c.data + static_cast<int64_t>(there ? place.page : 0) * c.page_stride + of * c.head_stride;
      const int code = place.in * (c.head_dim / 2) + d0 / 2, group = place.in * (c.head_dim / 16) + d0 / 16;
      from[0] = block + code, from[1] = from[0] + packed_v_codes(c.page_size, c.head_dim);
      scale[0] = block + packed_k_scales(c.page_size, c.head_dim) + group;
      scale[1] = block + packed_v_scales(c.page_size, c.head_dim) + group;
      layer_step = c.layer_stride, head_step = heads * c.head_stride;
    } else {
      const int64_t at = (static_cast<int64_t>(there ? place.page : 0) * c.page_stride + place.in * c.slot_stride + of * c.head_stride + d0) * ES;
      from[0] = c.k + at, from[1] = c.v + at;
      layer_step = c.layer_stride * ES, head_step = heads * c.head_stride * ES;
    }
    const int64_t out_at = (row * p.o_row + of * p.o_head + d0) * ES, out_layer = p.o_layer * ES, out_head = heads * p.o_head * ES;
    // A pass is a round over the heads of K or V of a layer.
    int layer = first / (2 * rounds), round = first - layer * 2 * rounds, which = round >= rounds ? 1 : 0;
    round -= which * rounds;
    for (int pass0 = first; pass0 < last; pass0 += kReadUnroll) {
      uint4 a[kReadUnroll][kPieces];
      uint2 code[kReadUnroll];
      uint32_t byte[kReadUnroll];
      char* to[kReadUnroll];
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u) {
        const bool have = pass0 + u < last && round < live;
        to[u] = have ? (which ? p.v : p.k) + out_at + layer * out_layer + round * out_head : nullptr;
        code[u] = make_uint2(0u, 0u), byte[u] = 0u;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) a[u][i] = make_uint4(0u, 0u, 0u, 0u);
        if (have && there) {
          const int64_t at = layer * layer_step + round * head_step;
          const char* f = (which ? from[1] : from[0]) + at;
          if constexpr (kPacked) {
            code[u] = *reinterpret_cast<const uint2*>(f);
            byte[u] = static_cast<unsigned char>((which ? scale[1] : scale[0])[at]);
          } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
              if (d0 * ES + i * 16 < p.dim * ES) a[u][i] = *reinterpret_cast<const uint4*>(f + i * 16);
          }
        }
        if (++round == rounds) round = 0, which ^= 1, layer += which ^ 1;
      }
#pragma unroll
      for (int u = 0; u < kReadUnroll; ++u) {
        if (!to[u]) continue;
        if constexpr (kPacked) {
          const uint32_t s2 = scale_pair(byte[u] | byte[u] << 16);
          uint32_t w[kCols * ES / 4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t f[4];
            unpack_codes(h ? code[u].y : code[u].x, f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v = mul_half2(f[i], s2);
              const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v));
              if (ES == 4)
                w[(h * 4 + i) * ES / 2] = __float_as_uint(x.x), w[(h * 4 + i) * ES / 2 + 1] = __float_as_uint(x.y);
              else
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[h * 4 + i]) : "f"(x.y), "f"(x.x));
            }
          }
#pragma unroll
          for (int i = 0; i < kPieces; ++i) a[u][i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if (d0 * ES + i * 16 < p.dim * ES) *reinterpret_cast<uint4*>(to[u] + i * 16) = a[u][i];
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
  const int lanes = (c.head_dim + kLaneCols<C> - 1) / kLaneCols<C>, heads = 32 / lanes;
  const int64_t passes = static_cast<int64_t>(num_layers) * 2 * ((c.heads + heads - 1) / heads);
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
