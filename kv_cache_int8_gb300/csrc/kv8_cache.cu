// kv8_cache.cu -- the 8-bit K/V cache: new tokens quantised into it, and its values read back.
//
// Source: "KV Cache 与长上下文推理", section "KV Cache 量化" (K and V kept in INT8 / FP8 with
// shared scales); section "KV Cache 回顾" (every step appends the new tokens' K and V).
//
// Both move each element once (bf16 in, one byte out, or the reverse) and are bound by memory,
// 3 bytes an element; a single token a sequence is bound by latency. One warp owns one block
// (page, kv head) of K or of V from its first byte to its last: 16 tokens x 128 channels are 64
// values a lane, which stay in registers between the maximum and the codes, so the input is
// read once and no shared memory or second launch is needed. Sequences share nothing, so any
// block of any sequence is one work item (new_block_items) and ragged batches balance.
//
// Measured (GB300, copy 6.8 TB/s, 8 kv heads): 108K new tokens of 8 prompts written in 108 us
// (664 MB, 6.1 TB/s), 117K tokens read back in 109 us (720 MB, 6.6 TB/s); one token of one
// sequence written in 2.3 us, of 256 sequences in 3.7, 1024 tokens read in 2.9. With offsets, one
// token of each of 256 sequences written in 6.05 us and read in 4.4 (found by bisection 7.2 and 5.6);
// 25 tokens of one sequence 2.7 and 2.2 (by the warp's search, which loads an offset first, 3.0 and
// 2.5), 8000 tokens 8.1 and 6.8 (8.8 and 7.2); 25 of each of four 3.1 and 2.6 either way.
#include "append.cuh"
#include "kv8.cuh"

namespace hsa {
namespace {

using namespace kv8_detail;
using append_detail::unpack8;

constexpr int kWarps = 8;  // work items a CTA

struct WriteSide {
  const __nv_bfloat16* x;  // rows
  long long stride;        // elements
  uint8_t* codes;
  float* scale;
};

// Lane l holds channels [8 (l % 16), 8 (l % 16) + 8) of tokens 2 i + l / 16, i = 0 .. 7: a warp
// reads two rows of 256 contiguous bytes an instruction and writes two rows of 128.
template <int F, bool kFew>
__global__ void __launch_bounds__(kWarps * 32) kv8_write_kernel(
    NewRows rows, WriteSide ks, WriteSide vs, const int32_t* __restrict__ page_table, int hkv,
    int num_pages, int units, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit == units) report_bad(rows, lane, err);
  if (unit >= units) return;
  const bool is_v = unit & 1;
  const int h = (unit >> 1) % hkv, item = (unit >> 1) / hkv;
  const WriteSide& w = is_v ? vs : ks;
  const int b = !rows.cu ? item
                : kFew   ? item_sequence_of_few(rows, item)
                         : item_sequence(rows, item, lane);
  if (!kFew && b < 0) return;
  const NewSpan sp = new_span(rows, b);
  const int j = rows.cu ? item - item_base(rows, b) : 0;
  const int end = sp.start + sp.n;  // N_b
  const long long p = (long long)sp.start / kPage + j;
  if (sp.n == 0 || j < 0 || p * kPage >= end) return;
  const int page = page_table[(size_t)b * rows.max_pages + p];
  if (page < 0 || page >= num_pages) {
    if (lane == 0) set_error(err, kDevErrCheck);
    return;
  }
  const int base = (int)p * kPage;
  const int first = max(sp.start - base, 0);        // slots [first, last) receive new tokens
  const int last = min(end - base, kPage);
  const size_t block = (size_t)page * hkv + h;
  const float s_old = w.scale[block];
  const int sub = lane >> 4, ch = (lane & 15) * 8;
  const __nv_bfloat16* x = w.x + ((long long)sp.row0 + base - sp.start + sub) * w.stride +
                           h * kHeadDim + ch;  // row of slot `sub`
  uint4 raw[8];
  uint32_t mx = 0;  // packed maxima of the magnitudes' bits
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int slot = 2 * i + sub;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= first && slot < last) raw[i] = ldg128_nc(x + 2 * i * w.stride);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    mx = __vmaxu2(mx, raw[i].x & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, raw[i].y & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, raw[i].z & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, raw[i].w & 0x7FFF7FFFu);
  }
  uint32_t m = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
  const bool odd_values = m >= 0x7F80u;  // an infinity or a NaN: the maximum of the finite ones
  if (odd_values) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const uint32_t lo = v[k] & 0x7FFFu, hi = (v[k] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) m = max(m, lo);
        if (hi < 0x7F80u) m = max(m, hi);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
  }
  float s = __fdiv_rn(__uint_as_float(m << 16), levels<F>());
  if (s < 1.17549435e-38f) s = 0.0f;
  if (first > 0) s = fmaxf(s_old, s);
  const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  uint8_t* dst = w.codes + block * kBlockBytesI8 + sub * kHeadDim + ch;
  if (first > 0 && s > s_old) {  // the older tokens' codes under the larger scale
    const float ratio = __fmul_rn(s_old, inv);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int slot = 2 * i + sub;
      if (slot >= first) continue;
      uint2* at = reinterpret_cast<uint2*>(dst + 2 * i * kHeadDim);
      const uint2 c = *at;
      float f[8];
      values4<F>(c.x, f);
      values4<F>(c.y, f + 4);
      *at = make_uint2(codes4<F>(f[0], f[1], f[2], f[3], ratio),
                       codes4<F>(f[4], f[5], f[6], f[7], ratio));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int slot = 2 * i + sub;
    if (slot < first || slot >= last) continue;
    float f[8];
    unpack8(raw[i], f);
    float by = inv;
    if (odd_values) {
#pragma unroll
      for (int k = 0; k < 8; k++) f[k] = tame<F>(f[k], inv);
      by = 1.0f;
    }
    *reinterpret_cast<uint2*>(dst + 2 * i * kHeadDim) =
        make_uint2(codes4<F>(f[0], f[1], f[2], f[3], by), codes4<F>(f[4], f[5], f[6], f[7], by));
  }
  if (lane == 0) w.scale[block] = s;
}

struct ReadSide {
  __nv_bfloat16* x;
  long long stride;
  const uint8_t* codes;
  const float* scale;
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Lanes as in the write: 8 bytes of codes in, 16 bytes of bf16 out.
template <int F, bool kFew>
__global__ void __launch_bounds__(kWarps * 32) kv8_read_kernel(
    NewRows rows, ReadSide ks, ReadSide vs, const int32_t* __restrict__ page_table, int hkv,
    int num_pages, int units, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit == units) report_bad(rows, lane, err);
  if (unit >= units) return;
  const bool is_v = unit & 1;
  const int h = (unit >> 1) % hkv, item = (unit >> 1) / hkv;
  const ReadSide& r = is_v ? vs : ks;
  const int b = !rows.cu ? item
                : kFew   ? item_sequence_of_few(rows, item)
                         : item_sequence(rows, item, lane);
  if (!kFew && b < 0) return;
  const NewSpan sp = new_span(rows, b);
  const int j = rows.cu ? item - item_base(rows, b) : 0;
  const int end = sp.start + sp.n;
  const long long p = (long long)sp.start / kPage + j;
  if (sp.n == 0 || j < 0 || p * kPage >= end) return;
  const int page = page_table[(size_t)b * rows.max_pages + p];
  if (page < 0 || page >= num_pages) {
    if (lane == 0) set_error(err, kDevErrCheck);
    return;
  }
  const int base = (int)p * kPage;
  const int first = max(sp.start - base, 0), last = min(end - base, kPage);
  const size_t block = (size_t)page * hkv + h;
  const int sub = lane >> 4, ch = (lane & 15) * 8;
  const uint8_t* src = r.codes + block * kBlockBytesI8 + sub * kHeadDim + ch;
  uint2 c[8];
#pragma unroll
  for (int i = 0; i < 8; i++) c[i] = ldg64_nc(src + 2 * i * kHeadDim);
  const float s = r.scale[block];
  __nv_bfloat16* x = r.x + ((long long)sp.row0 + base - sp.start + sub) * r.stride +
                     h * kHeadDim + ch;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int slot = 2 * i + sub;
    if (slot < first || slot >= last) continue;
    float f[8];
    values4<F>(c[i].x, f);
    values4<F>(c[i].y, f + 4);
#pragma unroll
    for (int k = 0; k < 8; k++) f[k] = __fmul_rn(f[k], s);
    *reinterpret_cast<uint4*>(x + 2 * i * r.stride) =
        make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]),
                   bf16_pair(f[6], f[7]));
  }
}

}  // namespace

cudaError_t launch_kv8_write(const Shape& s, const Kv8& c, const void* k_new, long long k_stride,
                             const void* v_new, long long v_stride, const int32_t* cu, int total,
                             const int32_t* page_table, const int32_t* seq_lens, int* err,
                             cudaStream_t st) {
  const NewRows rows = {cu, seq_lens, s.batch, total, s.max_pages};
  const WriteSide ks = {static_cast<const __nv_bfloat16*>(k_new), k_stride,
                        static_cast<uint8_t*>(c.k), c.k_scale};
  const WriteSide vs = {static_cast<const __nv_bfloat16*>(v_new), v_stride,
                        static_cast<uint8_t*>(c.v), c.v_scale};
  const int units = new_block_items(s.batch, total, cu != nullptr) * s.hkv * 2;
  const bool few = s.batch <= kFewSequences;
  auto kernel = c.format == kE4m3
                    ? (few ? kv8_write_kernel<kE4m3, true> : kv8_write_kernel<kE4m3, false>)
                    : (few ? kv8_write_kernel<kInt8, true> : kv8_write_kernel<kInt8, false>);
  return launch_kernel(kernel, dim3(units / kWarps + 1), dim3(kWarps * 32), 0, st,
                       true, rows, ks, vs, page_table, s.hkv, s.num_pages, units, err);
}

cudaError_t launch_kv8_read(const Shape& s, const Kv8& c, void* k_out, long long k_stride,
                            void* v_out, long long v_stride, const int32_t* cu, int total,
                            const int32_t* page_table, const int32_t* seq_lens, int* err,
                            cudaStream_t st) {
  const NewRows rows = {cu, seq_lens, s.batch, total, s.max_pages};
  const ReadSide ks = {static_cast<__nv_bfloat16*>(k_out), k_stride,
                       static_cast<const uint8_t*>(c.k), c.k_scale};
  const ReadSide vs = {static_cast<__nv_bfloat16*>(v_out), v_stride,
                       static_cast<const uint8_t*>(c.v), c.v_scale};
  const int units = new_block_items(s.batch, total, cu != nullptr) * s.hkv * 2;
  const bool few = s.batch <= kFewSequences;
  auto kernel = c.format == kE4m3
                    ? (few ? kv8_read_kernel<kE4m3, true> : kv8_read_kernel<kE4m3, false>)
                    : (few ? kv8_read_kernel<kInt8, true> : kv8_read_kernel<kInt8, false>);
  return launch_kernel(kernel, dim3(units / kWarps + 1), dim3(kWarps * 32), 0, st,
                       true, rows, ks, vs, page_table, s.hkv, s.num_pages, units, err);
}

}  // namespace hsa
