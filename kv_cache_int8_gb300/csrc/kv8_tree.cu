// kv8_tree.cu -- attention of drafted tokens over the 8-bit K/V cache: node i of a sequence's tree
// sees the context in front of the tree, itself and its ancestors.
//
// Source: "KV Cache 与长上下文推理", section "KV Cache 回顾" (decode attention equation); the pages
// have no drafted tokens.
//
// One warp has one (node, query head) and goes over all tokens, four channels a lane, with the
// running maximum and sum of the softmax in fp32.
#include <cmath>

#include "internal.h"
#include "kv8.cuh"

namespace hsa {
namespace {

using namespace kv8_detail;

constexpr int kWarps = 8;
constexpr int kWords = kKv8TreeNodes / 32;

struct Params {
  NewRows rows;
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* parents;
  const int32_t* page_table;
  __nv_bfloat16* out;
  float* lse;
  int* err;
  int hq, hkv, group, num_pages;
  float scale;
};

__device__ __forceinline__ float sum32(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

template <int F>
__global__ void __launch_bounds__(kWarps * 32) kv8_tree_kernel(const Params p) {
  __shared__ uint32_t branch[kWarps][kWords];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const int row = (int)(unit / p.hq), head = (int)(unit % p.hq);
  if (unit == (long long)p.rows.total * p.hq) report_bad(p.rows, lane, p.err);
  if (row >= p.rows.total) return;
  int b = row;
  if (p.rows.cu != nullptr) {
    int lo = 0, hi = p.rows.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.rows.cu[mid] <= row) lo = mid;
      else hi = mid;
    }
    b = lo;
    if (row < p.rows.cu[b] || row >= p.rows.cu[b + 1]) return;  // of no sequence
  }
  const NewSpan sp = new_span(p.rows, b);
  const size_t at = (size_t)row * p.hq + head;
  // sums of up to 256 tokens (l1, o1), added up in (l, o): a million adds one after the other
  // would be 5e-5 off
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float l1 = 0.0f, o1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto collect = [&]() {
    l += l1;
    l1 = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      o[k] += o1[k];
      o1[k] = 0.0f;
    }
  };
  if (sp.n > kKv8TreeNodes && lane == 0) set_error(p.err, kDevErrCheck);
  if (sp.n > 0 && sp.n <= kKv8TreeNodes) {
    if (lane < kWords) branch[warp][lane] = 0;
    __syncwarp();
    if (lane == 0) {
      for (int i = row - sp.row0; i >= 0;) {
        branch[warp][i >> 5] |= 1u << (i & 31);
        const int up = p.parents ? p.parents[sp.row0 + i] : i - 1;
        if (up < -1 || up >= i) {
          set_error(p.err, kDevErrCheck);
          break;
        }
        i = up;
      }
    }
    __syncwarp();
    const uint2 raw = *reinterpret_cast<const uint2*>(p.q + (long long)row * p.q_stride +
                                                      head * kHeadDim + 4 * lane);
    const float q[4] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y)};
    const int len = sp.start + sp.n, h = head / p.group;
    for (int t = 0; t < len; t++) {
      const int i = t - sp.start;
      if (i >= 0 && !(branch[warp][i >> 5] >> (i & 31) & 1)) continue;
      const int page = p.page_table[(size_t)b * p.rows.max_pages + t / kPage];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) set_error(p.err, kDevErrCheck);
        continue;
      }
      const size_t block = (size_t)page * p.hkv + h;
      const size_t off = block * kBlockBytesI8 + t % kPage * kHeadDim + 4 * lane;
      float f[4];
      values4<F>(*reinterpret_cast<const uint32_t*>(p.k + off), f);
      float x = q[0] * f[0] + q[1] * f[1] + q[2] * f[2] + q[3] * f[3];
      x = sum32(x) * p.k_scale[block] * p.scale;
      const float top = fmaxf(m, x);
      const float keep = m == -INFINITY ? 0.0f : expf(m - top), w = expf(x - top);
      values4<F>(*reinterpret_cast<const uint32_t*>(p.v + off), f);
      l *= keep;
      l1 = l1 * keep + w;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        o[k] *= keep;
        o1[k] = o1[k] * keep + w * f[k] * p.v_scale[block];
      }
      m = top;
      if (t % 256 == 255) collect();
    }
    collect();
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int k = 0; k < 4; k++) p.out[at * kHeadDim + 4 * lane + k] = __float2bfloat16(o[k] * inv);
  if (p.lse != nullptr && lane == 0) p.lse[at] = l != 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_kv8_tree(const Shape& s, const Kv8& c, const void* q, long long q_stride,
                            const int32_t* parents, const int32_t* cu, int total,
                            const int32_t* page_table, const int32_t* seq_lens, void* out,
                            float* lse, int* err, cudaStream_t st) {
  Params p;
  p.rows = NewRows{cu, seq_lens, s.batch, total, s.max_pages};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.parents = parents;
  p.page_table = page_table;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = err;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.group = s.group;
  p.num_pages = s.num_pages;
  p.scale = s.sm_scale;
  const long long units = (long long)total * s.hq;
  auto kernel = c.format == kE4m3 ? kv8_tree_kernel<kE4m3> : kv8_tree_kernel<kInt8>;
  return launch_kernel(kernel, dim3((unsigned)(units / kWarps + 1)), dim3(kWarps * 32), 0, st, true,
                       p);
}

}  // namespace hsa
