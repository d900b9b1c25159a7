// kv8.cuh -- what the kernels of the 8-bit K/V cache share: its layout, the rows of new tokens,
// and the exact conversions of its codes to fp16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace hsa {
namespace kv8_detail {

constexpr int kInt8 = 0, kE4m3 = 1;  // formats

// Sequences whose new tokens are given as rows [cu[b], cu[b + 1]) (cu == nullptr: row b).
struct NewRows {
  const int32_t* cu;
  const int32_t* seq_lens;
  int batch, total, max_pages;
};

struct NewSpan {
  int row0;   // first row
  int start;  // position of the first new token
  int n;      // new tokens (0 where the sequence does not fit)
  bool bad;
};

__device__ __forceinline__ NewSpan new_span(const NewRows& r, int b) {
  NewSpan s;
  const int len = r.seq_lens[b];
  s.row0 = r.cu ? r.cu[b] : b;
  s.n = r.cu ? r.cu[b + 1] - s.row0 : 1;
  s.start = len - s.n;
  s.bad = s.n < 0 || s.row0 < 0 || (long long)s.row0 + s.n > r.total || len < s.n ||
          len > r.max_pages * kPage;  // (start itself may have wrapped around)
  if (s.bad) s.n = 0;
  return s;
}

// Work items over the blocks that new tokens touch: sequence b's begin at item
// cu[b] / 16 + 2 b, which leaves room for every block (n tokens from any slot touch at most
// n / 16 + 2), so an item finds its sequence by bisection and no prefix sum is needed.
__host__ __device__ __forceinline__ int new_block_items(int batch, int total, bool ragged) {
  return ragged ? total / kPage + 2 * batch : batch;
}
__device__ __forceinline__ int item_base(const NewRows& r, int b) {
  return r.cu[b] / kPage + 2 * b;
}
__device__ __forceinline__ int item_sequence(const NewRows& r, int item) {
  int lo = 0, hi = r.batch;  // the last b in [lo, hi) with item_base(b) <= item
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (item_base(r, mid) <= item) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint2 ldg64_nc(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// Code bytes to fp16 pairs, exactly.
//  int8: the byte with its sign bit flipped, u = code + 128, under the byte 0x64 is the fp16
//    number 1024 + u; less 1152 that is the code (a permute and an add a pair).
//  E4M3: the conversion instruction, one a pair (moving the bits by hand, a permute, a shift and
//    two logic operations a pair, made a 128K-token decode 73.5 us instead of 53.5). Its NaN
//    code reads as NaN: callers zero the bytes that no token wrote.
template <int F>
struct Codes;

template <>
struct Codes<kInt8> {
  // to be applied to a word of four codes before `pair`
  static __device__ __forceinline__ uint32_t prepare(uint32_t w) { return w ^ 0x80808080u; }
  // fp16 pair of two of a prepared word's bytes: sel 0x4140 (bytes 0, 1) or 0x4342 (2, 3)
  template <int kHigh>
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    const uint32_t h = prmt(w, 0x64646464u, kHigh ? 0x4342u : 0x4140u);
    const __half2 off = __half2(__ushort_as_half(0xE480), __ushort_as_half(0xE480));  // -1152
    const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&h), off);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

template <>
struct Codes<kE4m3> {
  static __device__ __forceinline__ uint32_t prepare(uint32_t w) { return w; }
  template <int kHigh>
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    uint32_t d;
    if constexpr (kHigh)
      asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;}"
          : "=r"(d)
          : "r"(w));
    else
      asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;}"
          : "=r"(d)
          : "r"(w));
    return d;
  }
};

}  // namespace kv8_detail
}  // namespace hsa
