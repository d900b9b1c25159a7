// kv8.cuh -- what the kernels of the 8-bit K/V cache share: its layout, the rows of new tokens,
// the exact conversions of its codes to fp16 and fp32, and the codes of values.
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
// n / 16 + 2), so an item finds its sequence by a search and no prefix sum is needed.
__host__ __device__ __forceinline__ int new_block_items(int batch, int total, bool ragged) {
  return ragged ? total / kPage + 2 * batch : batch;
}
__device__ __forceinline__ int item_base(const NewRows& r, int b) {
  return r.cu[b] / kPage + 2 * b;
}
// The last b in [0, batch) with first(b) <= key, for ascending first: a warp together, 32 ways a
// step (1024 sequences: two loads one after the other, not ten). -1 where there is none.
template <typename First>
__device__ __forceinline__ int warp_search(int batch, int key, int lane, First first) {
  int lo = 0, n = batch;
  for (;;) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool below = at < n && first(lo + at) <= key;
    const int count = __popc(__ballot_sync(0xffffffffu, below));
    if (count == 0) return -1;
    lo += (count - 1) * step;
    n = min(step, n - (count - 1) * step);
    if (step == 1) return lo;
  }
}

// Up to kFewSequences a bisection by every lane for itself: no load for one sequence, two for four,
// and a smaller kernel (kv8_cache.cu has a form of its own for it).
constexpr int kFewSequences = 4;
__device__ __forceinline__ int item_sequence_of_few(const NewRows& r, int item) {
  int lo = 0, hi = r.batch;  // the last b in [lo, hi) with item_base(b) <= item
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (item_base(r, mid) <= item) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int item_sequence(const NewRows& r, int item, int lane) {
  return warp_search(r.batch, item, lane, [&](int b) { return item_base(r, b); });
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

// One warp behind the units: sequences that do not fit (offsets that lead outside the arrays may
// have no unit at all).
__device__ __forceinline__ void report_bad(const NewRows& rows, int lane, int* err) {
  for (int b = lane; b < rows.batch; b += 32)
    if (new_span(rows, b).bad) set_error(err, kDevErrCheck);
}

template <int F>
__device__ __forceinline__ constexpr float levels() {
  return F == kE4m3 ? 448.0f : 127.0f;
}

// Codes of four values: f32(x * inv) rounded to the format, halves to even. int8: adding
// 1.5 * 2^23 leaves the rounded integer in the low byte (|x * inv| <= 127 (1 + 2^-22)).
template <int F>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  a = __fmul_rn(a, inv);
  b = __fmul_rn(b, inv);
  c = __fmul_rn(c, inv);
  d = __fmul_rn(d, inv);
  if constexpr (F == kInt8) {
    const float magic = 12582912.0f;
    const uint32_t ab = prmt(__float_as_uint(__fadd_rn(a, magic)),
                             __float_as_uint(__fadd_rn(b, magic)), 0x0040u);
    const uint32_t cd = prmt(__float_as_uint(__fadd_rn(c, magic)),
                             __float_as_uint(__fadd_rn(d, magic)), 0x0040u);
    return prmt(ab, cd, 0x5410u);
  } else {
    uint16_t ab, cd;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(ab) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(cd) : "f"(d), "f"(c));
    return (uint32_t)ab | ((uint32_t)cd << 16);
  }
}

// One value with NaN as 0 and infinities at the largest code.
template <int F>
__device__ __forceinline__ float tame(float x, float inv) {
  if (x != x) return 0.0f;
  const float y = __fmul_rn(x, inv);
  if (y != y) return 0.0f;  // infinity under inv = 0
  return fminf(fmaxf(y, -levels<F>()), levels<F>());
}

// Values of four codes (exact).
template <int F>
__device__ __forceinline__ void values4(uint32_t w, float* f) {
  if constexpr (F == kInt8) {
    w ^= 0x80808080u;  // code + 128 under 0x4B is the number 2^23 + 128 + code
#pragma unroll
    for (int i = 0; i < 4; i++)
      f[i] = __fadd_rn(__uint_as_float(prmt(w, 0x4B000000u, 0x7440u + i)), -8388736.0f);
  } else {
    const uint32_t lo = Codes<kE4m3>::pair<0>(w), hi = Codes<kE4m3>::pair<1>(w);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  }
}

}  // namespace kv8_detail
}  // namespace hsa
