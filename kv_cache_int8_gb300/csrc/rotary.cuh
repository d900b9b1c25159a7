// rotary.cuh -- rotary positions on rows of 128 channels: which channels a lane holds, and the
// turn itself. Shared by the rotation of rows (rotary.cu) and the rotated write into the 8-bit
// cache (kv8_draft.cu).
//
// Mathematics (rotary position embedding, Su et al. 2021): channel pair i of a head turns by the
// angle p f_i at position p,
//   y_a = x_a cos - x_b sin      y_b = x_b cos + x_a sin
// with (a, b) = (i, i + dim / 2) or, neighbours, (2 i, 2 i + 1); channels from dim on stay. Every
// product and sum is rounded to fp32 by itself (no fused multiply-add), so that the values that
// are quantised, and with them the codes, are the same wherever they are computed.
#pragma once

#include "common.cuh"

namespace hsa {
namespace rotary_detail {

// cos, then sin, of a position's dim / 2 angles: table [rows][dim].
struct Rotary {
  const float* table;
  int rows, dim;
  const int32_t* positions;  // of every row; nullptr: the token's place in its sequence
};

// 16 lanes share a row of 128 channels. A lane holds two runs of four channels, at `a` and `b`,
// that are made of whole pairs: halves take a run of the first half and its partners (8-byte
// accesses, whole 128-byte lines over the lanes), so no value is exchanged between lanes; lanes
// without angles, and neighbours, take eight channels in a row. Angles 4 j .. 4 j + 3 are lane
// j's in both.
struct Place {
  int a, b;
  bool turns;
};
template <bool kNeighbours>
__device__ __forceinline__ Place place(int j, int dim) {
  Place p;
  p.turns = 8 * j < dim;
  p.a = !kNeighbours && p.turns ? 4 * j : 8 * j;
  p.b = !kNeighbours && p.turns ? 4 * j + dim / 2 : 8 * j + 4;
  return p;
}

struct Angles {
  float4 c, s;
};
__device__ __forceinline__ Angles angles(const Rotary& r, int position, int j) {
  const float* row = r.table + (size_t)position * r.dim + 4 * j;
  return {__ldg(reinterpret_cast<const float4*>(row)),
          __ldg(reinterpret_cast<const float4*>(row + r.dim / 2))};
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float y = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = y;
}

// x[0..3]: channels from `a` on, x[4..7]: from `b` on.
template <bool kNeighbours>
__device__ __forceinline__ void turn(float (&x)[8], const Angles& g) {
  if constexpr (kNeighbours) {
    turn_pair(x[0], x[1], g.c.x, g.s.x);
    turn_pair(x[2], x[3], g.c.y, g.s.y);
    turn_pair(x[4], x[5], g.c.z, g.s.z);
    turn_pair(x[6], x[7], g.c.w, g.s.w);
  } else {
    turn_pair(x[0], x[4], g.c.x, g.s.x);
    turn_pair(x[1], x[5], g.c.y, g.s.y);
    turn_pair(x[2], x[6], g.c.z, g.s.z);
    turn_pair(x[3], x[7], g.c.w, g.s.w);
  }
}

// (not through the read-only path: rows may be turned in place)
__device__ __forceinline__ uint2 load4(const __nv_bfloat16* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void unpack(uint2 u, uint2 v, float (&x)[8]) {
  x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x);
  x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
  x[4] = bf16_lo(v.x); x[5] = bf16_hi(v.x);
  x[6] = bf16_lo(v.y); x[7] = bf16_hi(v.y);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The warp turns heads [h0, h0 + 16) of one row of `heads` heads, two at a time (one a half
// warp), all reads before the first write: rows may be turned in place.
struct RowSide {
  const __nv_bfloat16* x;
  long long x_stride;
  __nv_bfloat16* y;
  long long y_stride;
  int heads;
};
constexpr int kRowHeads = 16;
__host__ __device__ __forceinline__ int row_units(int heads) {
  return (heads + kRowHeads - 1) / kRowHeads;
}
template <bool kNeighbours>
__device__ __forceinline__ void turn_row(const RowSide& r, const Rotary& rot, long long row, int h0,
                                         int position, int lane) {
  const int sub = lane >> 4, j = lane & 15;
  const Place p = place<kNeighbours>(j, rot.dim);
  uint2 u[8], v[8];
  const __nv_bfloat16* x = r.x + row * r.x_stride + (long long)(h0 + sub) * kHeadDim;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    u[i] = v[i] = make_uint2(0u, 0u);
    if (h0 + 2 * i + sub < r.heads) {
      u[i] = load4(x + 2 * i * kHeadDim + p.a);
      v[i] = load4(x + 2 * i * kHeadDim + p.b);
    }
  }
  Angles g = {make_float4(1.0f, 1.0f, 1.0f, 1.0f), make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  if (p.turns) g = angles(rot, position, j);
  __syncwarp();
  __nv_bfloat16* y = r.y + row * r.y_stride + (long long)(h0 + sub) * kHeadDim;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (h0 + 2 * i + sub >= r.heads) continue;
    if (p.turns) {
      float f[8];
      unpack(u[i], v[i], f);
      turn<kNeighbours>(f, g);
      u[i] = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
      v[i] = make_uint2(pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
    *reinterpret_cast<uint2*>(y + 2 * i * kHeadDim + p.a) = u[i];
    *reinterpret_cast<uint2*>(y + 2 * i * kHeadDim + p.b) = v[i];
  }
}

}  // namespace rotary_detail
}  // namespace hsa
