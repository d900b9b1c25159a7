// kv8_draft.cu -- drafted tokens and the 8-bit K/V cache: new tokens written with their rotary
// positions on, and the accepted branch of a drafted tree moved into place.
//
// Source: "KV Cache 与长上下文推理", sections "KV Cache 回顾" (every step appends the new tokens' K
// and V) and "KV Cache 量化"; formulas of the rotation: rotary.cuh. The pages have no drafted
// tokens: a tree of them takes the places behind the context, and of an accepted branch only
// the first child of every node already lies where it belongs.
//
// As in kv8_cache.cu one warp owns one block (page, kv head) of K or of V, 64 values a lane in
// registers between the maximum and the codes, here in fp32: a rotated key is quantised as it is
// computed, not rounded to bf16 in between (that would add 2^-9 of a value to half a code step,
// 2^-8 of the block's largest). The queries of the same tokens turn in the same launch.
#include <type_traits>

#include "internal.h"
#include "kv8.cuh"
#include "rotary.cuh"

namespace hsa {
namespace {

using namespace kv8_detail;
using namespace rotary_detail;

constexpr int kWarps = 8;

// max |x| of three values, NaN if one is
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(m), "f"(a), "f"(b));
  return y;
}

// The codes of one block from its new values: lane l has, of tokens t0 + 2 i + l / 16 (i < N),
// channels a .. a + 3 (x[i][0..3]) and b .. b + 3; slots [first, last) are new, x is zero in the
// others. `codes` points at the block, s_old is its scale (read before: it is one load less on the
// way). kRow: b = a + 4. most(v): the largest of the v of the warps
// that share the block; it orders their reads of the block before their writes.
template <int F, bool kRow, int N, typename Most>
__device__ __forceinline__ void put_block(float (&x)[N][8], int t0, int first, int last,
                                          uint8_t* codes, float s_old, float* scale, int a, int b,
                                          int lane, Most most) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++)
#pragma unroll
    for (int k = 0; k < 8; k += 2) m = max_abs3(m, x[i][k], x[i][k + 1]);
  // as bits, infinities and NaN above every number
  uint32_t top = most(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7FFFFFFFu));
  const bool odd_values = top >= 0x7F800000u;
  if (odd_values) {  // the maximum of the finite ones
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float v = fabsf(x[i][k]);
        if (v <= 3.402823466e38f) m = fmaxf(m, v);
      }
    top = most(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  }
  float s = __fdiv_rn(__uint_as_float(top), levels<F>());
  if (s < 1.17549435e-38f) s = 0.0f;
  if (first > 0) s = fmaxf(s_old, s);
  const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  const int token = t0 + (lane >> 4);  // of i = 0
  uint8_t* const at_a = codes + token * kHeadDim + a;
  uint8_t* const at_b = codes + token * kHeadDim + b;
  auto store = [&](int i, uint32_t lo, uint32_t hi) {
    if constexpr (kRow) {
      *reinterpret_cast<uint2*>(at_a + 2 * i * kHeadDim) = make_uint2(lo, hi);
    } else {
      *reinterpret_cast<uint32_t*>(at_a + 2 * i * kHeadDim) = lo;
      *reinterpret_cast<uint32_t*>(at_b + 2 * i * kHeadDim) = hi;
    }
  };
  if (first > 0 && s > s_old) {  // the older tokens' codes under the larger scale
    const float ratio = __fmul_rn(s_old, inv);
#pragma unroll
    for (int i = 0; i < N; i++) {
      if (token + 2 * i >= first) continue;
      float f[8];
      values4<F>(*reinterpret_cast<const uint32_t*>(at_a + 2 * i * kHeadDim), f);
      values4<F>(*reinterpret_cast<const uint32_t*>(at_b + 2 * i * kHeadDim), f + 4);
      store(i, codes4<F>(f[0], f[1], f[2], f[3], ratio), codes4<F>(f[4], f[5], f[6], f[7], ratio));
    }
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    const int slot = token + 2 * i;
    if (slot < first || slot >= last) continue;
    float by = inv;
    if (odd_values) {
#pragma unroll
      for (int k = 0; k < 8; k++) x[i][k] = tame<F>(x[i][k], inv);
      by = 1.0f;
    }
    store(i, codes4<F>(x[i][0], x[i][1], x[i][2], x[i][3], by),
          codes4<F>(x[i][4], x[i][5], x[i][6], x[i][7], by));
  }
  if (lane == 0 && t0 == 0) *scale = s;
}

struct WriteSide {
  const __nv_bfloat16* x;  // rows
  long long stride;        // elements
  uint8_t* codes;
  float* scale;
};

// Units: blocks x kv heads (or runs of `heads` of them) x halves, then (row, 16 query heads); one warp
// behind them reports sequences that do not fit. Two warps share a block of K and of V, eight tokens
// each, and meet over its maxima. Bound by memory: 108K new tokens of 32 + 8 heads (2.47 GB) take
// 390 us, 6.3 TB/s; one token 2.9 us, latency.
//
// A unit's way to its data (sequence, length, page, rows) is four loads one after the other. Where
// there are many blocks a warp goes it once for several kv heads (kMany); the positions' angles then
// come out of L1 (in registers they cost 32 and 2% of the time). One head a unit against four and
// eight: 4096 tokens of 8 heads with their read-back 22.6, 26.8, 40.7 us, 8192 46.8, 39.5, 47.7, 24000
// 132.5, 117.7, 114.6, 108K 541, 495, 491; so as many heads as leave 1024 runs (2048 warps, 13 an
// SM). kSplit: units of K and of V apart, for a token a sequence of few sequences, where the one
// behind the other only takes longer (one sequence of 8 kv heads 2.9 us a call, not 3.4; 256
// sequences 8.1, not 6.3, as the warps no longer fit the GPU at once). Both hold for 1, 2 and 4 kv
// heads too: 8 x 4096 tokens 25.5, 37.2, 62 us (one head a unit 25.5, 38, 67.5; hkv heads wherever 64
// runs are left: 4096 tokens of 2 and 4 heads 8.6 and 15.4 us, not 5.6 and 8.4); one sequence 3.2 to
// 3.3 us apart and 3.5 to 3.9 together, 1024, 1024 and 512 sequences 4.3, 6.4 and 6.6 together, 5.6,
// 8.0 and 8.0 apart.
constexpr int kBlocksAHead = 1024;
constexpr int kSplitUnits = 2048;  // 13 warps an SM, of 24
template <int F, bool kNeighbours, bool kSplit, bool kMany>
__global__ void __launch_bounds__(kWarps * 32, 3)
    kv8_write_rotated_kernel(const NewRows rows, const Rotary rot, const WriteSide ks,
                             const WriteSide vs, const RowSide qs,
                             const int32_t* __restrict__ page_table, int hkv, int heads,
                             int num_pages, int block_units, int units, int* err) {
  __shared__ uint32_t tops[4][kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + warp;
  if (unit == units) report_bad(rows, lane, err);
  if (unit >= units) return;
  if (unit >= block_units) {  // queries
    const int per = row_units(qs.heads);
    const int row = (unit - block_units) / per, part = (unit - block_units) % per;
    const int b = rows.cu ? warp_search(rows.batch, row, lane, [&](int i) { return rows.cu[i]; })
                          : row;
    if (b < 0) return;
    const NewSpan sp = new_span(rows, b);
    if (row < sp.row0 || row - sp.row0 >= sp.n) return;
    const int position = rot.positions ? rot.positions[row] : sp.start + (row - sp.row0);
    if (position < 0 || position >= rot.rows) {
      if (lane == 0) set_error(err, kDevErrCheck);
      return;
    }
    turn_row<kNeighbours>(qs, rot, row, part * kRowHeads, position, lane);
    return;
  }
  const int t0 = 8 * (unit & 1);
  const int pair = kSplit ? unit >> 2 : unit >> 1, groups = kMany ? (hkv + heads - 1) / heads : hkv;
  const int h0 = kMany ? pair % groups * heads : pair % groups, item = pair / groups;
  const bool do_k = !kSplit || !(unit & 2), do_v = !kSplit || (unit & 2);
  const int b = rows.cu ? item_sequence(rows, item, lane) : item;
  if (b < 0) return;
  const NewSpan sp = new_span(rows, b);
  const int j = rows.cu ? item - item_base(rows, b) : 0;
  const int end = sp.start + sp.n;  // N_b
  const long long p = (long long)sp.start / kPage + j;
  if (sp.n == 0 || j < 0 || p * kPage >= end) return;
  const int page = page_table[(size_t)b * rows.max_pages + p];
  const int base = (int)p * kPage;
  const int first = max(sp.start - base, 0), last = min(end - base, kPage);
  const long long row = (long long)sp.row0 + base - sp.start;  // of slot 0
  // lane l: position of slot l
  int position = base + lane;
  bool bad = page < 0 || page >= num_pages;
  if (lane >= first && lane < last) {
    if (rot.positions) position = rot.positions[row + lane];
    bad = bad || position < 0 || position >= rot.rows;
  }
  if (__any_sync(0xffffffffu, bad)) {  // (both warps of a block alike)
    if (lane == 0) set_error(err, kDevErrCheck);
    return;
  }
  int turn_of = 0;
  auto most = [&](uint32_t v) {  // of the block's two warps
    const int at = turn_of++ & 3;
    if (lane == 0) tops[at][warp] = v;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp >> 1)) : "memory");
    return max(v, tops[at][warp ^ 1]);
  };
  const int token = t0 + (lane >> 4), l16 = lane & 15;
  const Place pl = place<kNeighbours>(l16, rot.dim);
  const int h1 = kMany ? min(h0 + heads, hkv) : h0 + 1;
#pragma unroll 1
  for (int h = h0; h < h1; h++) {
    const size_t block = (size_t)page * hkv + h;
    const float k_old = first > 0 ? __ldcg(ks.scale + block) : 0.0f;
    const float v_old = first > 0 ? __ldcg(vs.scale + block) : 0.0f;
    const __nv_bfloat16* k_src = ks.x + (row + token) * ks.stride + h * kHeadDim;
    const __nv_bfloat16* v_src = vs.x + (row + token) * vs.stride + h * kHeadDim + 8 * l16;
    uint2 u[4], v[4];
    uint4 raw[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int slot = token + 2 * i;
      u[i] = v[i] = make_uint2(0u, 0u);
      if (do_k && slot >= first && slot < last) {
        u[i] = load4(k_src + 2 * i * ks.stride + pl.a);
        v[i] = load4(k_src + 2 * i * ks.stride + pl.b);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int slot = token + 2 * i;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (do_v && slot >= first && slot < last) raw[i] = ldg128_nc(v_src + 2 * i * vs.stride);
    }
    float x[4][8];
    if (do_k) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int slot = token + 2 * i;
        const int at = __shfl_sync(0xffffffffu, position, slot);
        unpack(u[i], v[i], x[i]);
        if (pl.turns && slot >= first && slot < last) turn<kNeighbours>(x[i], angles(rot, at, l16));
      }
      put_block<F, kNeighbours>(x, t0, first, last, ks.codes + block * kBlockBytesI8, k_old,
                                ks.scale + block, pl.a, pl.b, lane, most);
    }
    if (!do_v) continue;
#pragma unroll
    for (int i = 0; i < 4; i++)
      unpack(make_uint2(raw[i].x, raw[i].y), make_uint2(raw[i].z, raw[i].w), x[i]);
    put_block<F, true>(x, t0, first, last, vs.codes + block * kBlockBytesI8, v_old,
                       vs.scale + block, 8 * l16, 8 * l16 + 4, lane, most);
  }
}

// ------------------------------------------------------------- the accepted branch into place
//
// A warp has one (sequence, kv head) of K or of V and goes through the blocks that receive kept
// tokens, first to last: node idx_j moves from place start + idx_j to start + j, never upwards,
// so what a block receives lies in itself or behind it, where this warp has not written yet.
// Latency counts (a branch is a few tokens): lengths, indices, pages and codes are four loads one
// after the other. One branch of 8 kv heads 3.3 us, 256 branches of 0 to 8 tokens 7.8 us. Three CTAs
// an SM leave 80 registers a thread, and some 190 bytes are spilled; with two there are none (one
// branch 2.9 us, 256 the same), with four 3.5 and 9.2 us.
struct KeepArgs {
  NewRows rows;
  const int32_t* idx;  // [batch][stride]
  const int32_t* count;
  int stride;
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  int32_t* new_lens;
  int hkv, num_pages;
  int* err;
};

template <int F>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_keep_kernel(const KeepArgs p) {
  grid_dep_wait();
  grid_dep_launch();
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= p.rows.batch * p.hkv * 2) return;
  const int b = unit / (2 * p.hkv), h = unit / 2 % p.hkv, side = unit & 1;
  const int m = p.count[b];
  const int32_t* idx = p.idx + (size_t)b * p.stride;
  // an index is asked for before it is known to count: the row has `stride` of them
  int node = lane < p.stride ? idx[lane] : -1;
  const NewSpan sp = new_span(p.rows, b);
  const int32_t* table = p.page_table + (size_t)b * p.rows.max_pages;
  auto page_ok = [&](int pos) {
    const int page = table[pos / kPage];
    return page >= 0 && page < p.num_pages;
  };
  bool bad = sp.bad || m < 0 || m > sp.n || m > p.stride;
  if (!bad) {  // every index and page, before anything is written
    for (int j0 = 0; j0 < m; j0 += 32) {
      const int j = j0 + lane;
      if (j < m) {
        const int i = j0 == 0 ? node : idx[j];
        const int before = j == 0 ? -1 : idx[j - 1];
        bad = bad || i <= before || i >= sp.n;
        if (!bad) bad = !page_ok(sp.start + i) || !page_ok(sp.start + j);
      }
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad && lane == 0) set_error(p.err, kDevErrCheck);
  if (p.new_lens != nullptr && h == 0 && side == 0 && lane == 0)
    p.new_lens[b] = bad ? p.rows.seq_lens[b] : sp.start + m;
  if (bad || m == 0) return;
  uint8_t* const codes = side ? p.v : p.k;
  float* const scale = side ? p.v_scale : p.k_scale;
  const int sub = lane >> 4, l16 = lane & 15;
  const int end = sp.start + m;
  for (int base = sp.start / kPage * kPage; base < end; base += kPage) {
    const int first = max(sp.start - base, 0), last = min(end - base, kPage);
    // lane l: where slot l comes from, and its scale
    long long from = 0;
    float s = 0.0f;
    if (lane >= first && lane < last) {
      const int src = sp.start + idx[base + lane - sp.start];
      const size_t block = (size_t)table[src / kPage] * p.hkv + h;
      from = (long long)block * kBlockBytesI8 + src % kPage * kHeadDim;
      s = __ldcg(scale + block);
    }
    const size_t to = (size_t)table[base / kPage] * p.hkv + h;
    const float s_old = first > 0 ? __ldcg(scale + to) : 0.0f;
    uint2 raw[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int slot = 2 * i + sub;
      const long long at = __shfl_sync(0xffffffffu, from, slot);
      raw[i] = make_uint2(0u, 0u);
      if (slot >= first && slot < last)
        raw[i] = __ldcg(reinterpret_cast<const uint2*>(codes + at) + l16);
    }
    float x[8][8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int slot = 2 * i + sub;
      const float by = __shfl_sync(0xffffffffu, s, slot);
      values4<F>(raw[i].x, x[i]);
      values4<F>(raw[i].y, x[i] + 4);
#pragma unroll
      for (int k = 0; k < 8; k++)
        x[i][k] = slot >= first && slot < last ? __fmul_rn(x[i][k], by) : 0.0f;
    }
    // (the maximum over the lanes orders all their reads before the first write)
    put_block<F, true>(x, 0, first, last, codes + to * kBlockBytesI8, s_old, scale + to, 8 * l16,
                       8 * l16 + 4, lane, [](uint32_t v) { return v; });
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_kv8_write_rotated(const Shape& s, const Kv8& c, const RotaryTable& t,
                                     const void* q, long long q_stride, void* q_out,
                                     long long q_out_stride, const void* k_new, long long k_stride,
                                     const void* v_new, long long v_stride,
                                     const int32_t* positions, const int32_t* cu, int total,
                                     const int32_t* page_table, const int32_t* seq_lens, int* err,
                                     cudaStream_t st) {
  const NewRows rows = {cu, seq_lens, s.batch, total, s.max_pages};
  const Rotary rot = {t.table, t.rows, t.dim, positions};
  const WriteSide ks = {static_cast<const __nv_bfloat16*>(k_new), k_stride,
                        static_cast<uint8_t*>(c.k), c.k_scale};
  const WriteSide vs = {static_cast<const __nv_bfloat16*>(v_new), v_stride,
                        static_cast<uint8_t*>(c.v), c.v_scale};
  const RowSide qs = {static_cast<const __nv_bfloat16*>(q), q_stride,
                      static_cast<__nv_bfloat16*>(q_out), q_out_stride, q ? s.hq : 0};
  const bool split = cu == nullptr && s.batch * s.hkv * 4 <= kSplitUnits;
  const int items = new_block_items(s.batch, total, cu != nullptr);
  const long long full = (long long)total / kPage * s.hkv;  // about as many blocks
  const int heads = (int)std::min(std::max(full / kBlocksAHead, 1ll), (long long)s.hkv);
  const int block_units = items * ((s.hkv + heads - 1) / heads) * (split ? 4 : 2);
  const int units = block_units + total * row_units(qs.heads);
  auto pick = [&](auto format) {
    constexpr int kF = decltype(format)::value;
    if (split)
      return t.neighbours ? kv8_write_rotated_kernel<kF, true, true, false>
                          : kv8_write_rotated_kernel<kF, false, true, false>;
    if (heads > 1)
      return t.neighbours ? kv8_write_rotated_kernel<kF, true, false, true>
                          : kv8_write_rotated_kernel<kF, false, false, true>;
    return t.neighbours ? kv8_write_rotated_kernel<kF, true, false, false>
                        : kv8_write_rotated_kernel<kF, false, false, false>;
  };
  auto kernel = c.format == kE4m3 ? pick(std::integral_constant<int, kE4m3>{})
                                  : pick(std::integral_constant<int, kInt8>{});
  return launch_kernel(kernel, dim3(units / kWarps + 1), dim3(kWarps * 32), 0, st, true, rows, rot,
                       ks, vs, qs, page_table, s.hkv, heads, s.num_pages, block_units, units, err);
}

cudaError_t launch_kv8_keep(const Shape& s, const Kv8& c, const int32_t* keep_idx, int keep_stride,
                            const int32_t* n_keep, const int32_t* cu, const int32_t* page_table,
                            const int32_t* seq_lens, int32_t* new_lens, int* err,
                            cudaStream_t st) {
  KeepArgs p;
  p.rows = NewRows{cu, seq_lens, s.batch, INT32_MAX, s.max_pages};
  p.idx = keep_idx;
  p.count = n_keep;
  p.stride = keep_stride;
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.page_table = page_table;
  p.new_lens = new_lens;
  p.hkv = s.hkv;
  p.num_pages = s.num_pages;
  p.err = err;
  const int units = s.batch * s.hkv * 2;
  auto kernel = c.format == kE4m3 ? kv8_keep_kernel<kE4m3> : kv8_keep_kernel<kInt8>;
  return launch_kernel(kernel, dim3((units + kWarps - 1) / kWarps), dim3(kWarps * 32), 0, st, true,
                       p);
}

}  // namespace hsa
