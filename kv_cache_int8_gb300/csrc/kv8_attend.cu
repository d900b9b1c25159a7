// kv8_attend.cu -- decode attention over the 8-bit K/V cache: one query token a sequence over
// every token (dense) or over the sink, the window and a list of kept blocks.
//
// Source: "KV Cache 与长上下文推理", section "KV Cache 回顾" (decode attention equation), section
// "KV Cache 量化"; the attended set is hsa_attend's.
//
// Mathematics. A block of 16 tokens has codes a_t, c_t (K, V) and scales s_k, s_v:
//   x_tj = (sm_scale log2 e s_k) q_j . a_t     out_j = sum_t 2^(x_tj - m) s_v c_t / sum_t 2^(..)
// Both products run on the matrix pipe with fp16 operands and fp32 sums, and nothing is rounded
// that matters: the codes are exact in fp16; a head's query is multiplied by the power of two
// that puts its largest value in [2^13, 2^14), which makes every bf16 value down to 2^-27 of
// that one exact in fp16; a probability p is split into fp16 hi + lo, 22 bits together (p is
// carried 2^6 larger than 2^(x - m), and m may lag the maximum by up to 2^8, so p stays below
// 2^14). The scales multiply the fp32 results, a block at a time.
//
// Layout. K's block is the left operand [16 tokens][128 channels], the group's heads (up to 8)
// the 8 columns of m16n8k16; V's block enters transposed, 8 tiles of 16 channels. So a group of
// 8 heads wastes no product, and scores, probabilities and outputs keep one layout: a lane has
// heads 2t, 2t + 1. Which channel a product's k index stands for is free as long as both sides
// agree: a lane takes whole 16-byte chunks, and the 128-byte swizzle of the tensor copies makes
// all its reads free of bank conflicts.
//
// Work. Memory bound: a block's 4 KiB cost an SM about 175 cycles at the HBM rate, the products
// a third of that. Every warp streams its own blocks through its own ring of tensor copies
// (kStages blocks of K and V), no barriers between warps. All blocks of all rows (sequence, kv
// head) form one line that is cut into equal slices, one a CTA, so ragged batches balance
// without the host knowing any length; where a slice ends inside a row, the row's parts meet in
// the workspace and the last CTA to arrive joins them in slice order (the result does not
// depend on which one that is).
#include "kv8.cuh"

#include <cmath>

namespace hsa {
namespace {

using namespace kv8_detail;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kUnitBytes = 2 * kBlockBytesI8;  // K block, then V block
constexpr int kMinUnits = kWarps;              // smallest slice: one block a warp
constexpr int kTile = 8 * kHeadDim;            // output values of a row (8 heads)
constexpr float kHeadroom = 6.0f;              // p is 2^(x - m + kHeadroom)
constexpr float kLag = 8.0f;                   // m follows a maximum that is this much larger

struct Params {
  const __nv_bfloat16* q;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_idx;  // kept blocks
  const int32_t* n_blocks;
  float* out;
  float* lse;
  float* part_ml;  // [2 CTAs][8 heads] (m, l)
  float* part_o;   // [2 CTAs][kTile]
  int* counters;   // [batch][rows]
  int* err;
  int batch, hq, hkv, rows, group, kv_div, max_pages, num_pages, sink, window, k2;
  float scale_log2;  // sm_scale log2 e
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Units (blocks to visit) of a row of a sequence of n tokens. Kept form: the sink's blocks, the
// window's, then k2 places for kept blocks.
template <bool kKept>
__device__ __forceinline__ int row_units(const Params& p, int n) {
  if (n <= 0) return 0;
  if (!kKept) return (n + kPage - 1) / kPage;
  const int head = min(p.sink, n), tail = max(n - p.window, head);
  return (head + kPage - 1) / kPage + ((n + kPage - 1) / kPage - tail / kPage) * (tail < n) +
         p.k2;
}

// One visit: the block's first row in the code arrays, its slots [lo, hi), its scales.
struct Unit {
  int y;
  int span;  // lo | hi << 8; 0: nothing to do
  float sk, sv;
};

template <bool kKept>
__device__ __forceinline__ Unit locate(const Params& p, const long long* pre, const int* lens,
                                       long long x) {
  int lo_b = 0, hi_b = p.batch;  // the sequence with pre[b] <= x < pre[b + 1]
  while (hi_b - lo_b > 1) {
    const int mid = (lo_b + hi_b) >> 1;
    if (pre[mid] <= x) lo_b = mid;
    else hi_b = mid;
  }
  const int b = lo_b, n = lens[b];
  const unsigned u = row_units<kKept>(p, n);
  const unsigned at = (unsigned)(x - pre[b]);
  const int row = at / u, i = at % u;
  int pg = i, lo = 0, hi = n;  // token range
  if (kKept) {
    const int head = min(p.sink, n), tail = max(n - p.window, head);
    const int ns = (head + kPage - 1) / kPage;
    const int nw = tail < n ? (n + kPage - 1) / kPage - tail / kPage : 0;
    if (i < ns) {
      hi = head;
    } else if (i < ns + nw) {
      pg = tail / kPage + i - ns;
      lo = tail;
    } else {
      const int k = i - ns - nw;
      const size_t r = (size_t)b * p.rows + row;
      pg = k < p.n_blocks[r] ? p.block_idx[r * p.k2 + k] : -1;
      lo = p.sink;
      hi = n - p.window;
    }
  }
  Unit t = {0, 0, 0.0f, 0.0f};
  if (pg < 0 || pg >= p.max_pages) return t;
  lo = max(lo - pg * kPage, 0);
  hi = min(hi - pg * kPage, kPage);
  if (hi <= lo) return t;
  const int page = p.page_table[(size_t)b * p.max_pages + pg];
  if (page < 0 || page >= p.num_pages) {
    set_error(p.err, kDevErrCheck);
    return t;
  }
  const int block = page * p.hkv + row / p.kv_div;
  t.y = block * kPage;
  t.span = lo | (hi << 8);
  t.sk = p.k_scale[block];
  t.sv = p.v_scale[block];
  return t;
}

struct Smem {
  alignas(1024) unsigned char ring[kWarps][kStages][kUnitBytes];
  float4 o[kWarps][8][32];  // the warps' outputs: [channel tile][lane]
  float ml[kWarps][8][2];
  float total[8][2];  // a joined row's (m, l)
  alignas(8) uint64_t full[kWarps][kStages];
  long long warp_sum[kWarps];
  int last;
};
// behind it: pre (long long [batch + 1]), lens (int [batch])

template <int F, bool kKept>
__global__ void __launch_bounds__(kThreads, 2)
    kv8_attend_kernel(const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const Params p) {
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  long long* pre = reinterpret_cast<long long*>(&sm + 1);
  int* lens = reinterpret_cast<int*>(pre + p.batch + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  // ---- the line of all units and this CTA's slice of it
  const int per_thread = (p.batch + kThreads - 1) / kThreads;
  long long sum = 0;
  for (int k = 0; k < per_thread; k++) {
    const int b = tid * per_thread + k;
    if (b >= p.batch) break;
    int n = p.seq_lens[b];
    if (n < 0 || n > p.max_pages * kPage) {
      set_error(p.err, kDevErrCheck);
      n = 0;
    }
    lens[b] = n;
    sum += (long long)row_units<kKept>(p, n) * p.rows;
  }
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  if (lane < kStages) mbar_init(&sm.full[warp][lane], 1);
  if (tid == 0) {
    tma_prefetch_descriptor(&k_map);
    tma_prefetch_descriptor(&v_map);
  }
  fence_barrier_init();
  __syncthreads();
  {
    long long before = incl - sum;
    for (int w = 0; w < warp; w++) before += sm.warp_sum[w];
    for (int k = 0; k < per_thread; k++) {
      const int b = tid * per_thread + k;
      if (b >= p.batch) break;
      pre[b] = before;
      before += (long long)row_units<kKept>(p, lens[b]) * p.rows;
      if (b == p.batch - 1) pre[p.batch] = before;
    }
  }
  __syncthreads();
  const long long all = pre[p.batch];
  const long long per = max((all + gridDim.x - 1) / gridDim.x, (long long)kMinUnits);
  const long long begin = min(blockIdx.x * per, all), end = min(begin + per, all);

  // rows of no units at all
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (pre[b + 1] != pre[b]) continue;
    for (int i = tid; i < p.hq * kHeadDim; i += kThreads)
      p.out[(size_t)b * p.hq * kHeadDim + i] = 0.0f;
    if (p.lse != nullptr)
      for (int i = tid; i < p.hq; i += kThreads) p.lse[(size_t)b * p.hq + i] = -INFINITY;
  }
  if (begin >= end) return;

  // ---- this warp's units: begin + warp + kWarps i; lane l holds those of i = 32 k + l
  const long long x0 = begin + warp;
  const int mine = x0 < end ? (int)((end - x0 + kWarps - 1) / kWarps) : 0;
  auto fetch = [&](int i0) {
    const long long x = x0 + (long long)kWarps * (i0 + lane);
    Unit u = {0, 0, 0.0f, 0.0f};
    if (x < end) u = locate<kKept>(p, pre, lens, x);
    return u;
  };
  Unit cur = fetch(0), next = mine > 32 ? fetch(32) : Unit{0, 0, 0.0f, 0.0f};
  const uint64_t policy = l2_evict_first_policy();
  int issued = 0, taken = 0;  // copies begun and waited for
  bool dead = false;
  auto issue = [&](int i, int batch0) {
    if (i >= mine) return;
    const bool ahead = (i >> 5) != batch0;
    const int span = __shfl_sync(0xffffffffu, ahead ? next.span : cur.span, i & 31);
    const int y = __shfl_sync(0xffffffffu, ahead ? next.y : cur.y, i & 31);
    if (span == 0 || dead) return;
    if (lane == 0) {
      const int st = issued % kStages;
      unsigned char* dst = sm.ring[warp][st];
      mbar_arrive_expect_tx(&sm.full[warp][st], kUnitBytes);
      tma_load_2d_hint(dst, &k_map, 0, y, &sm.full[warp][st], policy);
      tma_load_2d_hint(dst + kBlockBytesI8, &v_map, 0, y, &sm.full[warp][st], policy);
    }
    issued++;
  };
#pragma unroll
  for (int i = 0; i < kStages; i++) issue(i, 0);

  int i = 0;
  for (long long x = begin; x < end;) {
    // ---- the row at x, and how far this slice goes in it
    int lo_b = 0, hi_b = p.batch;
    while (hi_b - lo_b > 1) {
      const int mid = (lo_b + hi_b) >> 1;
      if (pre[mid] <= x) lo_b = mid;
      else hi_b = mid;
    }
    const int b = lo_b;
    const unsigned units = row_units<kKept>(p, lens[b]);
    const int row = (int)((unsigned)(x - pre[b]) / units);
    const long long row_begin = pre[b] + (long long)row * units, row_end = row_begin + units;
    const long long stop = min(row_end, end);

    // ---- the query as right operands: head g, channels of chunk 2t + c, word w
    uint32_t qf[16];
    float f0, f1;  // factors of heads 2t, 2t + 1
    {
      uint4 raw[4];
#pragma unroll
      for (int c = 0; c < 4; c++) raw[c] = make_uint4(0u, 0u, 0u, 0u);
      if (g < p.group) {
        const __nv_bfloat16* q =
            p.q + ((size_t)b * p.hq + (size_t)row * p.group + g) * kHeadDim + t * 32;
#pragma unroll
        for (int c = 0; c < 4; c++) raw[c] = *reinterpret_cast<const uint4*>(q + c * 8);
      }
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        mx = __vmaxu2(mx, __vmaxu2(raw[c].x & 0x7FFF7FFFu, raw[c].y & 0x7FFF7FFFu));
        mx = __vmaxu2(mx, __vmaxu2(raw[c].z & 0x7FFF7FFFu, raw[c].w & 0x7FFF7FFFu));
      }
      uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
      m16 = max(m16, __shfl_xor_sync(0xffffffffu, m16, 1));
      m16 = max(m16, __shfl_xor_sync(0xffffffffu, m16, 2));
      const int e = m16 >> 7;  // biased exponent of the largest magnitude
      const int shift = (m16 == 0 || e == 255) ? 0 : min(13 + 127 - e, 126);
      const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
      const float down = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int k = 0; k < 4; k++)
          qf[c * 4 + k] = half_pair(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
      }
      const float f = p.scale_log2 * Codes<F>::kUnit * down;
      f0 = __shfl_sync(0xffffffffu, f, (2 * t) * 4);
      f1 = __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4);
    }

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    float o[8][4];
#pragma unroll
    for (int k = 0; k < 8; k++)
#pragma unroll
      for (int c = 0; c < 4; c++) o[k][c] = 0.0f;

    for (; i < mine && x0 + (long long)kWarps * i < stop; i++) {
      if (i > 0 && (i & 31) == 0) {
        cur = next;
        next = fetch(i + 32);
      }
      const int src = i & 31;
      const int span = __shfl_sync(0xffffffffu, cur.span, src);
      if (span != 0 && !dead) {
        const float sk = __shfl_sync(0xffffffffu, cur.sk, src);
        const float sv = __shfl_sync(0xffffffffu, cur.sv, src) * Codes<F>::kUnit;
        const int st = taken % kStages;
        if (!mbar_wait(&sm.full[warp][st], (taken / kStages) & 1)) {
          set_error(p.err, kDevErrTimeout);
          dead = true;
        }
        taken++;
        const uint32_t kb = smem_addr(sm.ring[warp][st]), vb = kb + kBlockBytesI8;
        // scores of tokens g and g + 8
        float sa[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const uint32_t at = kb + g * kHeadDim + (((2 * t + c) ^ g) << 4);
          const uint4 ka = lds128(at), kc = lds128(at + 8 * kHeadDim);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
          for (int w = 0; w < 4; w++) {
            const uint32_t a = Codes<F>::prepare(wa[w]), d = Codes<F>::prepare(wc[w]);
            mma16816(w & 1 ? sb : sa, Codes<F>::template pair<0>(a),
                     Codes<F>::template pair<0>(d), Codes<F>::template pair<1>(a),
                     Codes<F>::template pair<1>(d), qf[c * 8 + w * 2], qf[c * 8 + w * 2 + 1]);
          }
        }
        const float g0 = f0 * sk, g1 = f1 * sk;
        float x00 = (sa[0] + sb[0]) * g0, x01 = (sa[1] + sb[1]) * g1;  // token g
        float x10 = (sa[2] + sb[2]) * g0, x11 = (sa[3] + sb[3]) * g1;  // token g + 8
        if (span != (kPage << 8)) {
          const int lo = span & 255, hi = span >> 8;
          if (g < lo || g >= hi) x00 = x01 = -INFINITY;
          if (g + 8 < lo || g + 8 >= hi) x10 = x11 = -INFINITY;
        }
        float n0 = fmaxf(x00, x10), n1 = fmaxf(x01, x11);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, d));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, d));
        }
        if (__any_sync(0xffffffffu, n0 > m0 + kLag || n1 > m1 + kLag)) {
          n0 = fmaxf(n0, m0);
          n1 = fmaxf(n1, m1);
          const float a0 = ex2(m0 - n0), a1 = ex2(m1 - n1);  // 0 from -inf: n is finite
          m0 = n0;
          m1 = n1;
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int k = 0; k < 8; k++) {
            o[k][0] *= a0;
            o[k][1] *= a1;
            o[k][2] *= a0;
            o[k][3] *= a1;
          }
        }
        const float p00 = ex2(x00 - m0 + kHeadroom), p01 = ex2(x01 - m1 + kHeadroom);
        const float p10 = ex2(x10 - m0 + kHeadroom), p11 = ex2(x11 - m1 + kHeadroom);
        l0 += p00 + p10;
        l1 += p01 + p11;
        const uint32_t ha = half_pair(p00, p01), hb = half_pair(p10, p11);
        const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&ha));
        const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&hb));
        const uint32_t b0 = transpose8x8(ha), b1 = transpose8x8(hb);
        const uint32_t r0 = transpose8x8(half_pair(p00 - fa.x, p01 - fa.y));
        const uint32_t r1 = transpose8x8(half_pair(p10 - fb.x, p11 - fb.y));
        // values: tokens 2t, 2t + 1, 2t + 8, 2t + 9 of channels [16 g, 16 g + 16)
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const int tok = 2 * t + (k & 1) + 8 * (k >> 1);
          v[k] = lds128(vb + tok * kHeadDim + ((g ^ (tok & 7)) << 4));
        }
        auto word = [](const uint4& u, int w) {
          return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w;
        };
#pragma unroll
        for (int w = 0; w < 4; w++) {
          const uint32_t ta = word(v[0], w), tb = word(v[1], w);
          const uint32_t tc = word(v[2], w), td = word(v[3], w);
#pragma unroll
          for (int half = 0; half < 2; half++) {  // channels 4 w + 2 half + {0, 1}
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            const uint32_t ab = Codes<F>::prepare(prmt(ta, tb, sel));
            const uint32_t cd = Codes<F>::prepare(prmt(tc, td, sel));
            const uint32_t a0 = Codes<F>::template pair<0>(ab);
            const uint32_t a1 = Codes<F>::template pair<1>(ab);
            const uint32_t a2 = Codes<F>::template pair<0>(cd);
            const uint32_t a3 = Codes<F>::template pair<1>(cd);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16816(acc, a0, a1, a2, a3, b0, b1);
            mma16816(acc, a0, a1, a2, a3, r0, r1);
#pragma unroll
            for (int c = 0; c < 4; c++) o[2 * w + half][c] += sv * acc[c];
          }
        }
        __syncwarp();  // the slot is read before it is filled again
      }
      issue(i + kStages, i >> 5);
    }

    // ---- the warps' parts of the row meet
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (g == 0) {
      sm.ml[warp][2 * t][0] = m0;
      sm.ml[warp][2 * t][1] = l0;
      sm.ml[warp][2 * t + 1][0] = m1;
      sm.ml[warp][2 * t + 1][1] = l1;
    }
#pragma unroll
    for (int k = 0; k < 8; k++) sm.o[warp][k][lane] = make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
    __syncthreads();
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float ma = -INFINITY, mb = -INFINITY, la = 0.0f, lb = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      ma = fmaxf(ma, sm.ml[w][2 * t][0]);
      mb = fmaxf(mb, sm.ml[w][2 * t + 1][0]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      const float wa = sm.ml[w][2 * t][0], wb = sm.ml[w][2 * t + 1][0];
      const float fa = wa == -INFINITY ? 0.0f : ex2(wa - ma);
      const float fb = wb == -INFINITY ? 0.0f : ex2(wb - mb);
      la += fa * sm.ml[w][2 * t][1];
      lb += fb * sm.ml[w][2 * t + 1][1];
      const float4 v = sm.o[w][warp][lane];
      acc.x += fa * v.x;
      acc.y += fb * v.y;
      acc.z += fa * v.z;
      acc.w += fb * v.w;
    }
    bool write = true;
    if (row_begin < begin || row_end > end) {  // a part of the row: to the workspace
      const long long c0 = row_begin / per, c1 = (row_end - 1) / per;
      const size_t slot = 2 * (size_t)blockIdx.x + (begin < row_begin ? 1 : 0);
      reinterpret_cast<float4*>(p.part_o + slot * kTile)[warp * 32 + lane] = acc;
      if (warp == 0 && g == 0)
        reinterpret_cast<float4*>(p.part_ml + slot * 16)[t] = make_float4(ma, la, mb, lb);
      __threadfence();
      __syncthreads();
      const int parts = (int)(c1 - c0) + 1;
      if (tid == 0) {
        int* counter = p.counters + (size_t)b * p.rows + row;
        const int last = atomic_add_acq_rel_gpu(counter, 1) == parts - 1;
        if (last) *counter = 0;
        sm.last = last;
      }
      __syncthreads();
      write = sm.last != 0;
      if (write) {
        // head `warp` of every part: its weight against the joint maximum
        float* weight = reinterpret_cast<float*>(sm.o);  // [parts][8]
        auto slot_of = [&](int c) {
          return 2 * (size_t)(c0 + c) + ((c0 + c) * per < row_begin ? 1 : 0);
        };
        float top = -INFINITY;
        for (int c = lane; c < parts; c += 32)
          top = fmaxf(top, __ldcg(p.part_ml + slot_of(c) * 16 + warp * 2));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float l = 0.0f;
        for (int c = lane; c < parts; c += 32) {
          const float2 v =
              __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot_of(c) * 16 + warp * 2));
          const float f = v.x == -INFINITY ? 0.0f : ex2(v.x - top);
          weight[c * 8 + warp] = f;
          l += f * v.y;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) {
          sm.total[warp][0] = top;
          sm.total[warp][1] = l;
        }
        __syncthreads();
        ma = sm.total[2 * t][0];
        la = sm.total[2 * t][1];
        mb = sm.total[2 * t + 1][0];
        lb = sm.total[2 * t + 1][1];
        acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int c = 0; c < parts; c++) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot_of(c) * kTile) +
                                  warp * 32 + lane);
          const float fa = weight[c * 8 + 2 * t], fb = weight[c * 8 + 2 * t + 1];
          acc.x += fa * v.x;
          acc.y += fb * v.y;
          acc.z += fa * v.z;
          acc.w += fb * v.w;
        }
      }
    }
    if (write) {
      // tile `warp`: channels 16 g + 2 warp + {0, 1} of heads 2t (x, z) and 2t + 1 (y, w)
      const size_t head = (size_t)b * p.hq + (size_t)row * p.group + 2 * t;
      const int ch = 16 * g + 2 * warp;
      if (2 * t < p.group) {
        const float r = la > 0.0f ? 1.0f / la : 0.0f;
        *reinterpret_cast<float2*>(p.out + head * kHeadDim + ch) =
            make_float2(acc.x * r, acc.z * r);
        if (p.lse != nullptr && warp == 0 && g == 0)
          p.lse[head] = (ma - kHeadroom + log2f(la)) * 0.693147180559945309f;
      }
      if (2 * t + 1 < p.group) {
        const float r = lb > 0.0f ? 1.0f / lb : 0.0f;
        *reinterpret_cast<float2*>(p.out + (head + 1) * kHeadDim + ch) =
            make_float2(acc.y * r, acc.w * r);
        if (p.lse != nullptr && warp == 0 && g == 0)
          p.lse[head + 1] = (mb - kHeadroom + log2f(lb)) * 0.693147180559945309f;
      }
    }
    __syncthreads();  // the meeting place is free for the next row
    x = stop;
  }
}

size_t smem_bytes(int batch) { return 1024 + sizeof(Smem) + 8 * (size_t)(batch + 1) + 4 * (size_t)batch; }

}  // namespace

int kv8_attend_ctas(int num_sms) { return std::min(2 * num_sms, kKv8MaxCtas); }

cudaError_t launch_kv8_attend(const Shape& s, bool kept, const Kv8& c, const CUtensorMap& k_map,
                              const CUtensorMap& v_map, const void* q, const int32_t* page_table,
                              const int32_t* seq_lens, const int32_t* block_idx,
                              const int32_t* n_blocks, float* out, float* lse, int* counters,
                              float* part_ml, float* part_o, int* err, int num_sms,
                              cudaStream_t st) {
  const bool per_head = kept && s.per_head;
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.block_idx = block_idx;
  p.n_blocks = n_blocks;
  p.out = out;
  p.lse = lse;
  p.part_ml = part_ml;
  p.part_o = part_o;
  p.counters = counters;
  p.err = err;
  p.batch = s.batch;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.rows = per_head ? s.hq : s.hkv;
  p.group = per_head ? 1 : s.group;
  p.kv_div = per_head ? s.group : 1;
  p.max_pages = s.max_pages;
  p.num_pages = s.num_pages;
  p.sink = s.sink;
  p.window = s.window;
  p.k2 = s.k2;
  p.scale_log2 = s.sm_scale * 1.44269504088896341f;
  // no more CTAs than the longest possible line has smallest slices
  const long long most_row =
      kept ? std::min<long long>((s.sink + kPage - 1) / kPage, s.max_pages) +
                 std::min<long long>(s.window / kPage + 2, s.max_pages) + s.k2
           : s.max_pages;
  const long long most = (most_row * p.rows * s.batch + kMinUnits - 1) / kMinUnits;
  const int grid = (int)std::max(1LL, std::min<long long>(kv8_attend_ctas(num_sms), most));
  auto kernel = c.format == kE4m3
                    ? (kept ? kv8_attend_kernel<kE4m3, true> : kv8_attend_kernel<kE4m3, false>)
                    : (kept ? kv8_attend_kernel<kInt8, true> : kv8_attend_kernel<kInt8, false>);
  const size_t smem = smem_bytes(s.batch);
  const cudaError_t e = set_kernel_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, st, false, k_map, v_map, p);
}

}  // namespace hsa
