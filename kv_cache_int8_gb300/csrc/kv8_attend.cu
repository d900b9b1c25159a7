// kv8_attend.cu -- decode attention over the 8-bit K/V cache: one query token a sequence over
// every token (dense) or over the sink, the window and a list of kept blocks.
//
// Source: "KV Cache 与长上下文推理", section "KV Cache 回顾" (decode attention equation), section
// "KV Cache 量化"; the attended set is hsa_attend's.
//
// Mathematics. A block of 16 tokens has codes a_t, c_t (K, V) and scales s_k, s_v:
//   x_tj = (sm_scale log2 e s_k) q_j . a_t     y_tj = x_tj + log2 s_v
//   out_j = sum_t 2^(y_tj - m) c_t / sum_t 2^(x_tj - m)
// Both products run on the matrix pipe with fp16 operands and fp32 sums, and nothing is rounded
// that matters: the codes are exact in fp16; a head's query is multiplied by the power of two
// that puts its largest value in [2^13, 2^14), which makes every bf16 value down to 2^-27 of
// that one exact in fp16; a probability is carried with V's scale as 2^(y - m + 10), where m
// follows the maximum of y and may lag it by up to 4, so at most 2^14, and is split into fp16
// hi + lo, 22 bits together. The sum of the weights takes them times 1 / s_v, a factor a block,
// as long as every s_v is within 2^-40 .. 2^40: below 2^54 a token then, and a token that matters
// is no smaller than 2^-70. From a row's first block on whose s_v is not (a block of zeros has
// none), a second form of the loop sums 2^x under a maximum of its own: right for any mixture of
// scales, at the price of more exponentials. log2 s_v takes log2f, not the fast instruction, as its
// error enters the result whole: one token under scales of 2^-10 to 2^-5 is 1.8e-7 off (7.7e-7),
// of 2^-40 1.8e-7 (2.8e-6), for 0.05 us a call. The relative error against 64 bits is 3 to 7e-7
// (2-norm).
//
// Layout. K's block is the left operand [16 tokens][128 channels], the group's heads (up to 8)
// the 8 columns of m16n8k16; V's block enters transposed, 8 tiles of 16 channels. So a group of
// 8 heads wastes no product, and scores, probabilities and outputs keep one layout: a lane has
// heads 2t, 2t + 1. Which channel a product's k index stands for is free as long as both sides
// agree: a lane takes whole 16-byte chunks, and the 128-byte swizzle of the tensor copies makes
// all its reads free of bank conflicts. (tcgen05 would want 128 rows of queries; there are 8.)
//
// Work. Memory bound: a block's 4 KiB cost an SM about 175 cycles at the HBM rate, its
// instructions about 100 of each scheduler's issue slots. Every warp streams its own blocks
// through its own ring of tensor copies, no barriers between warps, two blocks at a time (two
// independent chains of products). One CTA of 16 warps an SM: two of 8 had the same loop but
// twice the parts to join (128K tokens 59 us). All blocks of all rows (sequence, kv head) form
// one line that is cut into equal slices, one a CTA, so ragged batches balance without the host
// knowing any length; where a slice ends inside a row, the row's parts meet in the workspace
// and the last CTA to arrive joins them in slice order (the result does not depend on which one
// that is).
//
// Measured (GB300, copy 6.8 TB/s; 8 kv heads): 8 x 32-128K tokens, groups of 8, int8: 226 us,
// 6.2 TB/s; one sequence of 128K tokens, groups of 4: 53.5 us, 5.0 TB/s (a further byte costs
// 1 / 7.0 TB/s; about 7 us pass before the first blocks are there everywhere and 5 us in
// joining); 8K tokens of one kv head: 13 us; 128 kept blocks, sink and window of 128K: 12.2 us.
#include "kv8.cuh"

#include <climits>
#include <cmath>
#include <type_traits>

namespace hsa {
namespace {

using namespace kv8_detail;

constexpr int kWarps = 16;  // one CTA an SM
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;                     // a warp's ring: blocks in flight or in use
constexpr int kMeta = 32, kBatch = 16;         // a warp's visits known ahead, fetched 16 at once
constexpr int kUnitBytes = 2 * kBlockBytesI8;  // K block, then V block
constexpr int kMinUnits = kWarps;              // smallest slice: one block a warp
constexpr int kTile = 8 * kHeadDim;            // output values of a row (8 heads)
constexpr int kAhead = 24;                     // parts of a row joined at a time
constexpr float kHeadroom = 10.0f;             // p is 2^(x - m + kHeadroom)
constexpr float kLag = 4.0f;                   // m follows a maximum that is this much larger
constexpr float kPlainScale = 40.0f;           // largest |log2 s_v| of the loop's plain form
constexpr float kLow = -1e30f;                 // below any m

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
  int* counters;   // [CTAs]: of the row that begins in a CTA and goes on behind it
  int* err;
  int batch, hq, hkv, rows, group, kv_div, max_pages, num_pages, sink, window, k2;
  float scale_log2;  // sm_scale log2 e
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d = a b
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1,
                                              uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// c += a b
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// o += d. The products' own accumulation rounds towards zero: over the thousands of blocks that
// a warp adds up, that alone put results 3e-6 off.
__device__ __forceinline__ void add4(float (&o)[4], const float (&d)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2)
    asm("{.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;}"
        : "+f"(o[i]), "+f"(o[i + 1])
        : "f"(d[i]), "f"(d[i + 1]));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t word(const uint4& u, int w) {
  return w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w;
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float max32(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
// over the lanes of one pair of heads
__device__ __forceinline__ float max_tokens(float x) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
__device__ __forceinline__ float sum32(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// Waits with a limit, the warp's lanes alike: a wait that runs out does so for all of them, as
// what follows (shuffles, products) takes them all.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
    if (__any_sync(0xffffffffu, clock64() - t0 > kWaitLimitCycles)) return false;
  return true;
}

__device__ __noinline__ void wait_for_all(uint64_t* full, int slot, uint32_t ph, int n) {
  for (; n > 0; n--) {
    warp_wait(full + slot, ph);
    ph ^= slot == kStages - 1;
    slot = slot == kStages - 1 ? 0 : slot + 1;
  }
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
constexpr int kFar = INT_MIN;  // of a span: the loop's plain form does not take s_v
struct alignas(16) Unit {
  int y;
  int span;       // lo | hi << 8, negative with kFar; 0: nothing to do
  float sk, sv;  // the scales; sv as it is used: log2 s_v (-inf for a block of zeros)
};

// Places of a row on the line: with per > 0 a whole number of slices of `per`.
__device__ __forceinline__ unsigned row_places(unsigned units, unsigned per) {
  return per > 0 ? (units + per - 1) / per * per : units;
}

template <bool kKept>
__device__ __forceinline__ Unit locate(const Params& p, const long long* pre, const int* lens,
                                       unsigned per, long long x) {
  int lo_b = 0, hi_b = p.batch;  // the sequence with pre[b] <= x < pre[b + 1]
  while (hi_b - lo_b > 1) {
    const int mid = (lo_b + hi_b) >> 1;
    if (pre[mid] <= x) lo_b = mid;
    else hi_b = mid;
  }
  const int b = lo_b, n = lens[b];
  const int units = row_units<kKept>(p, n);
  const unsigned u = row_places(units, per);
  const unsigned at = (unsigned)(x - pre[b]);
  const int row = at / u, i = at % u;
  Unit t = {0, 0, 0.0f, 0.0f};
  if (i >= units) return t;
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
  const float sv = p.v_scale[block];
  t.sv = log2f(sv);
  if (!(fabsf(t.sv) <= kPlainScale)) t.span |= kFar;
  return t;
}

struct Smem {
  // a warp's blocks; where the warps' parts of a row meet, the slot it has just read holds its
  // outputs (float4 [channel tile][lane], 4 KiB as well)
  alignas(1024) unsigned char ring[kWarps][kStages][kUnitBytes];
  Unit meta[kWarps][kMeta];
  float2 ml[8][kWarps];      // a head's (m, l) of each warp
  float weight[kAhead][8];   // of the warps, then of the parts: 2^(m - the largest m)
  float2 total[4][8];        // a row's (m, l), of each team
  int slot[kWarps];   // the ring slot of each warp's outputs
  alignas(8) uint64_t full[kWarps][kStages];
  int last;
  long long per;
  unsigned align;
  int team;
};
// behind it: pre (long long [batch + 1]), lens (int [batch])

// kTeams: more rows than CTAs, which a team of 16, 4 or 1 warps may then take whole. (Without it
// the code is a fifth shorter, which a call of a few rows feels: 12.6 against 13.7 us.)
template <int F, bool kKept, bool kTeams>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_attend_kernel(const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const Params p) {
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  long long* pre = reinterpret_cast<long long*>(&sm + 1);
  int* lens = reinterpret_cast<int*>(pre + p.batch + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  if (tid == 0) {
    tma_prefetch_descriptor(&k_map);
    tma_prefetch_descriptor(&v_map);
  }
  grid_dep_wait();
  grid_dep_launch();

  // ---- the line of all units and this CTA's slice of it
  if (lane < kStages) mbar_init(&sm.full[warp][lane], 1);
  fence_barrier_init();
  if (warp == 0) {
    auto lay = [&](unsigned per) {  // pre from lens; the line's length
      long long sum = 0;
      for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        const unsigned units = b < p.batch ? row_units<kKept>(p, lens[b]) : 0;
        long long incl = (long long)row_places(units, per) * p.rows;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        if (b < p.batch) pre[b + 1] = sum + incl;
        sum += __shfl_sync(0xffffffffu, incl, 31);
      }
      return sum;
    };
    for (int b = lane; b < p.batch; b += 32) {
      int n = p.seq_lens[b];
      if (n < 0 || n > p.max_pages * kPage) {
        set_error(p.err, kDevErrCheck);
        n = 0;
      }
      lens[b] = n;
    }
    __syncwarp();
    const long long sum = lay(0);
    // How the line is cut, and how many warps share a row (rows: sequences x kv heads):
    //  - up to a row a CTA: 16 warps, slices of the smallest of 32 sizes from the even cut on
    //    under which every row begins with a slice of its own (a CTA that ends one row and
    //    begins the next joins parts twice, 5 us at 128K tokens, the time of 54 units);
    //  - else by what the three team sizes would take, in us, from fits to the cases below: the
    //    stream's 0.09 a unit and SM, or the rows that a team takes one after the other, and a
    //    last row that no other team helps with. Teams of 4 and of 1 take whole rows; teams of
    //    16 (a CTA) even slices, whatever rows they cut. Measured, teams of 16 alone and this
    //    rule: 8192 rows of 80 tokens 304 and 67 us, of 450 tokens 419 and 207; 2048 rows of 650
    //    147 and 89; 512 rows of 650 51 and 37, of 2500 (where it takes 16) 88 and 94; 240 rows
    //    of 28 33 and 9.3; 160 rows of 620 22.6 and 17.8.
    const long long rows = (long long)p.batch * p.rows;
    long long per = max((sum + gridDim.x - 1) / gridDim.x, (long long)kMinUnits);
    unsigned align = 0;
    int team = kWarps;
    if (!kTeams && rows <= gridDim.x) {
      const unsigned mine = (unsigned)per + lane;
      long long slices = 0;
      for (int b = 0; b < p.batch; b++)
        slices += (long long)((row_units<kKept>(p, lens[b]) + mine - 1) / mine) * p.rows;
      const unsigned fits = __ballot_sync(0xffffffffu, slices <= gridDim.x);
      if (fits != 0) {
        per = align = (unsigned)per + __ffs(fits) - 1;
        lay(align);
      }
    }
    if (kTeams) {
      int longest = 0;
      for (int b = lane; b < p.batch; b += 32) longest = max(longest, row_units<kKept>(p, lens[b]));
      longest = (int)max32((float)longest);
      const float stream = 0.09f * sum / gridDim.x, each = (float)rows / gridDim.x;
      const float mean = (float)sum / rows;
      const float t16 = stream + 5.0f * each + 15.0f;
      const float t4 = fmaxf(stream, each / 4 * (5.0f + 0.42f * mean)) + 0.3f * longest;
      const float t1 = fmaxf(stream, each / 16 * (8.0f + 1.45f * mean)) + 0.7f * longest;
      team = t1 <= fminf(t4, t16) ? 1 : t4 <= t16 ? 4 : kWarps;
      const long long teams = (long long)gridDim.x * (kWarps / team);
      if (team < kWarps) per = max((sum + teams - 1) / teams, 1LL);
    }
    if (lane == 0) {
      pre[0] = 0;
      sm.per = per;
      sm.align = align;
      sm.team = team;
    }
  }
  __syncthreads();
  const long long per = sm.per;
  const unsigned align = sm.align;
  const int team = kTeams ? sm.team : kWarps;  // warps that share a row: 16, 4 or 1
  const int first_warp = warp & ~(team - 1);
  const long long all = pre[p.batch];
  auto sequence_at = [&](long long x) {  // the b with pre[b] <= x < pre[b + 1]
    int lo_b = 0, hi_b = p.batch;
    while (hi_b - lo_b > 1) {
      const int mid = (lo_b + hi_b) >> 1;
      if (pre[mid] <= x) lo_b = mid;
      else hi_b = mid;
    }
    return lo_b;
  };
  auto row_from = [&](long long x) {  // where the first row from place x on begins
    if (x >= all) return all;
    const int b = sequence_at(x);
    const unsigned u = row_places(row_units<kKept>(p, lens[b]), align);
    return pre[b] + (long long)((unsigned)(x - pre[b] + u - 1) / u) * u;
  };
  const int slice = (blockIdx.x * kWarps + first_warp) / team;
  long long begin = min(slice * per, all), end = min(begin + per, all);
  if (kTeams && team < kWarps) {  // whole rows
    begin = row_from(begin);
    end = row_from(end);
  }
  auto team_sync = [&]() {
    asm volatile("bar.sync %0, %1;" ::"r"(team == kWarps ? 0 : 1 + first_warp / 4), "r"(team * 32)
                 : "memory");
  };

  // rows of no units at all
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (pre[b + 1] != pre[b]) continue;
    for (int i = tid; i < p.hq * kHeadDim; i += kThreads)
      p.out[(size_t)b * p.hq * kHeadDim + i] = 0.0f;
    if (p.lse != nullptr)
      for (int i = tid; i < p.hq; i += kThreads) p.lse[(size_t)b * p.hq + i] = -INFINITY;
  }
  if (begin >= end) return;

  // ---- this warp's visits: places x0 + stride i, located kBatch at a time
  const long long x0 = begin + (warp - first_warp);
  const int stride = team;
  const int mine = x0 < end ? (int)((end - x0 + stride - 1) / stride) : 0;
  auto fetch = [&](int i0) {
    const long long x = x0 + (long long)stride * (i0 + lane);
    Unit u = {0, 0, 0.0f, 0.0f};
    if (lane < kBatch && x < end) u = locate<kKept>(p, pre, lens, align, x);
    return u;
  };
  Unit* meta = sm.meta[warp];
  auto store = [&](int i0, const Unit& u) {
    __syncwarp();
    if (lane < kBatch) meta[(i0 + lane) % kMeta] = u;
    __syncwarp();
  };
  store(0, fetch(0));
  int filled = kBatch;
  bool pending = false;
  Unit ahead = {0, 0, 0.0f, 0.0f};
  const uint64_t policy = l2_evict_first_policy();
  int asked = 0;             // visits whose copies were begun (those that have any)
  int flying = 0;            // copies begun and not yet waited for
  int in = 0, out = 0;       // ring slots of the next copy to begin and to wait for
  uint32_t phase = 0;        // of the barriers that `out` comes to
  unsigned char* const ring = sm.ring[warp][0];
  uint64_t* const full = sm.full[warp];
  bool dead = false;  // a copy did not come: no further ones, no further work
  // Begins the copies of the visits before `upto`. Those of later rows (from visit `stop` on)
  // leave one slot of the ring free: the row's outputs will lie there.
  auto issue_to = [&](int upto, int stop) {
    for (upto = min(upto, mine); asked < upto; asked++) {
      const Unit& u = meta[asked % kMeta];
      if (u.span == 0 || dead) continue;
      if (flying >= kStages - (asked < stop ? 0 : 1)) break;
      if (lane == 0) {
        unsigned char* dst = ring + in * kUnitBytes;
        mbar_arrive_expect_tx(full + in, kUnitBytes);
        tma_load_2d_hint(dst, &k_map, 0, u.y, full + in, policy);
        tma_load_2d_hint(dst + kBlockBytesI8, &v_map, 0, u.y, full + in, policy);
      }
      in = in == kStages - 1 ? 0 : in + 1;
      flying++;
    }
  };

  int i = 0;
  for (long long x = begin; x < end;) {
    // ---- the row at x, and how far this slice goes in it
    const int b = sequence_at(x);
    const unsigned units = row_places(row_units<kKept>(p, lens[b]), align);
    const int row = (int)((unsigned)(x - pre[b]) / units);
    const long long row_begin = pre[b] + (long long)row * units, row_end = row_begin + units;
    const long long stop = min(row_end, end);
    const int i_stop = (int)((stop - x0 + stride - 1) / stride);  // this warp's visits before it
    issue_to(i + kStages, i_stop);

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
      const float f = p.scale_log2 * down;
      f0 = __shfl_sync(0xffffffffu, f, (2 * t) * 4);
      f1 = __shfl_sync(0xffffffffu, f, (2 * t + 1) * 4);
    }

    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    float o[8][4];
#pragma unroll
    for (int k = 0; k < 8; k++)
#pragma unroll
      for (int c = 0; c < 4; c++) o[k][c] = 0.0f;

    // Two visits at a time: two independent chains of products, one reduction of the maximum.
    // kApart: one, and l0 and l1 are the lanes' sums of 2^(x - top), not of 2^(y - m + kHeadroom)
    // / s_v.
    bool apart = false;
    float top0, top1;
    auto visit = [&](auto form) {
      constexpr bool kApart = decltype(form)::value;
      constexpr int kPair = kApart ? 1 : 2;  // visits
      const int two = !kApart && i + 1 < i_stop;
      if (!pending && filled < mine && filled - i <= kBatch) {
        ahead = fetch(filled);
        pending = true;
      } else if (pending && filled - i <= kBatch / 2) {
        store(filled, ahead);
        filled += kBatch;
        pending = false;
      }
      const Unit ua = meta[i % kMeta];
      Unit ub = meta[(i + 1) % kMeta];
      if (!two) ub.span = 0;
      const int spans = ua.span | ub.span;
      if (kApart ? spans != 0 && !dead : spans > 0 && !dead) {
        uint32_t kb[2];
        const int mask = kApart ? ~kFar : -1;
        const int span[2] = {ua.span & mask, ub.span & mask};
#pragma unroll
        for (int h = 0; h < kPair; h++) {
          kb[h] = smem_addr(ring) + out * kUnitBytes;
          if (span[h] == 0) continue;
          if (!warp_wait(full + out, phase)) {
            set_error(p.err, kDevErrTimeout);
            dead = true;
            // copies under way write this CTA's shared memory: one more wait for each
            wait_for_all(full, out, phase, flying);
          }
          flying--;
          out++;
          if (out == kStages) {
            out = 0;
            phase ^= 1;
          }
        }
        // scores of tokens g (x[h][0], x[h][1]) and g + 8 (x[h][2], x[h][3])
        float x[2][4];
#pragma unroll
        for (int c = 0; c < 2; c++) {
          uint4 ka[2], kc[2];
#pragma unroll
          for (int h = 0; h < kPair; h++) {
            const uint32_t at = kb[h] + g * kHeadDim + (((2 * t + c) ^ g) << 4);
            ka[h] = lds128(at);
            kc[h] = lds128(at + 8 * kHeadDim);
          }
#pragma unroll
          for (int w = 0; w < 4; w++)
#pragma unroll
            for (int h = 0; h < kPair; h++) {
              const uint32_t a = Codes<F>::prepare(word(ka[h], w));
              const uint32_t d = Codes<F>::prepare(word(kc[h], w));
              const uint32_t a0 = Codes<F>::template pair<0>(a), a1 = Codes<F>::template pair<0>(d);
              const uint32_t a2 = Codes<F>::template pair<1>(a), a3 = Codes<F>::template pair<1>(d);
              if (c == 0 && w == 0)
                mma16816_zero(x[h], a0, a1, a2, a3, qf[0], qf[1]);
              else
                mma16816(x[h], a0, a1, a2, a3, qf[c * 8 + w * 2], qf[c * 8 + w * 2 + 1]);
            }
        }
        const float cv[2] = {ua.sv, ub.sv};
        if (kApart) {
          float z[4];
          const int lo = span[0] & 255, hi = span[0] >> 8;
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const int tok = g + 4 * (c & 2);
            z[c] = tok >= lo && tok < hi ? x[0][c] * ((c & 1 ? f1 : f0) * ua.sk) : -INFINITY;
          }
          float z0 = fmaxf(top0, fmaxf(z[0], z[2])), z1 = fmaxf(top1, fmaxf(z[1], z[3]));
          z0 = max_tokens(z0);  // finite, as one token at least is seen
          z1 = max_tokens(z1);
          l0 = l0 * ex2(top0 - z0) + (ex2(z[0] - z0) + ex2(z[2] - z0));
          l1 = l1 * ex2(top1 - z1) + (ex2(z[1] - z1) + ex2(z[3] - z1));
          top0 = z0;
          top1 = z1;
        }
        float n0 = -INFINITY, n1 = -INFINITY;
#pragma unroll
        for (int h = 0; h < kPair; h++) {  // y = x + log2 s_v
          const float sk = h ? ub.sk : ua.sk;
          x[h][0] = fmaf(x[h][0], f0 * sk, cv[h]);
          x[h][1] = fmaf(x[h][1], f1 * sk, cv[h]);
          x[h][2] = fmaf(x[h][2], f0 * sk, cv[h]);
          x[h][3] = fmaf(x[h][3], f1 * sk, cv[h]);
          if (span[h] != (kPage << 8)) {
            const int lo = span[h] & 255, hi = span[h] >> 8;
            if (g < lo || g >= hi) x[h][0] = x[h][1] = -INFINITY;
            if (g + 8 < lo || g + 8 >= hi) x[h][2] = x[h][3] = -INFINITY;
          }
          n0 = fmaxf(n0, fmaxf(x[h][0], x[h][2]));
          n1 = fmaxf(n1, fmaxf(x[h][1], x[h][3]));
        }
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
          if (!kApart) {
            l0 *= a0;
            l1 *= a1;
          }
#pragma unroll
          for (int k = 0; k < 8; k++) {
            o[k][0] *= a0;
            o[k][1] *= a1;
            o[k][2] *= a0;
            o[k][3] *= a1;
          }
        }
        const float ref0 = m0 - kHeadroom, ref1 = m1 - kHeadroom;
#pragma unroll
        for (int h = 0; h < kPair; h++) {
          if (span[h] == 0) continue;
          const float p00 = ex2(x[h][0] - ref0), p01 = ex2(x[h][1] - ref1);
          const float p10 = ex2(x[h][2] - ref0), p11 = ex2(x[h][3] - ref1);
          if (!kApart) {
            const float per_s = ex2(-cv[h]);  // 1 / s_v
            l0 = fmaf(p00 + p10, per_s, l0);
            l1 = fmaf(p01 + p11, per_s, l1);
          }
          const uint32_t ha = half_pair(p00, p01), hb = half_pair(p10, p11);
          const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&ha));
          const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&hb));
          const uint32_t b0 = transpose8x8(ha), b1 = transpose8x8(hb);
          const uint32_t r0 = transpose8x8(half_pair(p00 - fa.x, p01 - fa.y));
          const uint32_t r1 = transpose8x8(half_pair(p10 - fb.x, p11 - fb.y));
          // values: tokens 2t, 2t + 1, 2t + 8, 2t + 9 of channels [16 g, 16 g + 16)
          const uint32_t vb = kb[h] + kBlockBytesI8;
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const int tok = 2 * t + (k & 1) + 8 * (k >> 1);
            v[k] = lds128(vb + tok * kHeadDim + ((g ^ (tok & 7)) << 4));
          }
          if (F == kE4m3 && span[h] != (kPage << 8)) {  // bytes no token wrote may be NaN
            const int lo = span[h] & 255, hi = span[h] >> 8;
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const int tok = 2 * t + (k & 1) + 8 * (k >> 1);
              if (tok < lo || tok >= hi) v[k] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
#pragma unroll
          for (int w = 0; w < 4; w++) {
#pragma unroll
            for (int c = 0; c < 2; c++) {  // channels 4 w + 2 c + {0, 1}
              const uint32_t sel = c ? 0x7362u : 0x5140u;
              const uint32_t ab = Codes<F>::prepare(prmt(word(v[0], w), word(v[1], w), sel));
              const uint32_t cd = Codes<F>::prepare(prmt(word(v[2], w), word(v[3], w), sel));
              const uint32_t a0 = Codes<F>::template pair<0>(ab);
              const uint32_t a1 = Codes<F>::template pair<1>(ab);
              const uint32_t a2 = Codes<F>::template pair<0>(cd);
              const uint32_t a3 = Codes<F>::template pair<1>(cd);
              float d[4];
              mma16816_zero(d, a0, a1, a2, a3, b0, b1);
              mma16816(d, a0, a1, a2, a3, r0, r1);
              add4(o[2 * w + c], d);
            }
          }
        }
      } else if (!kApart && __builtin_expect(spans < 0, 0)) {
        apart = true;
        return;
      }
      i += 1 + two;
      __syncwarp();  // the slots are read before they are filled again
      issue_to(i + kStages, i_stop);
    };
    while (i < i_stop && !apart) visit(std::false_type{});
    if (__builtin_expect(apart, 0)) {
      top0 = m0 - kHeadroom;
      top1 = m1 - kHeadroom;
      m0 = fmaxf(m0, kLow);  // before any block but those of zeros: y is -inf, m must not be
      m1 = fmaxf(m1, kLow);
      while (i < i_stop) visit(std::true_type{});
      // Back into one frame, within 2^50 of the sums' own: o (the result times the sum, in that
      // frame) and l stay in fp32's range, and of two parts that are joined the frames differ by
      // 2^100 at most beside their sums: a factor that fp32 flushes to 0, below 2^-126, belongs
      // to a part that counts for less than 2^-26.
      const float was0 = m0 - kHeadroom, was1 = m1 - kHeadroom;
      m0 = fminf(fmaxf(was0, top0 - 50.0f), top0 + 50.0f) + kHeadroom;
      m1 = fminf(fmaxf(was1, top1 - 50.0f), top1 + 50.0f) + kHeadroom;
      const float to0 = m0 - kHeadroom, to1 = m1 - kHeadroom;  // as they are read again
      // in two factors, as one alone may leave the range
      const float a0 = ex2(0.5f * (was0 - to0)), a1 = ex2(0.5f * (was1 - to1));
#pragma unroll
      for (int k = 0; k < 8; k++) {
        o[k][0] = o[k][0] * a0 * a0;
        o[k][1] = o[k][1] * a1 * a1;
        o[k][2] = o[k][2] * a0 * a0;
        o[k][3] = o[k][3] * a1 * a1;
      }
      l0 *= ex2(top0 - to0);
      l1 *= ex2(top1 - to1);
    }

    // ---- the warps' parts of the row meet
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (kTeams && team == 1) {  // the row is this warp's
      const size_t head = (size_t)b * p.hq + (size_t)row * p.group + 2 * t;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if (2 * t + h >= p.group) continue;
        const float l = h ? l1 : l0;
        const float r = l != 0.0f ? 1.0f / l : 0.0f;
        float4* dst = reinterpret_cast<float4*>(p.out + (head + h) * kHeadDim + 16 * g);
#pragma unroll
        for (int k = 0; k < 8; k += 2)
          dst[k / 2] = make_float4(o[k][h] * r, o[k][2 + h] * r, o[k + 1][h] * r, o[k + 1][2 + h] * r);
        if (p.lse != nullptr && g == 0)
          p.lse[head + h] = ((h ? m1 : m0) - kHeadroom + log2f(l)) * 0.693147180559945309f;
      }
      x = stop;
      continue;
    }
    if (g == 0) {
      sm.ml[2 * t][warp] = make_float2(m0, l0);
      sm.ml[2 * t + 1][warp] = make_float2(m1, l1);
    }
    {
      const int slot = out == 0 ? kStages - 1 : out - 1;  // free: see issue_to
      float4* dst = reinterpret_cast<float4*>(sm.ring[warp][slot]);
#pragma unroll
      for (int k = 0; k < 8; k++)
        dst[k * 32 + lane] = make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
      if (lane == 0) sm.slot[warp] = slot;
    }
    team_sync();
    // joins (m, l) pairs of a head, one a lane (n of them), into `sum`, and leaves their weights
    // from place `at` on
    auto weigh = [&](float2 v, float2 sum, int head, int at, int n) {
      const float top = fmaxf(max32(v.x), sum.x);
      const float ref = top == -INFINITY ? 0.0f : top;
      const float f = ex2(v.x - ref);  // 0 from -inf
      if (lane < n) sm.weight[at + lane][head] = f;
      return make_float2(top, sum32(f * v.y) + ex2(sum.x - ref) * sum.y);
    };
    const float2 nothing = make_float2(-INFINITY, 0.0f);
    float2* const total = sm.total[first_warp / 4];
    for (int h = warp - first_warp; h < 8; h += team) {
      const float2 v =
          weigh(lane < team ? sm.ml[h][first_warp + lane] : nothing, nothing, h, first_warp, team);
      if (lane == 0) total[h] = v;
    }
    team_sync();
    if (kTeams && team < kWarps) {  // the row is complete: value pairs i of the tile (see below)
      for (int i = tid - first_warp * 32; i < kTile / 2; i += team * 32) {
        const int hl = (i >> 1) & 31, ht = hl & 3;
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const int w = first_warp + k;
          const float2 f = *reinterpret_cast<const float2*>(&sm.weight[w][2 * ht]);
          const float2 v = reinterpret_cast<const float2*>(sm.ring[w][sm.slot[w]])[i];
          acc.x += f.x * v.x;
          acc.y += f.y * v.y;
        }
        const float2 ta = total[2 * ht], tb = total[2 * ht + 1];
        const size_t head = (size_t)b * p.hq + (size_t)row * p.group + 2 * ht;
        const int ch = 16 * (hl >> 2) + 2 * (i >> 6) + (i & 1);
        const bool sums = p.lse != nullptr && i < 8 && (i & 1) == 0;
        if (2 * ht < p.group) {
          p.out[head * kHeadDim + ch] = ta.y != 0.0f ? acc.x / ta.y : 0.0f;
          if (sums) p.lse[head] = (ta.x - kHeadroom + log2f(ta.y)) * 0.693147180559945309f;
        }
        if (2 * ht + 1 < p.group) {
          p.out[(head + 1) * kHeadDim + ch] = tb.y != 0.0f ? acc.y / tb.y : 0.0f;
          if (sums) p.lse[head + 1] = (tb.x - kHeadroom + log2f(tb.y)) * 0.693147180559945309f;
        }
      }
      fence_proxy_async();
      team_sync();  // the slots are free for the next row's blocks
      x = stop;
      continue;
    }
    // values 2 tid, 2 tid + 1 of the tile: channel 16 g' + tid / 64 * 2 + (tid & 1) of heads
    // 2t', 2t' + 1, where lane 4 g' + t' = (tid / 2) % 32 held them
    const int hl = (tid >> 1) & 31, ht = hl & 3;
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int w = 0; w < kWarps; w++) {
      const float2 f = *reinterpret_cast<const float2*>(&sm.weight[w][2 * ht]);
      const float2 v = reinterpret_cast<const float2*>(sm.ring[w][sm.slot[w]])[tid];
      acc.x += f.x * v.x;
      acc.y += f.y * v.y;
    }
    bool write = true;
    if (row_begin < begin || row_end > end) {  // a part of the row: to the workspace
      const int c0 = (int)(row_begin / per), parts = (int)((row_end - 1) / per) - c0 + 1;
      const size_t slot = 2 * (size_t)blockIdx.x + (begin < row_begin ? 1 : 0);
      reinterpret_cast<float2*>(p.part_o + slot * kTile)[tid] = acc;
      if (tid < 8) reinterpret_cast<float2*>(p.part_ml + slot * 16)[tid] = total[tid];
      __syncthreads();
      if (tid == 0) {  // releases what the barrier has ordered before it
        int* counter = p.counters + c0;
        const int last = atomic_add_acq_rel_gpu(counter, 1) == parts - 1;
        if (last) *counter = 0;
        sm.last = last;
      }
      __syncthreads();
      write = sm.last != 0;
      if (write) {
        // What is left of the call's time is the latency of these loads: kAhead parts' values
        // and their (m, l) are under way at once. Part c is the first one of CTA c0 + c, but
        // for c = 0 where that CTA has an earlier row.
        const size_t first = 2 * (size_t)c0 + (c0 * per < row_begin ? 1 : 0);
        const float2* values = reinterpret_cast<const float2*>(p.part_o) + tid;
        auto slot_of = [&](int c) { return c == 0 ? first : 2 * (size_t)(c0 + c); };
        acc = make_float2(0.0f, 0.0f);
        float2 sum = nothing;  // head `warp`
        float2 was = make_float2(-INFINITY, -INFINITY);  // the maxima under which acc is kept
        for (int c = 0; c < parts; c += kAhead) {
          float2 ml = nothing, v[kAhead];
          if (warp < 8 && lane < kAhead && c + lane < parts)
            ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + slot_of(c + lane) * 16) +
                        warp);
          v[0] = __ldcg(values + slot_of(c) * (kTile / 2));
          const float2* more = values + (size_t)(c0 + c) * kTile;
#pragma unroll
          for (int k = 1; k < kAhead; k++) {
            v[k] = make_float2(0.0f, 0.0f);
            if (c + k < parts) v[k] = __ldcg(more + k * kTile);
          }
          if (warp < 8) {
            sum = weigh(ml, sum, warp, 0, kAhead);
            if (lane == 0) total[warp] = sum;
          }
          __syncthreads();
          const float2 now = make_float2(fmaxf(total[2 * ht].x, -1e30f),
                                         fmaxf(total[2 * ht + 1].x, -1e30f));
          acc.x *= ex2(was.x - now.x);  // by 0 the first time
          acc.y *= ex2(was.y - now.y);
          was = now;
#pragma unroll
          for (int k = 0; k < kAhead; k++) {
            const float2 f = *reinterpret_cast<const float2*>(&sm.weight[k][2 * ht]);
            acc.x += f.x * v[k].x;
            acc.y += f.y * v[k].y;
          }
          if (c + kAhead < parts) __syncthreads();  // the weights are read
        }
      }
    }
    if (write) {
      const float2 ta = total[2 * ht], tb = total[2 * ht + 1];
      const size_t head = (size_t)b * p.hq + (size_t)row * p.group + 2 * ht;
      const int ch = 16 * (hl >> 2) + 2 * (tid >> 6) + (tid & 1);
      const bool sums = p.lse != nullptr && tid < 8 && (tid & 1) == 0;
      if (2 * ht < p.group) {
        p.out[head * kHeadDim + ch] = ta.y != 0.0f ? acc.x / ta.y : 0.0f;
        if (sums) p.lse[head] = (ta.x - kHeadroom + log2f(ta.y)) * 0.693147180559945309f;
      }
      if (2 * ht + 1 < p.group) {
        p.out[(head + 1) * kHeadDim + ch] = tb.y != 0.0f ? acc.y / tb.y : 0.0f;
        if (sums) p.lse[head + 1] = (tb.x - kHeadroom + log2f(tb.y)) * 0.693147180559945309f;
      }
    }
    fence_proxy_async();  // the slots were written here and are free for copies again
    __syncthreads();
    x = stop;
  }
}

size_t smem_bytes(int batch) { return 1024 + sizeof(Smem) + 8 * (size_t)(batch + 1) + 4 * (size_t)batch; }

}  // namespace

int kv8_attend_ctas(int num_sms) { return std::min(num_sms, kKv8MaxCtas); }

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
      kept ? std::min<long long>(s.sink / kPage + 1, s.max_pages) +
                 std::min<long long>(s.window / kPage + 2, s.max_pages) + s.k2
           : s.max_pages;
  const long long most = (most_row * p.rows * s.batch + kMinUnits - 1) / kMinUnits;
  const int grid = (int)std::max(
      1LL, std::min<long long>(kv8_attend_ctas(num_sms),
                               std::max(most, (long long)s.batch * p.rows)));
  const bool teams = (long long)s.batch * p.rows > grid;
  auto kernel = kv8_attend_kernel<kInt8, false, false>;
  if (c.format == kE4m3) {
    if (kept) kernel = teams ? kv8_attend_kernel<kE4m3, true, true> : kv8_attend_kernel<kE4m3, true, false>;
    else kernel = teams ? kv8_attend_kernel<kE4m3, false, true> : kv8_attend_kernel<kE4m3, false, false>;
  } else {
    if (kept) kernel = teams ? kv8_attend_kernel<kInt8, true, true> : kv8_attend_kernel<kInt8, true, false>;
    else kernel = teams ? kv8_attend_kernel<kInt8, false, true> : kv8_attend_kernel<kInt8, false, false>;
  }
  const size_t smem = smem_bytes(s.batch);
  const cudaError_t e = set_kernel_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, st, true, k_map, v_map, p);
}

}  // namespace hsa
