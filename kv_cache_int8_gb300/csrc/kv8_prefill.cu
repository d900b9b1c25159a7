// kv8_prefill.cu -- causal attention of many new tokens over the 8-bit K/V cache, on the
// 5th-generation tensor cores.
//
// Source: "KV Cache 与长上下文推理", sections "KV Cache 回顾" (the prompt's attention fills and
// reads the cache) and "KV Cache 量化".
//
// Mathematics. As in the decode attention, the codes enter the products exactly (fp16) and the
// blocks' scales (16 tokens) are applied in fp32: with row factor f = sm_scale log2 e 2^-shift,
//   y_t = f s_k S_t + log2 s_v,   out = sum_t 2^(y_t - M) c_t / sum_t 2^(y_t - M) / s_v
// so V's scale costs nothing but the offset of an exponent that is computed anyway, and the sum
// takes one multiplication a block, as long as every s_v is within 2^-40 .. 2^40 (P / s_v then
// stays below 2^55, and above 2^-73 where it matters). From the first half tile on that has
// another s_v (or a block of zeros, that has none), the rest of a stretch of tiles sums
// 2^(x - its own maximum) beside P, in a second form of the step: right for any mixture of
// scales. P = 2^(y - M + 7) is rounded to fp16 (11 bits, against 8 of the bf16 result); M lags the
// running maximum by at most 8, so the output accumulator is rarely rescaled (with 10 and 4: 2048
// tokens behind 30K 767 us, not 756; 8K prompt 465, not 443).
//
// Layout. 256 rows (a kv head's group of query heads x 256 / group tokens) as two tiles of 128
// against tiles of 128 tokens. Warps 0-3 and 4-7: one row a thread, softmax of tile 0 and 1;
// warps 8-15 turn the codes into swizzled fp16 tiles (two buffers of K and of V); warp 16 issues
// the products. While one tile's scores are in the softmax, the tensor cores work on the other
// tile. TMEM: S0 S1 O0 O1, 128 columns each; P overwrites its S (a product that reads P is
// issued before the product that overwrites it, and they run in order).
//
// Work. All steps (row block, token tile) of all sequences and heads form one line, cut into
// equal slices, one CTA each, as in the decode attention; parts of a row block meet in the
// workspace.
//
// A row block of one tile (up to 128 rows) takes the buffers of S in turn, so its softmax finds
// the next step's scores ready: a step 1.55 us instead of 1.9 (16 tokens over 128K, 8 heads over
// one: 89 -> 76 us).
//
// Measured (GB300, 1884 TFLOP/s bf16 burst, 1693 sustained; 32 query heads over 8; figures beside
// a choice below are of one box, which differ by 3 %): 2048 tokens behind 30K 770-788 us, 1380
// TFLOP/s; an 8K prompt 450-460 us, 1210 TFLOP/s of what its rows see (a diagonal tile is computed
// whole); 4 x 7-24 tokens behind 6-12K 39.4 us; 2048 behind 126K 3245 us (3195 with the products
// adding up over all 1024 tiles, see kMaxTiles). A step's products take
// 2048 cycles, a step 3600: each tile's way from S over the softmax and P V to its next S is one
// chain, and two tiles overlap it only in part. Instructions: 1880 a step and scheduler, half its
// slots (1/3 of them the conversion). With registers to spare nothing changes (144 / 80 / 32 and
// 136 / 88 / 32 instead of 136 / 80 / 48: 765-775, 466-471, 40 us); queries loaded two rows an
// instruction instead of a row a thread: 767, 468, 40.
#include "kv8.cuh"
#include "tcgen05.cuh"

#include <climits>
#include <cmath>
#include <type_traits>

namespace hsa {
namespace {

using namespace kv8_detail;

constexpr int kRows = 256;         // rows of a block: two tiles
constexpr int kTokens = 128;       // tokens of a step
constexpr int kTilePages = kTokens / kPage;
constexpr int kTileBytes = 128 * kHeadDim * 2;
constexpr int kHalfBytes = kTileBytes / 2;  // 64 channels of 128 rows
constexpr int kSoftmaxWarps = 8, kConvertWarps = 8;  // 0-7, 8-15
constexpr int kMmaWarp = 16;
constexpr int kThreads = 640;  // five warpgroups; the last is warp 16 and three idle ones
// registers a thread of the softmax, conversion and product warpgroups: 96 on average
constexpr int kSoftmaxRegs = 136, kConvertRegs = 80, kMmaRegs = 48;
static_assert(2 * kSoftmaxRegs + 2 * kConvertRegs + kMmaRegs == 5 * 96, "the launch's registers");
static_assert(kConvertWarps == kTilePages, "a warp converts one block of K and of V a step");
constexpr float kPartCost = 1.3f, kStepCost = 1.55f;  // us
constexpr int kPageRing = 4;
constexpr int kBlockCost = 4;  // what a row block costs beside its tiles, in tiles (see Walk)
// P = 2^(y - M + kHeadroom), y - M up to kLag: at most 2^15. A smaller headroom leaves small
// probabilities in fp16's subnormals, 2^-25 off each: 2^20 tokens off the same way and together
// as heavy as the largest make 2^-5 of 2^7, 2^-12 of the result (bf16 rounds it to 2^-9).
constexpr float kHeadroom = 7.0f;
constexpr float kLag = 8.0f;
// The products' own accumulation rounds towards zero: 1M tokens added up in O (65536 products)
// gave results 2.6e-3 (equal scores) to 5e-3 (normal ones) too small, more than bf16's own
// rounding. So O takes at most that many tiles' products, below 2048 x 2^-23 = 2.4e-4, and a
// longer stretch is added up in fp32 outside. (Ending a stretch costs about four steps.)
constexpr int kMaxTiles = 256;
constexpr float kPlainScale = 40.0f;  // largest |log2 s_v| under which the sum is made of P / s_v
constexpr float kTiny = 1e-37f;  // scales of scores are at least that: a masked -inf stays one
// s_full and p_full of the tiles and, where a row block has one tile, of its odd steps
constexpr int kOdd = 2;
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns; tile i at + 128 i

struct Params {
  NewRows rows;
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  __nv_bfloat16* out;
  float* lse;
  float* part_ml;  // [2 CTAs][kRows] (M, l)
  float* part_o;   // [2 CTAs][32][kRows] float4
  int* counters;   // [CTAs][2 tiles]
  int* err;
  int hq, hkv, group, num_pages, block_tokens;  // block_tokens = kRows / group
  float scale_log2;
};

struct Smem {
  alignas(1024) unsigned char q[2][kTileBytes];
  unsigned char k[2][kTileBytes];
  unsigned char v[2][kTileBytes];
  // Of a step's blocks: x = w, but +inf where |w| is above kPlainScale; y = 1 / s_v (any number
  // above 0 for zeros, 0 where there are no tokens); z = s_k; w = log2 s_v (-inf for both). x and
  // y are read alone, as an aligned pair.
  float4 page[kPageRing][kTilePages];
  alignas(8) uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[3],
      p_full[3][2], o_full[2];  // s_full, p_full: kOdd; p_full[..][half of the tokens]
  uint64_t pv_done, h_done[2];  // products with V complete: one tile's step, a first half
  uint64_t all_done;            // all products, after a wait that ran out
  long long per;
  int start_b, start_h, start_q, start_off;
  uint32_t tmem;
  int last[2];
  int dead;
};
// behind it: pre (long long [batch + 1]), then len, n, row0 (int [batch] each)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// a * m + c and a + b on two values at once
__device__ __forceinline__ float2 fma2(float2 a, float2 m, float2 c) {
  float2 y;
  asm("{.reg .b64 a, m, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 m, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 a, a, m, c;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(m.x), "f"(m.y), "f"(c.x), "f"(c.y));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t bf16_max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// 64 bytes of an output row, one thread a row: stores of 32 bytes fill whole sectors.
__device__ __forceinline__ void store_row_part(__nv_bfloat16* dst, const uint32_t (&w)[16]) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
    for (int k = 0; k < 16; k += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 2 * k),
                   "r"(w[k]), "r"(w[k + 1]), "r"(w[k + 2]), "r"(w[k + 3]), "r"(w[k + 4]),
                   "r"(w[k + 5]), "r"(w[k + 6]), "r"(w[k + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      *reinterpret_cast<uint4*>(dst + 2 * k) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
  }
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Waits with a limit, a whole warp alike; once a wait has run out every wait of the CTA gives up.
__device__ __forceinline__ bool wait(Smem& sm, uint64_t* bar, uint32_t parity, int* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = mbar_try_wait(bar, parity))) {
      if (*reinterpret_cast<volatile int*>(&sm.dead)) break;
      if (clock64() - t0 > kWaitLimitCycles) {
        *reinterpret_cast<volatile int*>(&sm.dead) = 1;
        set_error(err, kDevErrTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

struct Seqs {
  const long long* pre;
  const int* len;
  const int* n;
  const int* row0;
};

// Token tiles that row block q of a sequence visits.
__device__ __forceinline__ int block_tiles(int len, int n, int block_tokens, int q) {
  return (len - n + min((q + 1) * block_tokens, n) - 1) / kTokens + 1;
}

// A stretch of one row block's tiles: what a CTA does at a time.
struct Piece {
  int b, h, q;       // sequence, kv head, row block
  int tile, tiles;   // first tile, number of tiles
  int all_tiles;     // of the whole row block
  int rows;          // rows of the block that exist
  long long begin;   // the row block's first place on the line
};

// The pieces of the slice [x, end) of the line, in order. A row block's places are kBlockCost
// for what it costs beside its tiles (queries in, results out), then
// one a tile. Without the first, the CTAs with a head's first, short row blocks would take half
// as long again as the others (8K prompt: 624 us without, 472 with 4 when that was found; now 454
// with 3, 442 with 4, 444 with 5).
struct Walk {
  const Seqs s;
  int batch, hkv, group, block_tokens;
  long long x, end;
  int b, h, q, off;  // off: place in the row block

  __device__ __forceinline__ bool next(Piece& p) {
    for (;;) {
      if (x >= end) return false;
      p.b = b;
      p.h = h;
      p.q = q;
      p.begin = x - off;
      p.all_tiles = block_tiles(s.len[b], s.n[b], block_tokens, q);
      p.rows = min(block_tokens, s.n[b] - q * block_tokens) * group;
      int stop = (int)min((long long)(p.all_tiles + kBlockCost), off + (end - x));
      p.tile = max(off - kBlockCost, 0);
      p.tiles = max(stop - kBlockCost, 0) - p.tile;
      if (p.tiles > kMaxTiles) {  // the rest of the stretch is the next piece
        p.tiles = kMaxTiles;
        stop = p.tile + kMaxTiles + kBlockCost;
        x += stop - off;
        off = stop;
        return true;
      }
      x += stop - off;
      off = 0;
      if ((q + 1) * block_tokens < s.n[b]) {
        q++;
      } else {
        q = 0;
        if (++h == hkv) {
          h = 0;
          do b++;
          while (b < batch && s.n[b] == 0);
        }
      }
      if (p.tiles > 0) return true;
    }
  }
};

template <int F>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(const Params p) {
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int batch = p.rows.batch;
  long long* pre = reinterpret_cast<long long*>(&sm + 1);
  int* len = reinterpret_cast<int*>(pre + batch + 1);
  int* num = len + batch;
  int* row0 = num + batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.q_full[i], 128);
      mbar_init(&sm.k_full[i], kTilePages);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], kTilePages);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 128);
      mbar_init(&sm.p_full[i][1], 128);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.h_done[i], 1);
    }
    mbar_init(&sm.s_full[kOdd], 1);
    mbar_init(&sm.p_full[kOdd][0], 128);
    mbar_init(&sm.p_full[kOdd][1], 128);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.all_done, 1);
    sm.dead = 0;
    fence_barrier_init();
  }
  // TMEM is taken once the kernels in front are done and before the next one may start: whichever
  // of two kernels holds it on an SM never waits for the other.
  grid_dep_wait();
  if (warp == kMmaWarp) tc::alloc(&sm.tmem, 512);

  // ---- the line of all steps; warp 0 finds where this CTA's slice begins
  if (warp == 0) {
    long long sum = 0, all_blocks = 0;
    for (int b0 = 0; b0 < batch; b0 += 32) {
      const int b = b0 + lane;
      NewSpan sp = {0, 0, 0, false};
      int blocks = 0;
      long long tiles = 0;  // places of the sequence's row blocks under one head
      if (b < batch) {
        sp = new_span(p.rows, b);
        if (sp.bad) set_error(p.err, kDevErrCheck);
        len[b] = sp.start + sp.n;
        num[b] = sp.n;
        row0[b] = sp.row0;
        blocks = (sp.n + p.block_tokens - 1) / p.block_tokens;
        if (blocks <= 8)
          for (int q = 0; q < blocks; q++)
            tiles += block_tiles(sp.start + sp.n, sp.n, p.block_tokens, q) + kBlockCost;
      }
      // sequences of many row blocks: the warp together
      for (unsigned many = __ballot_sync(0xffffffffu, blocks > 8); many != 0; many &= many - 1) {
        const int from = __ffs(many) - 1;
        const int n = __shfl_sync(0xffffffffu, sp.n, from);
        const int l = __shfl_sync(0xffffffffu, sp.start, from) + n;
        const int bl = __shfl_sync(0xffffffffu, blocks, from);
        long long t = 0;
        for (int q = lane; q < bl; q += 32)
          t += block_tiles(l, n, p.block_tokens, q) + kBlockCost;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
        if (lane == from) tiles = t;
      }
      long long incl = tiles * p.hkv;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (b < batch) pre[b + 1] = sum + incl;
      sum += __shfl_sync(0xffffffffu, incl, 31);
      all_blocks += (long long)__reduce_add_sync(0xffffffffu, blocks) * p.hkv;
    }
    if (lane == 0) pre[0] = 0;
    __syncwarp();
    // Equal slices, but none so short that joining costs more than it saves: a step of a row block
    // of one tile (few rows; else every slice is longer) is kStepCost, a further part of a row
    // block kPartCost in the joining CTA, so with t tiles a block slices of t' have the least of
    // kStepCost t' + kPartCost t / t'.
    const float mean = all_blocks > 0 ? (float)sum / all_blocks : 0.0f;
    const long long per = max((sum + gridDim.x - 1) / gridDim.x,
                              max((long long)(sqrtf(kPartCost / kStepCost * mean) + 0.5f), 2LL));
    const long long begin = min(blockIdx.x * per, sum);
    if (lane == 0) sm.per = per;
    if (begin < sum) {
      int lo = 0, hi = batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= begin) lo = mid;
        else hi = mid;
      }
      const int b = lo;
      const long long tiles = (pre[b + 1] - pre[b]) / p.hkv;
      const long long at = begin - pre[b];
      const int h = (int)(at / tiles);
      long long rem = at - h * tiles;
      const int blocks = (num[b] + p.block_tokens - 1) / p.block_tokens;
      int q0 = 0;
      for (;; q0 += 32) {  // the block that holds place `rem`
        const int q = q0 + lane;
        const unsigned t =  // 32 blocks' places: at most 2^28
            q < blocks ? block_tiles(len[b], num[b], p.block_tokens, q) + kBlockCost : 0;
        unsigned incl = t;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const unsigned v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, rem < incl);
        if (hit != 0) {
          if (lane == __ffs(hit) - 1) {
            sm.start_b = b;
            sm.start_h = h;
            sm.start_q = q;
            sm.start_off = (int)(rem - (incl - t));
          }
          break;
        }
        rem -= __shfl_sync(0xffffffffu, incl, 31);
        if (q0 + 32 >= blocks) break;
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  grid_dep_launch();
  const uint32_t tmem = sm.tmem;
  const long long per = sm.per, all = pre[batch];
  const long long begin = min(blockIdx.x * per, all), end = min(begin + per, all);
  Walk walk = {{pre, len, num, row0}, batch, p.hkv, p.group, p.block_tokens, begin, end,
               sm.start_b, sm.start_h, sm.start_q, sm.start_off};
  Piece pc;

  if (warp < kSoftmaxWarps) {
    tc::more_registers<kSoftmaxRegs>();
    // ================================================= softmax: one row a thread
    const int tile = warp >> 2, r = tid & 127, row = tile * 128 + r;
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
    const uint32_t o_col = at + kColO + 128 * tile;
    uint32_t s_phase = 0, odd_phase = 0, o_phase = 0, pv_phase = 0, h_phase = 0;
    int step = 0;  // steps of all pieces so far (the ring of scales)
    // After a wait that ran out a warp goes on through the pieces without work: the barriers of
    // a tile's four warps must find all of them.
    bool failed = false;
    // rows of sequences that do not fit: 0 and -inf
    for (int b = blockIdx.x; b < batch; b += gridDim.x) {
      if (p.rows.cu == nullptr ? num[b] != 0 : p.rows.cu[b + 1] - p.rows.cu[b] == num[b]) continue;
      const int first = max(row0[b], 0);
      const int count = min(p.rows.cu ? p.rows.cu[b + 1] : b + 1, p.rows.total) - first;
      for (long long i = tid; i < (long long)count * p.hq * (kHeadDim / 8); i += 256)
        reinterpret_cast<uint4*>(p.out + (size_t)first * p.hq * kHeadDim)[i] =
            make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr)
        for (long long i = tid; i < (long long)count * p.hq; i += 256)
          p.lse[(size_t)first * p.hq + i] = -INFINITY;
    }
    while (walk.next(pc)) {
      const bool two = pc.rows > 128;
      if (tile == 1 && !two) {
        step += pc.tiles;
        continue;
      }
      // ---- the query row in fp16, its largest value in [2^13, 2^14)
      const bool real = row < pc.rows;
      const int token = pc.q * p.block_tokens + row / p.group;  // among the new tokens
      const int head = pc.h * p.group + row % p.group;
      // its position; rows that do not exist (zeros) see everything and are not stored
      const int pos = real ? len[pc.b] - num[pc.b] + token : INT_MAX;
      const size_t out_row = (size_t)(row0[pc.b] + token) * p.hq + head;
      float f;
      // the row's sum starts as NaN where the query has an infinity: its scores may all be -inf,
      // which would look like a row that sees nothing (a NaN makes every score NaN by itself)
      float l;
      {
        const uint4* q = reinterpret_cast<const uint4*>(
            p.q + (long long)(row0[pc.b] + token) * p.q_stride + head * kHeadDim);
        uint4 raw[16];
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < 16; c++) {
          raw[c] = real ? q[c] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int c = 0; c < 16; c++) {
          mx = bf16_max2(mx, bf16_max2(raw[c].x & 0x7FFF7FFFu, raw[c].y & 0x7FFF7FFFu));
          mx = bf16_max2(mx, bf16_max2(raw[c].z & 0x7FFF7FFFu, raw[c].w & 0x7FFF7FFFu));
        }
        const uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
        const int e = m16 >> 7;
        l = e == 255 ? NAN : 0.0f;
        const int shift = (m16 == 0 || e == 255) ? 0 : min(13 + 127 - e, 126);
        const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
        f = p.scale_log2 * __uint_as_float((uint32_t)(127 - shift) << 23);
        unsigned char* dst = sm.q[tile] + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
        for (int c = 0; c < 16; c++) {
          const uint4 w = make_uint4(half_pair(bf16_lo(raw[c].x) * up, bf16_hi(raw[c].x) * up),
                                     half_pair(bf16_lo(raw[c].y) * up, bf16_hi(raw[c].y) * up),
                                     half_pair(bf16_lo(raw[c].z) * up, bf16_hi(raw[c].z) * up),
                                     half_pair(bf16_lo(raw[c].w) * up, bf16_hi(raw[c].w) * up));
          *reinterpret_cast<uint4*>(dst + (c >> 3) * kHalfBytes + (((c & 7) ^ (r & 7)) << 4)) = w;
        }
        fence_proxy_async();
        mbar_arrive(&sm.q_full[tile]);
      }
      // the first position of this tile's rows: tiles of tokens up to it need no mask
      const int first_pos = len[pc.b] - num[pc.b] + pc.q * p.block_tokens +
                            tile * 128 / p.group;
      float m = -INFINITY;
      int j = 0;
      auto scores_ready = [&]() {
        const bool odd = !two && (j & 1);
        if (!wait(sm, &sm.s_full[odd ? kOdd : tile], odd ? odd_phase : s_phase, p.err)) {
          failed = true;
          return false;
        }
        if (odd) odd_phase ^= 1;
        else s_phase ^= 1;
        tc::fence_after();
        return true;
      };
      // One step from half c0 on; returns the half that it stopped before. The plain form stops
      // before a block whose s_v is zero or far from 1: from there on in the piece kApart, in
      // which l is the sum of 2^(x - top_x), not of P / s_v.
      float top_x;
      auto one_step = [&](auto form, int c0) {
        constexpr bool kApart = decltype(form)::value;
        const int base = (pc.tile + j) * kTokens;
        const bool odd = !two && (j & 1);  // one tile: its S and P alternate between the buffers
        const uint32_t s_col = at + kColS + 128 * (odd ? 1 : tile);
        const float4* page = sm.page[step % kPageRing];
        const int limit = pos - base;  // columns up to it are seen
        // ---- S to P, 64 columns at a time (the products with V begin after the first half): a
        // half's maximum comes with its load (in 64 instructions instead, and in a pass of its
        // own over both halves: chunk 792 us, not 756; 8K prompt 480, not 440)
        const bool masked = base + kTokens - 1 > first_pos;
        auto scores = [&](int c, uint32_t (&s)[2][32]) {
          tc::load32(s_col + c * 64, s[0]);
          tc::load32(s_col + c * 64 + 32, s[1]);
          tc::wait_ld();
          if (masked) {
#pragma unroll
            for (int k = 0; k < 64; k++)
              if (c * 64 + k > limit) s[k >> 5][k & 31] = 0xFF800000u;
          }
        };
#pragma unroll 1
        for (int c = c0; c < 2; c++) {
          uint32_t s[2][32], w[32];
          float of[4];  // the blocks' largest scores
          float top = -INFINITY;
          if (!masked) {
#pragma unroll
            for (int g = 0; g < 4; g++)
              tc::load16_max(s_col + c * 64 + g * 16, &s[g >> 1][16 * (g & 1)], of[g]);
            tc::wait_ld();
          } else {
            scores(c, s);
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const uint32_t* v = &s[g >> 1][16 * (g & 1)];
              float a = __uint_as_float(v[0]);
#pragma unroll
              for (int k = 1; k < 15; k += 2)
                a = max3(a, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
              of[g] = fmaxf(a, __uint_as_float(v[15]));
              // a block that the warp's rows may not see: -inf from it would turn into NaN
              if (!kApart && page[4 * c + g].x == INFINITY) top = INFINITY;
            }
          }
          if (kApart) {
            float z = top_x;
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const float4 pg = page[4 * c + g];
              if (pg.y > 0.0f) z = fmaxf(z, of[g] * fmaxf(f * pg.z, kTiny));
            }
            const float ref_x = z == -INFINITY ? 0.0f : z;  // nothing seen so far
            l *= ex2(top_x - ref_x);
            top_x = z;
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const float4 pg = page[4 * c + g];
              const float mul = fmaxf(f * pg.z, kTiny);
              float sum = 0.0f;
#pragma unroll
              for (int k = 0; k < 16; k++)
                sum += ex2(fmaf(__uint_as_float(s[g >> 1][16 * (g & 1) + k]), mul, -ref_x));
              if (pg.y > 0.0f) l += sum;
            }
          }
#pragma unroll
          for (int g = 0; g < 4; g++) {
            const float4 pg = page[4 * c + g];
            top = fmaxf(top, fmaf(of[g], fmaxf(f * pg.z, kTiny), kApart ? pg.w : pg.x));
          }
          // the accumulator follows a maximum that has grown by more than kLag
          if (__any_sync(0xffffffffu, top > m + kLag)) {
            if (!kApart && __any_sync(0xffffffffu, top == INFINITY)) return c;
            top = fmaxf(top, m);
            const float by = m == -INFINITY ? 0.0f : ex2(m - top);
            m = top;
            if (!kApart) l *= by;
            if (j > 0 || c > 0) {
              // the products with V in front are complete: one tile's S may come before the last
              // step's, a second half before the first half's
              if (!two && j > 0 && !wait(sm, &sm.pv_done, pv_phase ^ ((j - 1) & 1), p.err))
                failed = true;
              if (c > 0 && !wait(sm, &sm.h_done[tile], h_phase, p.err)) failed = true;
              if (failed) return c;
              tc::fence_after();
#pragma unroll 1
              for (int k0 = 0; k0 < 8; k0++) {
                uint32_t o[16];
                tc::load16(o_col + k0 * 16, o);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
                tc::store16(o_col + k0 * 16, o);
              }
            }
          }
          const float ref = (m == -INFINITY ? 0.0f : m) - kHeadroom;
#pragma unroll
          for (int g = 0; g < 4; g++) {
            const float4 pg = page[4 * c + g];
            const float add = (kApart ? pg.w : pg.x) - ref, mul = fmaxf(f * pg.z, kTiny);
            const float2 mul2 = make_float2(mul, mul);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const uint32_t* v = &s[g >> 1][16 * (g & 1) + k];
              float2 y = fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), mul2,
                              make_float2(add, add));
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              sum = k == 0 ? y : add2(sum, y);
              w[8 * g + k / 2] = half_pair(y.x, y.y);
            }
            if (!kApart) l = fmaf(sum.x + sum.y, pg.y, l);
          }
          tc::store32(s_col + c * 32, w);
          tc::wait_st();
          tc::fence_before();
          mbar_arrive(&sm.p_full[odd ? kOdd : tile][c]);
        }
        return 2;
      };
      bool apart = false;
      for (; !failed && j < pc.tiles && scores_ready(); j++, step++) {
        int c = 0;
        if (!apart) {
          c = one_step(std::false_type{}, 0);
          if (c < 2 && !failed) {
            apart = true;
            top_x = m - kHeadroom;
          }
        }
        if (apart) one_step(std::true_type{}, c);
        h_phase ^= 1;
      }
      if (!two) pv_phase ^= (pc.tiles - 1) & 1;
      // ---- the result
      if (!wait(sm, &sm.o_full[tile], o_phase, p.err)) failed = true;
      o_phase ^= 1;
      tc::fence_after();
      if (apart) {
        // Back into one frame, within 2^50 of the sum's own: O (the result times the sum, in that
        // frame) and l stay in fp32's range, and of two parts that are joined the frames differ
        // by 2^100 at most beside their sums: a factor that fp32 flushes to 0, below 2^-126,
        // belongs to a part that counts for less than 2^-26.
        const float ref = m - kHeadroom;
        m = fminf(fmaxf(ref, top_x - 50.0f), top_x + 50.0f) + kHeadroom;
        const float to = m - kHeadroom;  // as it is read again
        const bool none = top_x == -INFINITY;
        // in two factors, as one alone may leave the range
        const float by = none ? 1.0f : ex2(0.5f * (ref - to));
        if (!none) l *= ex2(top_x - to);
#pragma unroll 1
        for (int k0 = 0; k0 < 8; k0++) {
          uint32_t o[16];
          tc::load16(o_col + k0 * 16, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 16; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * by * by);
          tc::store16(o_col + k0 * 16, o);
        }
        tc::wait_st();
      }
      const long long tiles_begin = pc.begin + kBlockCost, tiles_end = tiles_begin + pc.all_tiles;
      // of the same stretch: a piece in front of this one, a piece behind it
      const bool after = pc.tile > 0 && tiles_begin + pc.tile > begin;
      const bool before = tiles_begin + pc.tile + pc.tiles < min(tiles_end, end);
      const size_t slot = 2 * (size_t)blockIdx.x + (begin < pc.begin ? 1 : 0);
      float4* const po = reinterpret_cast<float4*>(p.part_o) + slot * 32 * kRows + row;
      float2* const pml = reinterpret_cast<float2*>(p.part_ml);
      if (after) {
        // The piece in front is in the CTA's part, which only this thread reads and writes until
        // the stretch ends: added to this one.
        const float2 was = real ? __ldcg(pml + slot * kRows + row) : make_float2(-INFINITY, 0.0f);
        const float top = fmaxf(m, was.x), ref = top == -INFINITY ? 0.0f : top;
        const float keep = ex2(m - ref), add = ex2(was.x - ref);
        l = l * keep + was.y * add;
        m = top;
#pragma unroll 1
        for (int k0 = 0; k0 < 8; k0++) {
          uint32_t o[16];
          tc::load16(o_col + k0 * 16, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const float4 v =
                real ? __ldcg(po + (k0 * 4 + k) * kRows) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * keep + v.x * add);
            o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * keep + v.y * add);
            o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * keep + v.z * add);
            o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * keep + v.w * add);
          }
          tc::store16(o_col + k0 * 16, o);
        }
        tc::wait_st();
      }
      if (!before && begin <= tiles_begin && tiles_end <= end) {  // the whole row block
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          uint32_t o[32];
          tc::load32(o_col + c * 32, o);
          tc::wait_ld();
          if (real) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; i++)
              w[i] = bf16_pair(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            store_row_part(p.out + out_row * kHeadDim + c * 32, w);
          }
        }
        if (real && p.lse != nullptr)
          p.lse[out_row] = (m - kHeadroom + log2f(l)) * 0.693147180559945309f;
      } else {
        // a part: to the workspace; the last of the block's CTAs to arrive joins them
        const int c0 = (int)(tiles_begin / per);
        const int parts = (int)((tiles_end - 1) / per) - c0 + 1;
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          uint32_t o[32];
          tc::load32(o_col + c * 32, o);
          tc::wait_ld();
          if (real) {
#pragma unroll
            for (int k = 0; k < 8; k++)
              po[(c * 8 + k) * kRows] =
                  make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                              __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
          }
        }
        if (real) pml[slot * kRows + row] = make_float2(m, l);
        if (before) {
          tc::fence_before();
          continue;
        }
        named_sync(1 + tile, 128);
        if (r == 0) {
          int* counter = p.counters + 2 * c0 + tile;
          const int last = atomic_add_acq_rel_gpu(counter, 1) == parts - 1;
          if (last) *counter = 0;
          sm.last[tile] = last;
        }
        named_sync(1 + tile, 128);
        if (sm.last[tile] && real) {
          const size_t first = 2 * (size_t)c0 + (c0 * per < pc.begin ? 1 : 0);
          auto slot_of = [&](int c) { return c == 0 ? first : 2 * (size_t)(c0 + c); };
          float top = -INFINITY, sum = 0.0f;
          for (int c = 0; c < parts; c++)
            top = fmaxf(top, __ldcg(pml + slot_of(c) * kRows + row).x);
          const float ref = top == -INFINITY ? 0.0f : top;
          for (int c = 0; c < parts; c++) {
            const float2 v = __ldcg(pml + slot_of(c) * kRows + row);
            sum += ex2(v.x - ref) * v.y;
          }
          const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll 1
          for (int c4 = 0; c4 < 4; c4++) {  // 32 channels at a time
            float4 acc[8];
#pragma unroll
            for (int k = 0; k < 8; k++) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float4* src =
                reinterpret_cast<const float4*>(p.part_o) + c4 * 8 * kRows + row;
            for (int c = 0; c < parts; c += 2) {  // two parts' loads under way at once
              const bool two = c + 1 < parts;
              const size_t s0 = slot_of(c), s1 = two ? slot_of(c + 1) : s0;
              float4 v[2][8];
              const float m0 = __ldcg(pml + s0 * kRows + row).x;
              const float m1 = __ldcg(pml + s1 * kRows + row).x;
#pragma unroll
              for (int k = 0; k < 8; k++) {
                v[0][k] = __ldcg(src + (s0 * 32 + k) * kRows);
                v[1][k] = __ldcg(src + (s1 * 32 + k) * kRows);
              }
              const float w[2] = {ex2(m0 - ref) * inv, two ? ex2(m1 - ref) * inv : 0.0f};
#pragma unroll
              for (int h = 0; h < 2; h++)
#pragma unroll
                for (int k = 0; k < 8; k++) {
                  acc[k].x += w[h] * v[h][k].x;
                  acc[k].y += w[h] * v[h][k].y;
                  acc[k].z += w[h] * v[h][k].z;
                  acc[k].w += w[h] * v[h][k].w;
                }
            }
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 8; k++) {
              w[2 * k] = bf16_pair(acc[k].x, acc[k].y);
              w[2 * k + 1] = bf16_pair(acc[k].z, acc[k].w);
            }
            store_row_part(p.out + out_row * kHeadDim + c4 * 32, w);
          }
          if (p.lse != nullptr)
            p.lse[out_row] = (top - kHeadroom + log2f(sum)) * 0.693147180559945309f;
        }
      }
      tc::fence_before();
    }
  } else if (warp < kMmaWarp) {
    tc::fewer_registers<kConvertRegs>();
    // ================================================= codes to fp16 tiles
    // Warp w turns block w of each tile, of K and of V. Lane: 8 channels of tokens 2 i +
    // lane / 16. Pages and scales of 32 tiles ahead are fetched at once, one tile a lane, and
    // the codes of the next step are under way while this one's are converted.
    const int w = warp - kSoftmaxWarps, sub = lane >> 4, ch = lane & 15;
    uint32_t off[4];  // of token 2 i + sub, i < 4, in the block's part of the tile
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int t = 2 * i + sub;
      off[i] = w * (kPage * 128) + (ch >> 3) * kHalfBytes + t * 128 + (((ch & 7) ^ t) << 4);
    }
    struct Ahead {      // 32 tiles of a piece
      int count;        // of them, in the piece (0: the end)
      int block;        // this lane's tile: the block in the code arrays
      int valid;        // its first tokens that exist
      float sk, sv;
    };
    bool more = walk.next(pc);
    int done = 0;  // tiles of the piece that were fetched
    auto fetch = [&]() {
      Ahead a = {0, 0, 0, 0.0f, -1.0f};
      if (!more) return a;
      a.count = min(pc.tiles - done, 32);
      const int i = (pc.tile + done + lane) * kTilePages + w;
      if (lane < a.count) {
        a.valid = min(max(len[pc.b] - i * kPage, 0), kPage);
        if (a.valid > 0) {
          const int page = p.page_table[(size_t)pc.b * p.rows.max_pages + i];
          if (page >= 0 && page < p.num_pages) {
            a.block = page * p.hkv + pc.h;
            a.sk = p.k_scale[a.block];
            a.sv = p.v_scale[a.block];
          } else {
            set_error(p.err, kDevErrCheck);
            a.valid = 0;
          }
        }
      }
      done += a.count;
      if (done == pc.tiles) {
        done = 0;
        more = walk.next(pc);
      }
      return a;
    };
    auto load = [&](const uint8_t* codes, const Ahead& a, int j, uint2 (&raw)[8]) {
      const int valid = __shfl_sync(0xffffffffu, a.valid, j);
      const uint8_t* src = codes +
                           (size_t)__shfl_sync(0xffffffffu, a.block, j) * kBlockBytesI8 +
                           sub * kHeadDim + ch * 8;
      if (valid == kPage) {
#pragma unroll
        for (int i = 0; i < 8; i++) raw[i] = ldg64_nc(src + 2 * i * kHeadDim);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          raw[i] = make_uint2(0u, 0u);
          if (2 * i + sub < valid) raw[i] = ldg64_nc(src + 2 * i * kHeadDim);
        }
      }
    };
    auto put = [&](unsigned char* tile, const uint2 (&raw)[8]) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const uint32_t x = Codes<F>::prepare(raw[i].x), y = Codes<F>::prepare(raw[i].y);
        *reinterpret_cast<uint4*>(tile + off[i & 3] + (i >> 2) * 1024) =
            make_uint4(Codes<F>::template pair<0>(x), Codes<F>::template pair<1>(x),
                       Codes<F>::template pair<0>(y), Codes<F>::template pair<1>(y));
      }
      fence_proxy_async();
      __syncwarp();
    };
    Ahead cur = fetch(), next = fetch();
    uint2 rk[8], rv[8];
    if (cur.count > 0) {
      load(p.k, cur, 0, rk);
      load(p.v, cur, 0, rv);
    }
    int step = 0;
    bool ok = true;
    while (ok && cur.count > 0) {
      for (int j = 0; j < cur.count; j++, step++) {
        const int st = step & 1, parity = ((step >> 1) & 1) ^ 1;
        const bool turn = j + 1 == cur.count;  // the next step is the next 32's first
        const bool another = !turn || next.count > 0;
        const int nj = turn ? 0 : j + 1;
        ok = wait(sm, &sm.k_empty[st], parity, p.err);
        if (!ok) break;
        const float sk = __shfl_sync(0xffffffffu, cur.sk, j);
        const float sv = __shfl_sync(0xffffffffu, cur.sv, j);
        if (lane == 0) {
          const float log = lg2(sv);
          sm.page[step % kPageRing][w] =
              sv < 0.0f ? make_float4(-INFINITY, 0.0f, sk, -INFINITY)
                        : make_float4(fabsf(log) <= kPlainScale ? log : INFINITY,
                                      sv == 0.0f ? 1.0f : 1.0f / sv, sk, log);
        }
        put(sm.k[st], rk);
        if (lane == 0) mbar_arrive(&sm.k_full[st]);
        if (another) load(p.k, turn ? next : cur, nj, rk);
        ok = wait(sm, &sm.v_empty[st], parity, p.err);
        if (!ok) break;
        put(sm.v[st], rv);
        if (lane == 0) mbar_arrive(&sm.v_full[st]);
        if (another) load(p.v, turn ? next : cur, nj, rv);
      }
      cur = next;
      next = fetch();
    }
  } else {
    tc::fewer_registers<kMmaRegs>();
  }
  if (warp == kMmaWarp) {
    // ================================================= the products
    constexpr uint32_t kQk = tc::instr_f16(128, kTokens, false);
    constexpr uint32_t kPv = tc::instr_f16(128, kHeadDim, true);
    const uint32_t q_low = tc::desc_low(smem_addr(sm.q[0]), 16);
    const uint32_t k_low = tc::desc_low(smem_addr(sm.k[0]), 16);
    const uint32_t v_low = tc::desc_low(smem_addr(sm.v[0]), kHalfBytes);
    const bool lead = tc::elect();
    int step = 0;
    uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0}, odd_phase = 0;
    bool ok = true;
    // S of tile i against the K tile of step `at`, into buffer `buf`
    auto scores = [&](int i, int buf, int at, uint64_t* full) {
      if (lead) {
        const uint32_t q = q_low + i * (kTileBytes >> 4), k = k_low + (at & 1) * (kTileBytes >> 4);
#pragma unroll
        for (int c = 0; c < 8; c++) {
          const uint32_t off = ((c >> 2) * kHalfBytes + (c & 3) * 32) >> 4;
          tc::mma_ss<kQk>(tmem + kColS + 128 * buf, q + off, k + off, c > 0);
        }
        tc::commit(full);
      }
    };
    // O of tile i += P V of half h of step `at`, P in buffer `buf`
    auto values = [&](int i, int buf, int h, int at, bool add) {
      if (lead) {
        const uint32_t v = v_low + (at & 1) * (kTileBytes >> 4);
#pragma unroll
        for (int c = 4 * h; c < 4 * h + 4; c++)
          tc::mma_ts<kPv>(tmem + kColO + 128 * i, tmem + kColS + 128 * buf + c * 8,
                          v + c * (2048 >> 4), add || c > 0);
      }
    };
    while (ok && walk.next(pc)) {
      const bool two = pc.rows > 128;
      ok = wait(sm, &sm.k_full[step & 1], (step >> 1) & 1, p.err);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if (!ok || (i == 1 && !two)) continue;
        ok = wait(sm, &sm.q_full[i], q_phase[i], p.err);
        if (!ok) continue;
        q_phase[i] ^= 1;
        tc::fence_after();
        scores(i, i, step, &sm.s_full[i]);
      }
      if (!ok) break;
      if (lead) tc::commit(&sm.k_empty[step & 1]);
      // One tile: the next step's scores go into the other tile's buffer of S while this step's
      // are in the softmax, which then never waits for them (pv_done: see there).
      for (int j = 0; ok && !two && j < pc.tiles; j++, step++) {
        const bool more = j + 1 < pc.tiles;
        const int buf = j & 1;
        if (more) {
          ok = wait(sm, &sm.k_full[(step + 1) & 1], ((step + 1) >> 1) & 1, p.err);
          if (!ok) break;
          tc::fence_after();
          scores(0, buf ^ 1, step + 1, &sm.s_full[buf ? 0 : kOdd]);
          if (lead) tc::commit(&sm.k_empty[(step + 1) & 1]);
        }
        ok = wait(sm, &sm.v_full[step & 1], (step >> 1) & 1, p.err);
        uint64_t* const full = sm.p_full[buf ? kOdd : 0];
        const uint32_t phase = buf ? odd_phase : p_phase[0];
        if (ok) ok = wait(sm, full, phase, p.err);
        if (!ok) break;
        tc::fence_after();
        values(0, buf, 0, step, j > 0);
        if (lead) tc::commit(&sm.h_done[0]);
        ok = wait(sm, full + 1, phase, p.err);
        if (!ok) break;
        if (buf) odd_phase ^= 1;
        else p_phase[0] ^= 1;
        tc::fence_after();
        values(0, buf, 1, step, true);
        if (lead) {
          tc::commit(more ? &sm.pv_done : &sm.o_full[0]);
          tc::commit(&sm.v_empty[step & 1]);
        }
        __syncwarp();
      }
      for (int j = 0; ok && two && j < pc.tiles; j++, step++) {
        const bool more = j + 1 < pc.tiles;
        ok = wait(sm, &sm.v_full[step & 1], (step >> 1) & 1, p.err);
        if (ok && more) ok = wait(sm, &sm.k_full[(step + 1) & 1], ((step + 1) >> 1) & 1, p.err);
#pragma unroll
        for (int i = 0; i < 2; i++) {
          if (!ok || (i == 1 && !two)) continue;
          ok = wait(sm, &sm.p_full[i][0], p_phase[i], p.err);
          if (!ok) continue;
          tc::fence_after();
          values(i, i, 0, step, j > 0);
          if (lead) tc::commit(&sm.h_done[i]);
          ok = wait(sm, &sm.p_full[i][1], p_phase[i], p.err);
          if (!ok) continue;
          p_phase[i] ^= 1;
          tc::fence_after();
          values(i, i, 1, step, true);
          if (more) scores(i, i, step + 1, &sm.s_full[i]);
          else if (lead) tc::commit(&sm.o_full[i]);
        }
        if (ok && lead) {
          tc::commit(&sm.v_empty[step & 1]);
          if (more) tc::commit(&sm.k_empty[(step + 1) & 1]);
        }
        __syncwarp();
      }
    }
    // the last arrivals on the barriers come before the CTA ends
    if (ok && step > 0) {
      wait(sm, &sm.k_empty[(step - 1) & 1], ((step - 1) >> 1) & 1, p.err);
      wait(sm, &sm.v_empty[(step - 1) & 1], ((step - 1) >> 1) & 1, p.err);
    }
    // nor may products go on in shared and tensor memory that are given up
    if (!ok) {
      if (lead) tc::commit(&sm.all_done);
      mbar_wait(&sm.all_done, 0);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

size_t smem_bytes(int batch) {
  return 1024 + sizeof(Smem) + 8 * (size_t)(batch + 1) + 12 * (size_t)batch;
}

}  // namespace

size_t kv8_prefill_part_floats() { return (size_t)2 * kKv8MaxCtas * kRows * kHeadDim; }
size_t kv8_prefill_ml_floats() { return (size_t)2 * kKv8MaxCtas * kRows * 2; }

cudaError_t launch_kv8_prefill(const Shape& s, const Kv8& c, const void* q, long long q_stride,
                               const int32_t* cu, int total, const int32_t* page_table,
                               const int32_t* seq_lens, void* out, float* lse, int* counters,
                               float* part_ml, float* part_o, int* err, int num_sms,
                               cudaStream_t st) {
  Params p;
  p.rows = NewRows{cu, seq_lens, s.batch, total, s.max_pages};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.page_table = page_table;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part_ml = part_ml;
  p.part_o = part_o;
  p.counters = counters;
  p.err = err;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.group = s.group;
  p.num_pages = s.num_pages;
  p.block_tokens = kRows / s.group;
  p.scale_log2 = s.sm_scale * 1.44269504088896341f;
  auto kernel = c.format == kE4m3 ? kv8_prefill_kernel<kE4m3> : kv8_prefill_kernel<kInt8>;
  const size_t smem = smem_bytes(s.batch);
  const cudaError_t e = set_kernel_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(std::min(num_sms, kKv8MaxCtas)), dim3(kThreads), smem, st,
                       true, p);
}

}  // namespace hsa
