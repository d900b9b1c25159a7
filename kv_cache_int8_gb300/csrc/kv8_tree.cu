// kv8_tree.cu -- attention of drafted tokens over the 8-bit K/V cache: node i of a sequence's tree
// sees the context in front of the tree, itself and its ancestors.
//
// Source: "KV Cache 与长上下文推理", section "KV Cache 回顾" (decode attention equation), section
// "KV Cache 量化"; the pages have no drafted tokens.
//
// Mathematics. As in the prompt attention, the codes enter the products exactly (fp16) and the
// blocks' scales (16 tokens) are applied in fp32: with row factor f = sm_scale log2 e 2^-shift,
//   x_t = f s_k S_t    y_t = x_t + log2 s_v
//   out = sum_t 2^(y_t - M) c_t / sum_t 2^(x_t - M)
// The sum takes 2^(y - M) / s_v, one factor a token, as long as every s_v is within 2^-40 ..
// 2^40; from the first step on that has another (or a block of zeros), a second form of the step
// sums 2^x under a maximum of its own. P = 2^(y - M + 7) is rounded to fp16 (11 bits, against 8 of
// the bf16 result: one product with V and 16 KB of shared memory a buffer, where two numbers would
// take two and 32), below 2^-14 to steps of 2^-24: a weight is off by 2^-11 of itself or by 2^-32
// of the row's largest, and the sum, which takes the fp32 numbers, keeps what P loses. n tokens lose
// n 2^-32 of the largest value at most: 2^-12 at 1M. M lags the running maximum by at most 8.
//
// Layout. A tree is few rows against many tokens (a kv head's group of query heads x the nodes:
// up to 128 rows here), so the products are turned round: the tokens are the 128 rows of the
// tensor core's tile and the queries its columns,
//   S^T [128 tokens][64 queries] = K Q^T        O^T [128 channels][64 queries] += V^T P^T
// and everything but the turning of codes into fp16 costs what there are queries. A lane has the
// scores of four tokens (of two blocks: its scales are a few numbers) and sixteen rows, whose sums
// and maxima stay in registers; the maxima are only looked at (one vote of 128 threads a step), and
// found when a score passes the lag. The codes of K and V
// become left operands in tensor memory, V's turned on the way (ldmatrix on bytes), so shared
// memory, whose bandwidth the products' right operands need, sees each code twice.
//   warps 0-3, 4-7: the softmax of two streams. More than 64 rows: each has its rows of every step;
//     up to 64: both have all rows and take the steps in turn, with a maximum, a sum and an O of
//     its own, joined where the rows end.
//   warps 8-11 K's codes, 12-15 V's, warp 16 the products, 17 and 18 the copies (TMA, a block
//     each) of K and V, several steps ahead.
// Tensor memory: S 2 streams x 2 steps x 64 columns, O 2 x 64, K 64, V 64 (while the products with
// one of them run, the other's next codes come in). Shared memory: the queries 32 KB, three steps of
// codes 96, two of P for each stream 64.
//
// Bounds. Memory, for few rows: the codes of a step are 32 KB, 0.73 us of one SM's share of 6.8 TB/s.
// 600K tokens of 8 heads (1.23 GB, 181 us at 6.8 TB/s) take 233 us where only the copies run, 262
// with 64 rows and 340 with 128, where the chain scores -> exponentials -> P of a stream is the
// longest: 1.3 us a step; tensor pipe 30 %, issue slots 53 %, exponentials 15 % busy. A call's fixed
// part is 14 us:
// lengths, plan, queries and the first copies 7.5, the first maxima 2, the results 2, the joining
// kernel 2 to 3. 8 nodes of 4 heads over 8K tokens 14.4 us, 25 nodes of 32 heads over 128K 88,
// 8 x 6-15 nodes of 64 heads over 32-128K tokens 390 (1.41 GB, 3.6 TB/s), 4 chats of 7-24 nodes 39.
// The other forms of a step are for rare data and far from that: with one block of V in 64 of another
// scale (or of zeros) 330 us behind 128K where all alike take 83, with queries of 2^10 194 (far
// scores). The kernel spills 80 bytes a thread (stack of 40).
//
// Work. All steps (row block, token tile) of all sequences and heads form one line, cut into equal
// slices, one CTA each; the parts of a row block that is cut go through the workspace to a second
// kernel that joins them, so that joining takes all SMs and no CTA waits.
#include <climits>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "kv8.cuh"
#include "tcgen05.cuh"

namespace hsa {
namespace {

using namespace kv8_detail;

constexpr int kRows = 128;        // rows of a block
constexpr int kStreamRows = 64;   // of a stream: columns of its S and O
constexpr int kTokens = 128;      // tokens of a step
constexpr int kTilePages = kTokens / kPage;
constexpr int kTileBytes = kRows * kHeadDim * 2;      // the queries
constexpr int kHalfBytes = kTileBytes / 2;            // 64 channels of 128 rows
constexpr int kRawBytes = kTokens * kHeadDim;         // codes of a step, of K or V
constexpr int kPBytes = kTokens * kStreamRows * 2;
constexpr int kStages = 3;                            // steps of raw codes, of K and of V
constexpr int kPageRing = 16;                         // steps whose scales are kept (see Smem)
constexpr int kPieces = 4;                            // pieces told ahead
constexpr int kKWarp = 8, kVWarp = 12, kMmaWarp = 16, kKLoad = 17, kVLoad = 18, kPlanWarp = 19;
constexpr int kThreads = 640;
// registers a thread: softmax warpgroups, converting ones, the last; 96 on average
constexpr int kSoftmaxRegs = 144, kConvertRegs = 72, kOtherRegs = 48;
static_assert(2 * kSoftmaxRegs + 2 * kConvertRegs + kOtherRegs == 5 * 96, "the launch's registers");
constexpr float kHeadroom = 7.0f, kLag = 8.0f;  // P up to 2^15
constexpr float kPlainScale = 40.0f; // largest |log2 s_v| of the plain form
constexpr float kTiny = 1e-37f;      // smallest factor of a score: a masked -inf stays one
constexpr float kLow = -3.4e38f;     // a maximum before any score
// Places on the line of steps (see the plan): a tile's, with one stream on it and with two, a row
// block's beside its tiles, and the shortest slice. In the order of their times: 600K tokens of 8
// heads take 262 us with 64 rows, 340 with 128. With 2 and 3 places a tile 8 x 32-128K tokens of 48
// to 120 rows take 420 us, with 3 and 4 391, 4 and 5 394, 5 and 7 396; 4 chats of 28 to 96 rows 38.2,
// 40.2, 38.8, 39.9. A block's are 11 tiles': with 3, 6, 11 and 18 those chats take 42.6, 41.0, 38.8
// and 41.4 us, 25 nodes behind 128K 89, 87, 82 and 82, 16 x 2K tokens 43.8, 43.6, 40.8 and 40.6, 64 x
// 4K 160, 159, 157 and 159, 600K tokens of 128 rows 332, 324, 326 and 327. Slices of 5 places at least
// take as long as of 8 everywhere, of 16 and 32 longer where they are short (8K tokens of one head
// 15.9 and 18.9 us, not 14.4).
constexpr int kTilePlaces = 4, kTwoPlaces = 5, kBlockPlaces = 44, kMinPlaces = 8;
static_assert(kMinPlaces >= kTwoPlaces, "no slice without the first place of a tile");
// O takes the products of at most this many steps: their own sums round to zero, 2^-23 a product
constexpr int kMaxSteps = 256;
// Of a step: an s_v that the plain form does not take; the exponent of its largest s_k (from bit 1
// on); a block without tokens.
constexpr int kFarScale = 1, kHidden = 1 << 16;
// A score is within 2^30 of its factors f s_k (128 channels of 2^14 by 2^9). Where f s_k is 2^-6 or
// more that is 2^24, and fp32's rounding of scores could come near the lag: the step is taken in
// the form that rounds them first.
constexpr int kFarFactors = 247;  // the sum of the two biased exponents
constexpr uint32_t kColS = 0, kColO = 256, kColK = 384, kColV = 448;

struct Record {  // a row block that begins in a CTA's slice and goes on behind it
  int rows, parts;
  int slot0, cta;  // the first part's slot; the CTA
  int row0, head0; // q's row of its first node, its first query head
  int pad[2];
};

struct Params {
  NewRows rows;
  const __nv_bfloat16* q;
  long long q_stride;
  const float* k_scale;
  const float* v_scale;
  const int32_t* parents;
  const int32_t* page_table;
  __nv_bfloat16* out;
  float* lse;
  float* part_ml;  // [2 CTAs][kRows] (M, l)
  float* part_o;   // [2 CTAs][kRows][kHeadDim]
  Record* records; // [CTAs]
  int* err;
  int hq, hkv, group, num_pages, block_nodes;  // block_nodes: most nodes of a row block
  float scale_log2;
};

// A stretch of one row block's tiles: what a CTA does at a time.
struct alignas(16) Piece {
  int tiles;         // 0: no more
  int tile;          // the first
  int rows;          // nodes x group
  int b, h;          // sequence, kv head
  int n_all, start;  // its tokens, those in front of the tree
  int node;          // the first node
  int row0;          // q's row of node 0
  int flags;         // kWhole ..
  int slot;          // of the parts
  int parts;         // kRecord: how many
};
// the whole row block; a piece of the same stretch in front; the first part, to be recorded; other
// row blocks read the same tokens
constexpr int kWhole = 1, kAfter = 2, kRecord = 4, kShared = 8;

struct Smem {
  alignas(1024) unsigned char q[kTileBytes];
  unsigned char p[2][2][kPBytes];  // two steps' of a stream each; between row blocks its scratch
  unsigned char k_raw[kStages][kRawBytes];
  unsigned char v_raw[kStages][kRawBytes];
  // Of a step's blocks: y = 1 / s_v (any number above 0 for zeros, 0 where there are no tokens);
  // z = s_k; w = log2 s_v (-inf for both). The copies of a step begin when the codes three steps
  // back are read, so when the scores five back are complete; their buffer was read by its
  // stream's softmax two of its own steps before, at most nine back, and the other stream's ten
  // back.
  float4 page[kPageRing][kTilePages];
  int flags[kPageRing];            // of a step: see kFarScale
  uint32_t seen[kKv8TreeNodes][kRows / 32];  // of each node: the rows that see it
  float c[2][kStreamRows];         // kHeadroom - m
  float m[2][kStreamRows];         // the rows' maxima
  float mx[2][kStreamRows];        // those under which the second form's sums are kept
  float by[2][kStreamRows];
  float f[kRows];                  // row factors (NaN where the query is not finite)
  float red[2][4][kStreamRows];    // of a stream's warps: maxima, then sums
  alignas(8) int v_valid[kStages][kTilePages];
  Piece piece[kPieces];
  alignas(8) uint64_t q_full, k_raw_full[kStages], k_raw_empty[kStages], v_raw_full[kStages],
      v_raw_empty[kStages], k_full, k_empty, v_full, v_empty, s_full[2][2], s_empty[2][2], p_full[2][2],
      pv_done[2][2], piece_full[kPieces], piece_empty[kPieces], all_done;
  uint32_t tmem;
  int2 exponents[kKWarp];
  int far;  // flags from here on: hidden tokens, or scores that may be far from 0
  int dead;
};
// behind it: len, n, row0, block_nodes, blocks (int [batch] each)

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
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 values in a pair of registers.
typedef unsigned long long F2;
__device__ __forceinline__ F2 pack(float lo, float hi) {
  F2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ F2 pack(const uint32_t* v) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(v[0]), "r"(v[1]));
  return r;
}
__device__ __forceinline__ F2 pack(float2 v) { return pack(v.x, v.y); }
__device__ __forceinline__ float2 unpack(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 m, F2 c) {
  F2 y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(a), "l"(m), "l"(c));
  return y;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 y;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 y;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
  return y;
}
__device__ __forceinline__ float2 ex2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// a barrier that tells whether any of its threads says so
__device__ __forceinline__ bool any_of(int id, int threads, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(id), "r"(threads), "r"((uint32_t)x)
      : "memory");
  return y != 0;
}

// 16 lanes x 32 columns of tensor memory: lane l gets columns 8 i + 2 (l % 4) + {0, 1} of rows l / 4
// (r[4 i], r[4 i + 1]) and l / 4 + 8 (r[4 i + 2], r[4 i + 3]), i < 4; tc::wait_ld() before use.
__device__ __forceinline__ void load_16x32(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}

// Four 8 x 8 matrices of 16-bit values: lane l points at row l % 8 of matrix l / 8 and holds, of each,
// row l / 4's values 2 (l % 4), + 1.
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                               uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Two 16 x 16 byte matrices, turned: lanes 0 .. 15 and 16 .. 31 point at their rows (tokens); lane
// l gets, of each, the bytes of rows 4 (l % 4) .. + 3 in columns (channels) l / 4 and l / 4 + 8.
__device__ __forceinline__ void load_turned(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 32 lanes x 8 columns, one lane's a lane; tc::wait_ld() before use.
__device__ __forceinline__ void load8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(addr));
}

// 16 lanes x 64 columns of tensor memory: lane l has columns 8 i + 2 (l % 4) + {0, 1} of rows l / 4
// (r[4 i], r[4 i + 1]) and l / 4 + 8 (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void store_16x64(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x8.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10,"
      " %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28,"
      " %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

// Waits with a limit (4 to 8 billion cycles); once a wait has run out every wait of the CTA gives
// up (false). What goes on then works on whatever is there, in bounds: a piece is always gone
// through to its end, as its barriers must find all threads.
__device__ __forceinline__ uint32_t clock_hi() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%clock_hi;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool wait(Smem& sm, uint64_t* bar, uint32_t parity) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint32_t t0 = clock_hi();
    while (!(ok = mbar_try_wait(bar, parity))) {
      if (*reinterpret_cast<volatile int*>(&sm.dead)) break;
      if (clock_hi() - t0 > 1) *reinterpret_cast<volatile int*>(&sm.dead) = 1;
    }
  }
  __syncwarp();
  return ok;
}

// Row blocks of a sequence of n nodes, as equal as they come: the nodes of each.
__device__ __forceinline__ int nodes_a_block(int n, int most) {
  const int blocks = max((n + most - 1) / most, 1);
  return (n + blocks - 1) / blocks;
}
__device__ __forceinline__ int token_tiles(int len) { return (len + kTokens - 1) / kTokens; }

template <int F>
__global__ void __launch_bounds__(kThreads, 1)
    kv8_tree_kernel(const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const Params p) {
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int batch = p.rows.batch;
  int* len = reinterpret_cast<int*>(&sm + 1);
  int* num = len + batch;
  int* row0 = num + batch;
  int* block_nodes = row0 + batch;
  int* blocks = block_nodes + batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    tma_prefetch_descriptor(&k_map);
    tma_prefetch_descriptor(&v_map);
    mbar_init(&sm.q_full, 256);
    for (int i = 0; i < kStages; i++) {
      mbar_init(&sm.k_raw_full[i], 1);
      mbar_init(&sm.k_raw_empty[i], 4);
      mbar_init(&sm.v_raw_full[i], 1);
      mbar_init(&sm.v_raw_empty[i], 4);
    }
    mbar_init(&sm.k_full, 128);
    mbar_init(&sm.k_empty, 1);
    mbar_init(&sm.v_full, 128);
    mbar_init(&sm.v_empty, 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(&sm.s_full[i][0], 1);
      mbar_init(&sm.s_full[i][1], 1);
      mbar_init(&sm.s_empty[i][0], 128);
      mbar_init(&sm.s_empty[i][1], 128);
      mbar_init(&sm.p_full[i][0], 128);
      mbar_init(&sm.p_full[i][1], 128);
      mbar_init(&sm.pv_done[i][0], 1);
      mbar_init(&sm.pv_done[i][1], 1);
    }
    for (int i = 0; i < kPieces; i++) {
      mbar_init(&sm.piece_full[i], 1);
      mbar_init(&sm.piece_empty[i], kPlanWarp);
    }
    mbar_init(&sm.all_done, 1);
    sm.dead = 0;
    fence_barrier_init();
  }
  // TMEM is taken once the kernels in front are done and before the next one may start: whichever
  // of two kernels holds it on an SM never waits for the other.
  grid_dep_wait();
  if (warp == kMmaWarp) tc::alloc(&sm.tmem, 512);
  for (int b = tid; b < batch; b += kThreads) {
    NewSpan sp = new_span(p.rows, b);
    if (sp.n > kKv8TreeNodes) {
      sp.bad = true;
      sp.n = 0;
    }
    if (sp.bad) set_error(p.err, kDevErrCheck);
    len[b] = sp.start + sp.n;
    num[b] = sp.n;
    row0[b] = sp.row0;
    // row blocks, as equal as they come
    const int most = max(nodes_a_block(sp.n, p.block_nodes), 1);
    block_nodes[b] = most;
    blocks[b] = (sp.n + most - 1) / most;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  grid_dep_launch();  // the joining kernel, whose CTAs take the places of those that end
  const uint32_t tmem = sm.tmem;
  // The pieces, as the plan's warp tells them; every other warp takes each and gives it back.
  int pieces = 0;
  auto take = [&](Piece& pc) {
    const int slot = pieces % kPieces;
    wait(sm, &sm.piece_full[slot], pieces / kPieces & 1);
    pc = sm.piece[slot];
    if (sm.dead) pc.tiles = 0;
    return __shfl_sync(0xffffffffu, pc.tiles, 0) > 0;
  };
  auto give_back = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.piece_empty[pieces % kPieces]);
    pieces++;
  };
  Piece pc;

  if (warp < kKWarp) {
    tc::more_registers<kSoftmaxRegs>();
    // ============================================ softmax
    const int st = warp >> 2, t = tid & 127;
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
    // A lane's share of a step, as the 16-lane loads give it: of each half h of its warp's 32 tokens
    // (a block of the cache) tokens tok + 8 i, and rows 8 b + col, + 1 of every b.
    const int tok = 32 * (warp & 3) + (lane >> 2), col = 2 * (lane & 3);
    // where it points stmatrix at, of P's rows 0 .. 15: token 32 w + (lane & 8) + lane % 8
    const uint32_t p_row = smem_addr(sm.p[0][st]) + (32 * (warp & 3) + (lane & 15)) * 128;
    const uint32_t p_chunk = ((lane >> 4) ^ (lane & 7)) << 4;
    uint32_t p_phase = 0;  // bit i: of buffer i of its P, uses so far
    uint32_t s_phase = 0;  // bit i: of buffer i of its S
    int step0 = 0;         // steps of the pieces so far
    for (;;) {
      const bool more = take(pc);
      // the row block before is read out of shared and tensor memory; after a wait that ran out all
      // leave together
      if (any_of(1, 256, !more)) break;
      const bool two = pc.rows > kStreamRows;
      const int base_row = two ? kStreamRows * st : 0;
      const int rows = min(pc.rows - base_row, kStreamRows);  // of this stream
      const bool wide = rows > 32;
      const int q_row = pc.row0 + pc.node;
      const bool branches = (pc.tile + pc.tiles) * kTokens > pc.start;
      if (branches) *reinterpret_cast<uint4*>(sm.seen[tid]) = make_uint4(0u, 0u, 0u, 0u);
      if (t < kStreamRows) {
        sm.m[st][t] = kLow;
        sm.mx[st][t] = kLow;
        sm.c[st][t] = kHeadroom - kLow;
      }
      // ---- the queries in fp16, four threads a row. All rows under one power of two that puts
      // the largest value in [2^13, 2^14), as long as the smallest row's largest is within 2^-15
      // of it: its largest is then 2^-2 or more, its values down to 2^-15 of that are exact in fp16,
      // and smaller ones, in steps of 2^-24, are off by 2^-25 or less, 2^-23 of it. Else each row
      // under its own, and the second form of the step.
      auto query = [&](int r) {
        return p.q + (long long)(q_row + r / p.group) * p.q_stride +
               (pc.h * p.group + r % p.group) * kHeadDim + (tid & 3) * 32;
      };
      auto exponent = [&](const uint4 (&v)[4]) {  // of the row's largest value; 0: zeros, 255: none
        uint32_t mx = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          mx = __vmaxu2(mx, __vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu));
          mx = __vmaxu2(mx, __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
        }
        uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
        m16 = max(m16, __shfl_xor_sync(0xffffffffu, m16, 1));
        m16 = max(m16, __shfl_xor_sync(0xffffffffu, m16, 2));
        return m16 == 0 ? -1 : (int)(m16 >> 7);
      };
      uint4 raw[2][4];
      int e[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int r = (tid >> 2) + 64 * i;
#pragma unroll
        for (int k = 0; k < 4; k++)
          raw[i][k] = r < pc.rows ? reinterpret_cast<const uint4*>(query(r))[k]
                                  : make_uint4(0u, 0u, 0u, 0u);
      }
      {
        int most = 0, least = 255;
#pragma unroll
        for (int i = 0; i < 2; i++) {
          e[i] = exponent(raw[i]);
          if (e[i] >= 0 && e[i] < 255) {
            most = max(most, e[i]);
            least = min(least, e[i]);
          }
        }
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane == 0) sm.exponents[warp] = make_int2(most, least);
      }
      named_sync(1, 256);
      // which rows see a node: its own, and those of the nodes below it
      if (branches && tid < pc.rows) {
        const int32_t* parents = p.parents ? p.parents + pc.row0 : nullptr;
        for (int i = pc.node + tid / p.group; i >= 0;) {
          atomicOr(&sm.seen[i][tid >> 5], 1u << (tid & 31));
          const int up = parents ? parents[i] : i - 1;
          if (up < -1 || up >= i) {
            set_error(p.err, kDevErrCheck);
            break;
          }
          i = up;
        }
      }
      int e_max = 0, e_min = 255;
#pragma unroll
      for (int k = 0; k < kKWarp; k++) {
        e_max = max(e_max, sm.exponents[k].x);
        e_min = min(e_min, sm.exponents[k].y);
      }
      bool general = e_max - e_min > 15;
      const int common = min(13 + 127 - e_max, 126);
      const float f = p.scale_log2 * __uint_as_float((uint32_t)(127 - common) << 23);
      if (tid == 0) sm.far = 2 * (kFarFactors - (int)(__float_as_uint(fabsf(f)) >> 23));
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if (i == 1 && !two) continue;
        const int r = (tid >> 2) + 64 * i, part = tid & 3;
        const int shift = general && e[i] >= 0 && e[i] < 255 ? min(13 + 127 - e[i], 126) : common;
        const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
        unsigned char* dst = sm.q + (part >> 1) * kHalfBytes + r * 128;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const uint4 v = raw[i][k];
          *reinterpret_cast<uint4*>(dst + ((((part & 1) * 4 + k) ^ (r & 7)) << 4)) =
              make_uint4(half_pair(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                         half_pair(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                         half_pair(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                         half_pair(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
        }
        if (part == 0)
          sm.f[r] =
              e[i] == 255 ? NAN : p.scale_log2 * __uint_as_float((uint32_t)(127 - shift) << 23);
      }
      fence_proxy_async();
      mbar_arrive(&sm.q_full);
      named_sync(1, 256);

      F2 l[8], c[8];  // the rows' sums over the lane's tokens, and kHeadroom - m
#pragma unroll
      for (int b = 0; b < 8; b++) l[b] = c[b] = 0;
      const int first = two ? 0 : st, stride = two ? 1 : 2;
      const uint32_t o_col = at + kColO + kStreamRows * st;
      // The maxima may be far off: before the first step, and behind one that rows saw nothing of.
      bool unknown = true;
      for (int j = first; j < pc.tiles; j += stride) {
        const int buf = (two ? j : j >> 1) & 1;
        wait(sm, &sm.s_full[st][buf], s_phase >> buf & 1);
        s_phase ^= 1u << buf;
        tc::fence_after();
        const int ring = (step0 + j) % kPageRing;
        const float4* pages = &sm.page[ring][2 * (warp & 3)];
        const int flags = sm.flags[ring];
        const uint32_t s_col = at + kColS + kStreamRows * st + 2 * kStreamRows * buf;
        // some of the tokens are hidden from some row, or scores may be far from 0
        const bool masked = flags >= sm.far || (pc.tile + j + 1) * kTokens > pc.start;
        auto load32 = [&](int h, int b, uint32_t (&s)[16]) {  // rows [8 b, 8 b + 32)
          load_16x32(s_col + ((uint32_t)(16 * h) << 16) + 8 * b, s);
        };
        // scores that a row does not see become -inf
        auto hide = [&](int h, int b0, const float4& pg, uint32_t (&s)[16]) {
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const int token = (pc.tile + j) * kTokens + tok + 16 * h + 8 * i;
            const int node = token - pc.start;
            uint32_t bits = node < 0 ? ~0u
                                     : sm.seen[node & (kKv8TreeNodes - 1)][(base_row + 8 * b0) >> 5];
            if (token >= pc.n_all || !(pg.y > 0.0f)) bits = 0;
            bits >>= col;
#pragma unroll
            for (int b = 0; b < 4; b++)
#pragma unroll
              for (int k = 0; k < 2; k++)
                if (!(bits & (1u << (8 * b + k)))) s[4 * b + 2 * i + k] = 0xFF800000u;
          }
        };
        auto factors = [&](const float4& pg, int b) {  // of rows 8 b + col, + 1, in the second form
          const float2 v = *reinterpret_cast<const float2*>(&sm.f[base_row + 8 * b + col]);
          return pack(fmaxf(v.x * pg.z, kTiny), fmaxf(v.y * pg.z, kTiny));
        };
        // The rows' maxima up to this step, over the stream's tokens, and what is kept under them.
        auto adjust = [&]() {
          const bool any_o = j > first;  // O holds something
          if (any_o) {
            wait(sm, &sm.pv_done[st][buf ^ 1], (p_phase >> (buf ^ 1) & 1) ^ 1);
            tc::fence_after();
          }
#pragma unroll 1
          for (int side = general ? 1 : 0; side >= 0; side--) {  // 1: of x, 0: of y
            float2 top[8];
#pragma unroll
            for (int b = 0; b < 8; b++) top[b] = make_float2(-INFINITY, -INFINITY);
#pragma unroll 1
            for (int h = 0; h < 2; h++) {
              const float4 pg = pages[h];
              const float add = side ? 0.0f : pg.w;
              const F2 w2 = pack(add, add);
#pragma unroll
              for (int b0 = 0; b0 < 8; b0 += 4) {
                if (b0 > 0 && !wide) continue;
                uint32_t s[16];
                load32(h, b0, s);
                tc::wait_ld();
                if (masked) hide(h, b0, pg, s);
#pragma unroll
                for (int b = b0; b < b0 + 4; b++) {
                  const F2 g2 = factors(pg, b);
                  const float2 v0 = unpack(fma2(pack(s + 4 * (b - b0)), g2, w2));
                  const float2 v1 = unpack(fma2(pack(s + 4 * (b - b0) + 2), g2, w2));
                  top[b] = make_float2(max3(top[b].x, v0.x, v1.x), max3(top[b].y, v0.y, v1.y));
                }
              }
            }
#pragma unroll
            for (int b = 0; b < 8; b++) {
              if (b >= 4 && !wide) continue;
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) {
                top[b].x = fmaxf(top[b].x, __shfl_xor_sync(0xffffffffu, top[b].x, d));
                top[b].y = fmaxf(top[b].y, __shfl_xor_sync(0xffffffffu, top[b].y, d));
              }
              if (lane < 4)
                *reinterpret_cast<float2*>(&sm.red[st][warp & 3][8 * b + col]) = top[b];
            }
            named_sync(2 + st, 128);
            if (t < (wide ? 64 : 32)) {
              float* const kept = side ? sm.mx[st] : sm.m[st];
              const float was = kept[t];
              const float now = fmaxf(max3(was, sm.red[st][0][t], sm.red[st][1][t]),
                                      fmaxf(sm.red[st][2][t], sm.red[st][3][t]));
              kept[t] = now;
              sm.by[st][t] = ex2(was - now);
              // (scores of a wait that ran out may be any: they must not pass the lag for ever)
              if (!side) sm.c[st][t] = sm.dead ? -INFINITY : kHeadroom - now;
            }
            named_sync(2 + st, 128);
#pragma unroll
            for (int b = 0; b < 8; b++) {
              if (b >= 4 && !wide) continue;
              if (side || !general)  // the sums
                l[b] = mul2(l[b], *reinterpret_cast<const F2*>(&sm.by[st][8 * b + col]));
              if (!side) c[b] = *reinterpret_cast<const F2*>(&sm.c[st][8 * b + col]);
            }
            if (!side && any_o) {  // the results
#pragma unroll 1
              for (int k0 = 0; k0 < rows; k0 += 16) {
                uint32_t o[16];
                tc::load16(o_col + k0, o);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k++)
                  o[k] = __float_as_uint(__uint_as_float(o[k]) * sm.by[st][k0 + k]);
                tc::store16(o_col + k0, o);
              }
              tc::wait_st();
            }
            if (side) named_sync(2 + st, 128);  // `by` is read
          }
        };
        // P of a half's rows [8 b, 8 b + 16): eight tokens and eight rows a matrix. The products two
        // of the stream's steps before have read theirs.
        const uint32_t p_buf = p_row + buf * (2 * kPBytes);
        auto put = [&](int h, int b, const uint32_t* w) {
          store_matrices(p_buf + h * (16 * 128) + (p_chunk ^ (b << 4)), w[0], w[1], w[2], w[3]);
        };
        if (!general && (flags & kFarScale)) {
          general = true;
          if (t < kStreamRows) sm.mx[st][t] = fmaxf(sm.m[st][t] - kHeadroom, kLow);
          unknown = true;
        }
        const bool slow = general || masked;
        if (j >= first + 2 * stride) wait(sm, &sm.pv_done[st][buf], (p_phase >> buf & 1) ^ 1);
        bool again = unknown || slow;
        unknown = slow;  // (hidden tokens: rows may still have no maximum)
        for (;;) {
          if (again) adjust();
          if (slow) {
            // ---- hidden tokens, far scores, or the second form: every row under its own factor. A
            // score is rounded as it is for the maxima before c is added: none is above its maximum,
            // and P is 2^8 at most however c is rounded.
#pragma unroll 1
            for (int h = 0; h < 2; h++) {
              const float4 pg = pages[h];
              const F2 w2 = pack(pg.w, pg.w), inv2 = pack(pg.y, pg.y);
              uint32_t s[16];
#pragma unroll
              for (int b = 0; b < 8; b += 2) {
                if (b >= 4 && !wide) continue;
                if (b % 4 == 0) {
                  load32(h, b, s);
                  tc::wait_ld();
                  if (masked) hide(h, b, pg, s);
                }
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 2; k++) {
                  const F2 g2 = factors(pg, b + k);
                  const uint32_t* v = &s[4 * (b % 4 + k)];
                  const F2 x0 = mul2(pack(v), g2), x1 = mul2(pack(v + 2), g2);
                  const float2 y0 = ex2(unpack(add2(fma2(pack(v), g2, w2), c[b + k])));
                  const float2 y1 = ex2(unpack(add2(fma2(pack(v + 2), g2, w2), c[b + k])));
                  w[2 * k] = half_pair(y0.x, y0.y);
                  w[2 * k + 1] = half_pair(y1.x, y1.y);
                  if (general) {
                    const float2 mx =
                        *reinterpret_cast<const float2*>(&sm.mx[st][8 * (b + k) + col]);
                    const F2 to = pack(-mx.x, -mx.y);
                    l[b + k] = add2(l[b + k], add2(pack(ex2(unpack(add2(x0, to)))),
                                                   pack(ex2(unpack(add2(x1, to))))));
                  } else {
                    l[b + k] = fma2(pack(y1), inv2, fma2(pack(y0), inv2, l[b + k]));
                  }
                }
                put(h, b, w);
              }
            }
            break;
          }
          // ---- P and the sums under the maxima as they are; taken back where a score has gone over
          // the lag (rare)
          F2 d[8];  // the step's sums
          float top = -INFINITY;
          uint32_t s[2][16];  // 32 rows of a half; the next ones are on their way meanwhile
          load32(0, 0, s[0]);
#pragma unroll
          for (int u = 0; u < 4; u++) {
            const int h = u & 1, b0 = 4 * (u >> 1);
            if (b0 > 0 && !wide) continue;
            tc::wait_ld();
            if (u == 0) load32(1, 0, s[1]);
            if (u == 1 && wide) load32(0, 4, s[0]);
            if (u == 2) load32(1, 4, s[1]);
            const float4 pg = pages[h];
            const float g = fmaxf(f * pg.z, kTiny);
            const F2 g2 = pack(g, g), w2 = pack(pg.w, pg.w), inv2 = pack(pg.y, pg.y);
            uint32_t w[4];
#pragma unroll
            for (int b = b0; b < b0 + 4; b++) {
              const uint32_t* v = &s[h][4 * (b - b0)];
              const F2 add = add2(c[b], w2);
              float2 y0 = unpack(fma2(pack(v), g2, add)), y1 = unpack(fma2(pack(v + 2), g2, add));
              top = max3(top, y0.x, y0.y);
              top = max3(top, y1.x, y1.y);
              y0 = ex2(y0);
              y1 = ex2(y1);
              w[2 * (b & 1)] = half_pair(y0.x, y0.y);
              w[2 * (b & 1) + 1] = half_pair(y1.x, y1.y);
              if (b & 1) put(h, b - 1, w);
              const F2 e = h == 0 ? mul2(pack(y0), inv2) : fma2(pack(y0), inv2, d[b]);
              d[b] = fma2(pack(y1), inv2, e);
            }
          }
          again = any_of(2 + st, 128, top > kHeadroom + kLag);
          if (!again) {
#pragma unroll
            for (int b = 0; b < 8; b++)
              if (b < 4 || wide) l[b] = add2(l[b], d[b]);
            break;
          }
        }
        tc::fence_before();
        mbar_arrive(&sm.s_empty[st][buf]);
        fence_proxy_async();
        mbar_arrive(&sm.p_full[st][buf]);
        p_phase ^= 1u << buf;
      }
      step0 += pc.tiles;
      const bool any = pc.tiles > first;  // this stream had steps
      if (any) {
        const int buf = (two ? pc.tiles - 1 : (pc.tiles - 1 - first) >> 1) & 1;  // the last step's
        wait(sm, &sm.pv_done[st][buf], (p_phase >> buf & 1) ^ 1);
      }

      // ---- the sums over the stream's tokens
#pragma unroll
      for (int b = 0; b < 8; b++) {
        if (b >= 4 && !wide) continue;
        float2 v = unpack(l[b]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
          v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
        }
        if (lane < 4) *reinterpret_cast<float2*>(&sm.red[st][warp & 3][8 * b + col]) = v;
      }
      if (t < kStreamRows) {
        // The second form's frames brought together, within 2^50 of the sum's own: O (the result
        // times the sum, in that frame) and l stay in fp32's range, and of two parts that are
        // joined the frames differ by 2^100 at most beside their sums: a factor that fp32 flushes
        // to 0 belongs to a part that counts for less than 2^-26. by: of O, in two factors; mx: of
        // l.
        float by = 1.0f, of_l = 1.0f;
        if (general) {
          const float ref = sm.m[st][t] - kHeadroom, top = sm.mx[st][t];
          const float to_m = fminf(fmaxf(ref, top - 50.0f), top + 50.0f) + kHeadroom;
          const float to = to_m - kHeadroom;  // as it is read again
          if (top > kLow) {
            sm.m[st][t] = to_m;
            by = ex2(0.5f * (ref - to));
            of_l = ex2(top - to);
          }
        }
        sm.by[st][t] = by;
        sm.mx[st][t] = of_l;
      }
      tc::fence_before();
      named_sync(1, 256);
      tc::fence_after();

      // ---- the rows' weights: thread t < 64 of each stream for the rows that it writes
      struct Weights {
        float4 of[kStreamRows];  // (O0 x y + O1 z w + part before `front`) inv
        float front[kStreamRows], inv[kStreamRows];
        long long out[kStreamRows];  // the output row
      };
      Weights& weights = *reinterpret_cast<Weights*>(sm.p[0][st]);
      const bool whole = pc.flags & kWhole, after = pc.flags & kAfter;
      const bool both = !two && pc.tiles > 1;
      float2* const pml = reinterpret_cast<float2*>(p.part_ml) + (size_t)pc.slot * kRows;
      float* const po = p.part_o + ((size_t)pc.slot * kRows + base_row) * kHeadDim + t;
      float m = kLow, sum = 0.0f;
      if (t < rows) {
        const int s0 = two ? st : 0, r = base_row + t;
        auto total = [&](int s) {
          return ((sm.red[s][0][t] + sm.red[s][1][t]) + (sm.red[s][2][t] + sm.red[s][3][t])) *
                 sm.mx[s][t];
        };
        m = sm.m[s0][t];
        sum = total(s0);
        float4 w = make_float4(sm.by[s0][t], sm.by[s0][t], 0.0f, 0.0f);
        if (both) {
          const float m0 = m, m1 = sm.m[1][t];
          m = fmaxf(m0, m1);
          w.y *= ex2(m0 - m);
          w.z = sm.by[1][t];
          w.w = w.z * ex2(m1 - m);
          sum = sum * ex2(m0 - m) + total(1) * ex2(m1 - m);
        }
        if (sm.f[r] != sm.f[r]) sum = NAN;
        if (after) {
          const float2 was = __ldcg(pml + r);
          const float top = fmaxf(m, was.x), keep = ex2(m - top), front = ex2(was.x - top);
          weights.front[t] = front;
          w.y *= keep;
          w.w *= keep;
          sum = sum * keep + was.y * front;
          m = top;
        }
        weights.of[t] = w;
        if (whole) {
          const long long out =
              (long long)(q_row + r / p.group) * p.hq + pc.h * p.group + r % p.group;
          weights.out[t] = out * kHeadDim;
          weights.inv[t] = sum != 0.0f ? 1.0f / sum : 0.0f;
          if (p.lse != nullptr && (two || st == 0))
            p.lse[out] = (m - kHeadroom + log2f(sum)) * 0.693147180559945309f;
        }
      }
      if (after) named_sync(1, 256);  // both streams have read what is written now
      if (!whole && t < rows && (two || st == 0)) pml[base_row + t] = make_float2(m, sum);
      named_sync(2 + st, 128);
      // ---- one channel a thread; of one block of rows the streams write 16 in turn
      const uint32_t o0 = at + kColO + (two ? kStreamRows * st : 0);
#pragma unroll 1
      for (int r0 = two ? 0 : 16 * st; r0 < rows; r0 += two || (r0 & 8) == 0 ? 8 : 24) {
        uint32_t x[8], y[8];
        float v[8];
        load8(o0 + r0, x);
        if (both) load8(at + kColO + kStreamRows + r0, y);
        tc::wait_ld();
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const float4 w = weights.of[r0 + k];
          v[k] = __uint_as_float(x[k]) * w.x * w.y;
          if (both) v[k] += __uint_as_float(y[k]) * w.z * w.w;
        }
        if (after) {
          float was[8];
#pragma unroll
          for (int k = 0; k < 8; k++)
            was[k] = r0 + k < rows ? __ldcg(po + (r0 + k) * kHeadDim) : 0.0f;
#pragma unroll
          for (int k = 0; k < 8; k++) v[k] += was[k] * weights.front[r0 + k];
        }
        if (whole) {
#pragma unroll
          for (int k = 0; k < 8; k++)
            if (r0 + k < rows)
              p.out[weights.out[r0 + k] + t] = __float2bfloat16(v[k] * weights.inv[r0 + k]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; k++)
            if (r0 + k < rows) po[(r0 + k) * kHeadDim] = v[k];
        }
      }
      // the block's parts are joined by the kernel behind this one
      if ((pc.flags & kRecord) && tid == 0) {
        Record rec;
        rec.rows = pc.rows;
        rec.parts = pc.parts;
        rec.slot0 = pc.slot;
        rec.cta = blockIdx.x;
        rec.row0 = q_row;
        rec.head0 = pc.h * p.group;
        rec.pad[0] = rec.pad[1] = 0;
        p.records[blockIdx.x] = rec;
      }
      tc::fence_before();
      give_back();
    }
  } else if (warp < kVWarp) {
    tc::fewer_registers<kConvertRegs>();
    // ============================================ K's codes: one token a thread, into TMEM
    const int t = tid & 127;
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21) + kColK;
    const uint32_t raw0 = smem_addr(sm.k_raw[0]) + t * 128, turn = (t & 7) << 4;
    int step = 0;
    while (take(pc)) {
#pragma unroll 1
      for (int j = 0; j < pc.tiles; j++, step++) {
        const int stage = step % kStages;
        wait(sm, &sm.k_raw_full[stage], step / kStages & 1);
#pragma unroll 1
        for (int h = 0; h < 2; h++) {  // 64 channels
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const uint4 v = lds128(raw0 + stage * kRawBytes + (((4 * h + c) << 4) ^ turn));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const uint32_t x = Codes<F>::prepare(u[k]);
              w[8 * c + 2 * k] = Codes<F>::template pair<0>(x);
              w[8 * c + 2 * k + 1] = Codes<F>::template pair<1>(x);
            }
          }
          if (h == 0) {
            wait(sm, &sm.k_empty, (step & 1) ^ 1);
            tc::fence_after();
          }
          tc::store32(at + 32 * h, w);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.k_raw_empty[stage]);
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&sm.k_full);
      }
      give_back();
    }
  } else if (warp < kMmaWarp) {
    tc::fewer_registers<kConvertRegs>();
    // ============================================ V's codes: turned, 32 channels a warp, into TMEM
    const int w = warp - kVWarp;
    const uint32_t at = tmem + ((uint32_t)w << 21) + kColV;
    // lane l points at token l of 32: the 16 channels of half 0, and those of half 1 beside them
    const uint32_t raw0 = smem_addr(sm.v_raw[0]) + lane * 128, turn = (lane & 7) << 4;
    int step = 0;
    while (take(pc)) {
#pragma unroll 1
      for (int j = 0; j < pc.tiles; j++, step++) {
        const int stage = step % kStages;
        wait(sm, &sm.v_raw_full[stage], step / kStages & 1);
        const int valid = sm.v_valid[stage][lane & 7];
        const bool partial = __any_sync(0xffffffffu, valid < kPage);
#pragma unroll 1
        for (int h = 0; h < 2; h++) {  // 16 channels
          uint32_t u[16], r[32];  // of each 16 tokens 2 words
#pragma unroll
          for (int i = 0; i < 4; i++)
            load_turned(raw0 + stage * kRawBytes + i * (32 * 128) + (((2 * w + h) << 4) ^ turn),
                        &u[4 * i]);
          if (partial) {
            // bytes no token wrote may be NaN, and a weight of 0 does not hide one
#pragma unroll
            for (int b = 0; b < kTilePages; b++) {
              const int left = __shfl_sync(0xffffffffu, valid, b) - 4 * (lane & 3);
              const uint32_t mask = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << 8 * left) - 1;
              u[2 * b] &= mask;
              u[2 * b + 1] &= mask;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; i++) {
            const uint32_t x = Codes<F>::prepare(u[i]);
            r[2 * i] = Codes<F>::template pair<0>(x);
            r[2 * i + 1] = Codes<F>::template pair<1>(x);
          }
          if (h == 0) {
            wait(sm, &sm.v_empty, (step & 1) ^ 1);
            tc::fence_after();
          }
          store_16x64(at + ((uint32_t)(16 * h) << 16), r);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_raw_empty[stage]);
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&sm.v_full);
      }
      give_back();
    }
  } else {
    tc::fewer_registers<kOtherRegs>();
  }
  if (warp == kMmaWarp) {
    // ============================================ the products
    const uint32_t q_low = tc::desc_low(smem_addr(sm.q), 16);
    const uint32_t p_low = tc::desc_low(smem_addr(sm.p[0][0]), kPBytes);
    const bool lead = tc::elect();
    int step = 0;
    uint32_t p_phase = 0;    // of the next wait for its P
    uint32_t s_phase = 0xF;  // bit 2 i + b: of the next wait for buffer b of stream i's S
    // 128 products of 16 values of k each: K's tile or V's, in TMEM, with the queries or P
    auto scores = [&](auto instr, uint32_t d) {  // from the queries of stream 0, or of both
      if (lead) {
#pragma unroll
        for (int c = 0; c < 8; c++)
          tc::mma_ts<decltype(instr)::value>(
              d, tmem + kColK + c * 8, q_low + (((c >> 2) * kHalfBytes + (c & 3) * 32) >> 4), c > 0);
      }
    };
    auto values = [&](auto instr, uint32_t d, uint32_t pp, bool add) {
      if (lead) {
#pragma unroll
        for (int c = 0; c < 8; c++)
          tc::mma_ts<decltype(instr)::value>(d, tmem + kColV + c * 8, pp + c * (2048 >> 4),
                                             add || c > 0);
      }
    };
    while (take(pc)) {
      const bool two = pc.rows > kStreamRows;
      // The products with V come one step (two streams on it) or two steps (in turn) behind the
      // scores, so that a stream's next scores are there when its softmax is done. Two streams'
      // products are one: 128 columns, K and V read once.
      const int behind = two ? 1 : 2;
      wait(sm, &sm.q_full, pieces & 1);
#pragma unroll 1
      for (int j = 0; j < pc.tiles + behind; j++) {
        if (j < pc.tiles) {
          const int buf = (two ? j : j >> 1) & 1;
          wait(sm, &sm.k_full, (step + j) & 1);
#pragma unroll
          for (int i = 0; i < 2; i++)
            if (two || (j & 1) == i) {
              wait(sm, &sm.s_empty[i][buf], s_phase >> (2 * i + buf) & 1);
              s_phase ^= 1u << (2 * i + buf);
            }
          tc::fence_after();
          const uint32_t d = tmem + kColS + 2 * kStreamRows * buf;
          if (two)
            scores(std::integral_constant<uint32_t, tc::instr_f16(128, 2 * kStreamRows, false)>{},
                   d);
          else
            scores(std::integral_constant<uint32_t, tc::instr_f16(128, kStreamRows, false)>{},
                   d + kStreamRows * (j & 1));
          if (lead) {
            tc::commit(&sm.k_empty);
            if (two || !(j & 1)) tc::commit(&sm.s_full[0][buf]);
            if (two || (j & 1)) tc::commit(&sm.s_full[1][buf]);
          }
          __syncwarp();
        }
        const int jj = j - behind;
        if (jj >= 0) {
          const int st = two ? 0 : jj & 1, buf = (two ? jj : jj >> 1) & 1;
          wait(sm, &sm.v_full, (step + jj) & 1);
#pragma unroll
          for (int i = 0; i < 2; i++)
            if (two || st == i) {
              wait(sm, &sm.p_full[i][buf], p_phase >> (2 * i + buf) & 1);
              p_phase ^= 1u << (2 * i + buf);
            }
          tc::fence_after();
          const uint32_t pp = p_low + (2 * buf + st) * (kPBytes >> 4);
          if (two)
            values(std::integral_constant<uint32_t, tc::instr_f16(128, 2 * kStreamRows, true)>{},
                   tmem + kColO, pp, jj > 0);
          else
            values(std::integral_constant<uint32_t, tc::instr_f16(128, kStreamRows, true)>{},
                   tmem + kColO + kStreamRows * st, pp, jj > 1);
          if (lead) {
            tc::commit(&sm.v_empty);
            tc::commit(&sm.pv_done[st][buf]);
            if (two) tc::commit(&sm.pv_done[1][buf]);
          }
          __syncwarp();
        }
      }
      step += pc.tiles;
      give_back();
    }
    // the last arrivals on the barriers come before the CTA ends, and no product goes on in shared
    // and tensor memory that are given up
    if (lead) tc::commit(&sm.all_done);
    mbar_wait(&sm.all_done, 0);
  } else if (warp == kKLoad || warp == kVLoad) {
    // ============================================ the copies: 4 tiles' blocks a batch, one a lane
    const bool is_k = warp == kKLoad;
    uint64_t* const full = is_k ? sm.k_raw_full : sm.v_raw_full;
    uint64_t* const empty = is_k ? sm.k_raw_empty : sm.v_raw_empty;
    unsigned char* const raw = is_k ? sm.k_raw[0] : sm.v_raw[0];
    const CUtensorMap* const map = is_k ? &k_map : &v_map;
    const uint64_t policy = l2_evict_first_policy();
    struct Ahead {
      int count;  // tiles of the batch (0: the end)
      int y;      // this lane's block: its first row in the code array
      int valid;  // its tokens
      bool again; // other row blocks read it too
      float sk, sv;
    };
    bool more = take(pc);
    int done = 0;  // tiles of the piece that were fetched
    auto fetch = [&]() {
      Ahead a = {0, 0, 0, false, 0.0f, -1.0f};
      if (!more) return a;
      a.count = min(pc.tiles - done, 4);
      const int i = (pc.tile + done) * kTilePages + lane;
      a.again = pc.flags & kShared;
      if (lane < a.count * kTilePages) {
        a.valid = min(max(pc.n_all - i * kPage, 0), kPage);
        if (a.valid > 0) {
          const int page = p.page_table[(size_t)pc.b * p.rows.max_pages + i];
          if (page >= 0 && page < p.num_pages) {
            const int block = page * p.hkv + pc.h;
            a.y = block * kPage;
            if (is_k) {
              a.sk = p.k_scale[block];
              a.sv = p.v_scale[block];
            }
          } else {
            set_error(p.err, kDevErrCheck);
            a.valid = 0;
          }
        }
      }
      done += a.count;
      if (done == pc.tiles) {
        done = 0;
        give_back();
        more = take(pc);
      }
      return a;
    };
    Ahead cur = fetch(), next = {0, 0, 0, false, 0.0f, -1.0f};
    int step = 0;
    bool ok = true;
    while (ok && cur.count > 0) {
#pragma unroll 1
      for (int j = 0; j < cur.count; j++, step++) {
        const int stage = step % kStages;
        ok = __all_sync(0xffffffffu, wait(sm, &empty[stage], (step / kStages & 1) ^ 1));
        if (!ok) break;
        const bool mine = lane >> 3 == j;
        const int blocks = __popc(__ballot_sync(0xffffffffu, mine && cur.valid > 0));
        if (mine && cur.valid > 0) {  // (before the scales are there; the bytes are told below)
          unsigned char* dst = raw + stage * kRawBytes + (lane & 7) * kBlockBytesI8;
          if (cur.again) tma_load_2d(dst, map, 0, cur.y, &full[stage]);
          else tma_load_2d_hint(dst, map, 0, cur.y, &full[stage], policy);
        }
        if (is_k) {
          const float log = log2f(cur.sv);
          const bool far = mine && cur.valid > 0 && !(fabsf(log) <= kPlainScale);
          const int largest = __reduce_max_sync(
              0xffffffffu, mine ? __float_as_uint(fabsf(cur.sk)) >> 23 : 0u);
          const int flags = (blocks < kTilePages ? kHidden : 0) | 2 * largest |
                            (__any_sync(0xffffffffu, far) ? kFarScale : 0);
          if (mine)
            sm.page[step % kPageRing][lane & 7] =
                cur.valid == 0 ? make_float4(0.0f, 0.0f, 0.0f, -INFINITY)
                               : make_float4(0.0f, cur.sv == 0.0f ? 1.0f : 1.0f / cur.sv, cur.sk,
                                             log);
          if (lane == 0) sm.flags[step % kPageRing] = flags;
        } else if (mine) {
          sm.v_valid[stage][lane & 7] = cur.valid;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], blocks * kBlockBytesI8);
        if (j == 0) next = fetch();  // while the first copies are on their way
      }
      cur = next;
      next.count = 0;
    }
    // Copies under way write this CTA's shared memory: one more wait for each. Not only where a wait
    // of this warp ran out: where another warp's did, the pieces end early, and nobody may have
    // waited for the last copies. (Else they have long arrived, as their codes were read.)
    for (int i = max(step - kStages, 0); i < step; i++)
      mbar_wait(&full[i % kStages], i / kStages & 1);
  } else if (warp == kPlanWarp) {
    // ============================================ the plan: this CTA's slice of the line of steps
    // All steps of all row blocks, under all heads, of all sequences, in equal slices. A row block has
    // kBlockPlaces for what it costs beside its tiles, then each tile's; a tile is the CTA's that has
    // its first place. The pieces are told in order.
    auto over = [](long long a, long long by) {  // a / by (a division of 64 bits takes a microsecond)
      return ((a | by) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)by) : a / by;
    };
    auto each = [&](int b) {  // places of a tile
      return block_nodes[b] * p.group > kStreamRows ? kTwoPlaces : kTilePlaces;
    };
    auto places = [&](int b) {  // of one row block
      return token_tiles(len[b]) * each(b) + kBlockPlaces;
    };
    auto sequence = [&](int b) {  // of all its row blocks under all heads
      return b < batch ? (long long)blocks[b] * p.hkv * places(b) : 0;
    };
    // inclusive sums over 32 sequences
    auto scan = [&](int b0) {
      long long incl = sequence(b0 + lane);
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      return incl;
    };
    long long incl = scan(0), all = __shfl_sync(0xffffffffu, incl, 31);
    for (int b0 = 32; b0 < batch; b0 += 32) all += __shfl_sync(0xffffffffu, scan(b0), 31);
    const long long per = max(over(all + gridDim.x - 1, gridDim.x), (long long)kMinPlaces);
    const long long begin = min(blockIdx.x * per, all), end = min(begin + per, all);
    int b = 0, h = 0, q = 0, off = 0;
    if (begin < end) {  // the sequence that holds place `begin`, and where in it that is
      long long before = 0;  // places in front of the 32 sequences looked at
      while (!__any_sync(0xffffffffu, before + incl > begin)) {
        before += __shfl_sync(0xffffffffu, incl, 31);
        b += 32;
        incl = scan(b);
      }
      const int i = __ffs(__ballot_sync(0xffffffffu, before + incl > begin)) - 1;
      b += i;
      before += __shfl_sync(0xffffffffu, incl, i) - sequence(b);
      const int one = places(b);
      const long long at = begin - before, head = (long long)blocks[b] * one;
      h = (int)over(at, head);
      const unsigned rest = (unsigned)(at - h * head);
      q = rest / one;
      off = rest % one;
    }
    int one = places(b);
    long long x = begin;
    int told = 0;
    auto tell = [&](const Piece& piece) {
      const int slot = told % kPieces;
      if (!__all_sync(0xffffffffu,
                      wait(sm, &sm.piece_empty[slot], (told / kPieces & 1) ^ 1)))
        return false;
      if (lane == 0) {
        sm.piece[slot] = piece;
        mbar_arrive(&sm.piece_full[slot]);
      }
      __syncwarp();
      told++;
      return true;
    };
    bool ok = true;
    if (lane == 0) p.records[blockIdx.x].rows = 0;
    while (ok && x < end) {
      const long long block_begin = x - off, tiles_begin = block_begin + kBlockPlaces;
      const int tile_places = each(b), all_tiles = token_tiles(len[b]);
      auto tile_at = [&](int place) {  // the first tile from this place of the row block on
        return (max(place - kBlockPlaces, 0) + tile_places - 1) / tile_places;
      };
      const long long last_begin = tiles_begin + (long long)(all_tiles - 1) * tile_places;
      int stop = (int)min((long long)one, off + (end - x));
      Piece piece = {};
      piece.tile = tile_at(off);
      piece.tiles = min(tile_at(stop), all_tiles) - piece.tile;
      const int most = block_nodes[b], nodes = min(most, num[b] - q * most);
      piece.rows = nodes * p.group;
      const int limit = piece.rows > kStreamRows ? kMaxSteps : 2 * kMaxSteps;
      const bool cut = piece.tiles > limit;  // the rest of the stretch is the next piece
      if (cut) {
        piece.tiles = limit;
        stop = (piece.tile + limit) * tile_places + kBlockPlaces;
      }
      if (piece.tiles > 0) {
        piece.b = b;
        piece.h = h;
        piece.n_all = len[b];
        piece.start = len[b] - num[b];
        piece.node = q * most;
        piece.row0 = row0[b];
        const bool after =
            piece.tile > 0 && tiles_begin + (piece.tile - 1) * tile_places >= begin;
        const bool whole = !cut && begin <= tiles_begin && last_begin < end;
        const int c0 = (int)over(tiles_begin, per);
        piece.flags = (whole ? kWhole : 0) | (after ? kAfter : 0) |
                      (!whole && !cut && tiles_begin >= begin ? kRecord : 0) |
                      (num[b] > nodes ? kShared : 0);
        piece.slot = 2 * blockIdx.x + (begin < block_begin ? 1 : 0);
        piece.parts = (int)over(last_begin, per) - c0 + 1;
        ok = tell(piece);
      }
      x += stop - off;
      off = stop;
      if (!cut) {
        off = 0;
        if (++q == blocks[b]) {
          q = 0;
          if (++h == p.hkv) {
            h = 0;
            do b++;
            while (b < batch && num[b] == 0);
            if (b < batch) one = places(b);
          }
        }
      }
    }
    if (ok) tell(Piece{});
    // rows of sequences that do not fit: 0 and -inf
    for (int s = blockIdx.x; s < batch; s += gridDim.x) {
      const int rows = p.rows.cu ? p.rows.cu[s + 1] - p.rows.cu[s] : 1;
      if (rows == num[s]) continue;
      const int first = max(row0[s], 0);
      const int count = min(p.rows.cu ? p.rows.cu[s + 1] : s + 1, p.rows.total) - first;
      for (long long i = lane; i < (long long)count * p.hq * (kHeadDim / 8); i += 32)
        reinterpret_cast<uint4*>(p.out + (size_t)first * p.hq * kHeadDim)[i] =
            make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr)
        for (long long i = lane; i < (long long)count * p.hq; i += 32)
          p.lse[(size_t)first * p.hq + i] = -INFINITY;
    }
  }
  tc::fence_before();
  __syncthreads();
  if (tid == 0 && sm.dead) set_error(p.err, kDevErrTimeout);
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------- row blocks that were cut, joined
//
// Rows of all records in one line, a warp each, or where they are few (two for each CTA at most) a
// CTA each, whose warps take the parts in turn (calls of 32 rows over 8K tokens 14.0 us, by warps
// 17.5; of 2400 rows over 4 contexts 38.2 by warps, by CTAs 58.5). A lane has four channels; values
// are asked for before their weights are known. Bound by latency.
constexpr int kJoinWarps = 8, kJoinAhead = 8;

struct JoinParams {
  const float* part_ml;
  const float* part_o;
  const Record* records;
  __nv_bfloat16* out;
  float* lse;
  int hq, group;
};

__global__ void __launch_bounds__(kJoinWarps * 32) kv8_tree_join_kernel(const JoinParams p) {
  __shared__ int upto[kKv8MaxCtas];  // rows of records 0 .. i
  __shared__ int sums[kJoinWarps];
  __shared__ float4 part_acc[kJoinWarps][32];
  __shared__ float2 part_sum[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  {
    static_assert(kJoinWarps * 32 >= kKv8MaxCtas, "a thread a record");
    int incl = threadIdx.x < gridDim.x ? p.records[threadIdx.x].rows : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; w++) incl += sums[w];
    upto[threadIdx.x] = incl;
    __syncthreads();
  }
  const int rows = upto[gridDim.x - 1];
  const bool shared = rows <= 2 * (int)gridDim.x;  // a row is the CTA's
  const int first = shared ? warp : 0, stride = shared ? kJoinWarps : 1;
  for (int u = shared ? blockIdx.x : blockIdx.x * kJoinWarps + warp; u < rows;
       u += gridDim.x * (shared ? 1 : kJoinWarps)) {
    int i = 0;  // the record that holds row u: the first with upto > u
    for (int step = kKv8MaxCtas / 2; step > 0; step >>= 1)
      if (i + step <= (int)gridDim.x && upto[i + step - 1] <= u) i += step;
    const Record rec = p.records[i];
    const int r = u - (i > 0 ? upto[i - 1] : 0);
    // part 0 in its own slot, part k in the first slot of the k-th CTA behind
    auto slot_of = [&](int k) { return (size_t)(k == 0 ? rec.slot0 : 2 * (rec.cta + k)); };
    const float4* src = reinterpret_cast<const float4*>(p.part_o) + r * (kHeadDim / 4) + lane;
    float top = kLow, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = first; k0 < rec.parts; k0 += 32 * stride) {
      const int mine = k0 + lane * stride;
      float2 ml = make_float2(kLow, 0.0f);
      if (mine < rec.parts)
        ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + slot_of(mine) * kRows + r);
      float weight = 0.0f;
      for (int j0 = 0; j0 < 32 && k0 + j0 * stride < rec.parts; j0 += kJoinAhead) {
        float4 v[kJoinAhead];
#pragma unroll
        for (int j = 0; j < kJoinAhead; j++) {
          const int k = k0 + (j0 + j) * stride;
          v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (k < rec.parts) v[j] = __ldcg(src + slot_of(k) * (kRows * kHeadDim / 4));
        }
        if (j0 == 0) {
          const float now = fmaxf(top, warp_max(ml.x)), keep = ex2(top - now);
          weight = mine < rec.parts ? ex2(ml.x - now) : 0.0f;
          float of = weight * ml.y;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) of += __shfl_xor_sync(0xffffffffu, of, d);
          sum = sum * keep + of;
          acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
          top = now;
        }
#pragma unroll
        for (int j = 0; j < kJoinAhead; j++) {
          const float w = __shfl_sync(0xffffffffu, weight, j0 + j);
          acc.x += w * v[j].x;
          acc.y += w * v[j].y;
          acc.z += w * v[j].z;
          acc.w += w * v[j].w;
        }
      }
    }
    if (shared) {
      part_acc[warp][lane] = acc;
      if (lane == 0) part_sum[warp] = make_float2(top, sum);
      __syncthreads();
      if (warp == 0) {
        const int ways = min(kJoinWarps, rec.parts);
        for (int w = 0; w < ways; w++) top = fmaxf(top, part_sum[w].x);
        sum = 0.0f;
        acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < ways; w++) {
          const float by = ex2(part_sum[w].x - top);
          const float4 v = part_acc[w][lane];
          sum += by * part_sum[w].y;
          acc.x += by * v.x;
          acc.y += by * v.y;
          acc.z += by * v.z;
          acc.w += by * v.w;
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    const size_t out = (size_t)(rec.row0 + r / p.group) * p.hq + rec.head0 + r % p.group;
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(p.out + out * kHeadDim)[lane] =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    if (lane == 0 && p.lse != nullptr)
      p.lse[out] = (top - kHeadroom + log2f(sum)) * 0.693147180559945309f;
  }
}

size_t smem_bytes(int batch) { return 1024 + sizeof(Smem) + 20 * (size_t)batch; }
static_assert(1024 + sizeof(Smem) + 20 * 1024 <= 227 * 1024, "shared memory for the largest batch");

}  // namespace

size_t kv8_tree_part_floats() { return (size_t)2 * kKv8MaxCtas * kRows * kHeadDim; }
size_t kv8_tree_ml_floats() { return (size_t)2 * kKv8MaxCtas * kRows * 2; }
size_t kv8_tree_record_bytes() { return (size_t)kKv8MaxCtas * sizeof(Record); }

cudaError_t launch_kv8_tree(const Shape& s, const Kv8& c, const CUtensorMap& k_map,
                            const CUtensorMap& v_map, const void* q, long long q_stride,
                            const int32_t* parents, const int32_t* cu, int total,
                            const int32_t* page_table, const int32_t* seq_lens, void* out,
                            float* lse, float* part_ml, float* part_o, void* records, int* err,
                            int num_sms, cudaStream_t st) {
  auto kernel = c.format == kE4m3 ? kv8_tree_kernel<kE4m3> : kv8_tree_kernel<kInt8>;
  const size_t smem = smem_bytes(s.batch);
  cudaError_t e = set_kernel_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  const int grid = std::min(num_sms, kKv8MaxCtas);
  Params p;
  p.rows = NewRows{cu, seq_lens, s.batch, total, s.max_pages};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.parents = parents;
  p.page_table = page_table;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part_ml = part_ml;
  p.part_o = part_o;
  p.records = static_cast<Record*>(records);
  p.err = err;
  p.hq = s.hq;
  p.hkv = s.hkv;
  p.group = s.group;
  p.num_pages = s.num_pages;
  p.block_nodes = kRows / s.group;
  p.scale_log2 = s.sm_scale * 1.44269504088896341f;
  e = launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, st, true, k_map, v_map, p);
  if (e != cudaSuccess) return e;
  const JoinParams jp = {part_ml, part_o, p.records, p.out, p.lse, s.hq, s.group};
  return launch_kernel(kv8_tree_join_kernel, dim3(grid), dim3(kJoinWarps * 32), 0, st, true, jp);
}

}  // namespace hsa
