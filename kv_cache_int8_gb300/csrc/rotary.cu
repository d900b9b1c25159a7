// rotary.cu -- rotary positions: the table of cosines and sines, and rows of queries and keys
// turned by it.
//
// The pages leave positions to the model ("KV Cache 与长上下文推理" caches keys that carry theirs);
// formulas: rotary.cuh; frequencies for long contexts: position interpolation (Chen et al. 2023)
// and interpolation by parts (Peng et al. 2023, YaRN).
//
// The rotation moves each value once, 4 bytes an element and 4 dim a row for the angles: bound by
// memory, one row by latency. A warp takes one row and 16 heads, so the angles are read once for
// 2048 channels and stay in registers. 108K rows of 32 + 8 heads (2.24 GB) 319 us, 7.0 TB/s; one
// row 1.8 us. The table is made once for every position to come and is bound by sincos in 64 bits:
// 8K rows of 64 angles 33 us, 128K 480, 1M 3.8 ms.
#include <cmath>

#include "internal.h"
#include "kv8.cuh"
#include "rotary.cuh"

namespace hsa {
namespace {

using namespace rotary_detail;
using kv8_detail::NewRows;
using kv8_detail::NewSpan;
using kv8_detail::new_span;
using kv8_detail::warp_search;

constexpr int kWarps = 8;

struct Frequencies {
  double f[kHeadDim / 2];
};

// One angle a thread, in 64 bits: fp32 would lose a position of 2^20 to 2^-4 radians.
__global__ void __launch_bounds__(256) rotary_table_kernel(const Frequencies f, float* table,
                                                           int rows, int half, double magnitude) {
  grid_dep_wait();
  grid_dep_launch();
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long p = t / half;
  const int i = (int)(t % half);
  if (p >= rows) return;
  double s, c;
  sincos((double)p * f.f[i], &s, &c);
  float* row = table + p * 2 * half;
  row[i] = (float)(c * magnitude);
  row[half + i] = (float)(s * magnitude);
}

// Units: (row, 16 heads) of q, then of k; one warp behind them reports sequences that do not fit.
template <bool kNeighbours>
__global__ void __launch_bounds__(kWarps * 32) rotate_kernel(const RowSide qs, const RowSide ks,
                                                             const Rotary rot, const NewRows rows,
                                                             int units, int* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit == units && rot.positions == nullptr) kv8_detail::report_bad(rows, lane, err);
  if (unit >= units) return;
  const int nq = row_units(qs.heads), per = nq + row_units(ks.heads);
  const int row = unit / per, part = unit % per;
  int position;
  if (rot.positions != nullptr) {
    position = rot.positions[row];
  } else {
    const int b = rows.cu ? warp_search(rows.batch, row, lane, [&](int i) { return rows.cu[i]; })
                          : row;
    if (b < 0) return;
    const NewSpan sp = new_span(rows, b);
    if (row < sp.row0 || row - sp.row0 >= sp.n) return;
    position = sp.start + (row - sp.row0);
  }
  if (position < 0 || position >= rot.rows) {
    if (lane == 0) set_error(err, kDevErrCheck);
    return;
  }
  if (part < nq) turn_row<kNeighbours>(qs, rot, row, part * kRowHeads, position, lane);
  else turn_row<kNeighbours>(ks, rot, row, (part - nq) * kRowHeads, position, lane);
}

}  // namespace

cudaError_t launch_rotary_table(const RotaryAngles& a, float* table, int rows, int dim,
                                cudaStream_t st) {
  Frequencies f;
  const int half = dim / 2;
  for (int i = 0; i < half; i++) {
    double w = std::pow(a.base, -2.0 * i / dim);
    if (a.scaling == 1) {
      w /= a.factor;
    } else if (a.scaling == 2) {
      // turns within the original context: those of `low` or fewer are slowed by the factor,
      // those of `high` or more kept
      const double turns = a.original * w / (2.0 * M_PI);
      const double keep = std::min(std::max((turns - a.low) / (a.high - a.low), 0.0), 1.0);
      w *= keep + (1.0 - keep) / a.factor;
    }
    f.f[i] = w;
  }
  const long long n = (long long)rows * half;
  return launch_kernel(rotary_table_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st,
                       true, f, table, rows, half, a.magnitude);
}

cudaError_t launch_rotate(const Shape& s, const RotaryTable& t, bool with_k, const void* q,
                          long long q_stride, void* q_out, long long q_out_stride, const void* k,
                          long long k_stride, void* k_out, long long k_out_stride,
                          const int32_t* positions, const int32_t* cu, int total,
                          const int32_t* seq_lens, int* err, cudaStream_t st) {
  const RowSide qs = {static_cast<const __nv_bfloat16*>(q), q_stride,
                      static_cast<__nv_bfloat16*>(q_out), q_out_stride, s.hq};
  const RowSide ks = {static_cast<const __nv_bfloat16*>(k), k_stride,
                      static_cast<__nv_bfloat16*>(k_out), k_out_stride, with_k ? s.hkv : 0};
  const Rotary rot = {t.table, t.rows, t.dim, positions};
  const NewRows rows = {cu, seq_lens, s.batch, total, INT32_MAX / kPage};
  const int units = total * (row_units(qs.heads) + row_units(ks.heads));
  auto kernel = t.neighbours ? rotate_kernel<true> : rotate_kernel<false>;
  return launch_kernel(kernel, dim3(units / kWarps + 1), dim3(kWarps * 32), 0, st, true, qs, ks,
                       rot, rows, units, err);
}

}  // namespace hsa
