// Host-side launchers of the separate expert operators (include/mok.h: pair
// sort, row permutation, 4-bit integer expert products).  Internal to libmok.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mok {

enum { kF32 = 0, kBF16 = 1, kF16 = 2 };  // mok_dtype

// Pairs per workgroup of the sort: sixteen waves, kSortIters rounds of 64.
constexpr int kSortIters = 2;
constexpr int kPairChunk = 16 * 64 * kSortIters;
// Chunk tables of up to this many chunks are summed by every placing
// workgroup itself; longer ones by a launch of their own in between.
constexpr int kSelfScanChunks = 64;

// Stable sort of P pairs by expert; `table` holds ceil(P / kPairChunk) * E
// int32 (unused when one chunk holds every pair).
hipError_t launch_sort_pairs(const int32_t* idx, int64_t P, int E, int eb, int ee, int32_t* counts, int32_t* offsets,
                             int32_t* row_of_pair, int32_t* pair_of_row, int32_t* table, hipStream_t s);

// One pass over the tokens of a pair map (row_of_pair [T, k], rows outside
// [0, nrows) are no rows).  w(t, j) = gate[t, j], or 1 without gate.
//   scatter:  rows[row] = w a[t]                  (dot == nullptr)
//             and dot[t, j] = <a[t], in[row]>     (dot and in given)
//   gather:   out[t] = sum_j w in[row]
//             and dot[t, j] = <a[t], in[row]>     (dot and a given)
struct PairRows {
  const void* a;
  const void* in;
  void* out;
  float* dot;
  const float* gate;
  const int32_t* rop;
  int64_t T;
  int k;
  int d;
  int dtype;
  int64_t nrows;
};
hipError_t launch_scatter_rows(const PairRows& p, hipStream_t s);
hipError_t launch_gather_rows(const PairRows& p, hipStream_t s);

}  // namespace mok
