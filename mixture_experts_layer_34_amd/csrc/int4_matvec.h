// Host-side launchers of the 4-bit integer expert products and their weight
// quantiser (include/mok.h).  Internal to libmok.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mok {

// An expert's rows [begin, end) as the offsets give them, cut to [0, rows) at
// both ends before anything is subtracted: any two int32 leave 0 <= begin <=
// end <= rows, and no rows where the end is not past the beginning.
struct RowRange {
  int begin, end;
};
__host__ __device__ inline RowRange cut_rows(int begin, int end, int rows) {
  const int b = begin < 0 ? 0 : begin > rows ? rows : begin;
  const int e = end < b ? b : end > rows ? rows : end;
  return RowRange{b, e};
}

struct Int4Args {
  const void* x;               // [x_rows, K]
  const int32_t* pair_of_row;  // x row of row r is pair_of_row[r] / k; null: r
  const int32_t* offsets;      // rows of expert e: [offsets[e], offsets[e + 1]); null: one matrix, every row
  const uint8_t* codes[2];     // [E_loc, N, K / 2]
  const void* scales[2];       // [E_loc, N, K / group]
  const uint8_t* zeros[2];     // like the scales, or null: 8
  void* out;                   // [rows, N]
  int rows, x_rows, k;
  int E, eb, E_loc;            // experts of the offsets; the local ones [eb, eb + E_loc)
  int N, K, group;
  int pair;                    // two matrices: out = silu(first) * second
};
// x below 2 GiB and an expert's codes below 4 GiB (32-bit buffer offsets).
hipError_t launch_int4_matvec_bf16(const Int4Args& a, hipStream_t s);
hipError_t launch_int4_matvec_f16(const Int4Args& a, hipStream_t s);

// zeros == nullptr: symmetric.
hipError_t launch_quantize_int4(const void* src, int64_t rows, int64_t K, int group, int dtype, uint8_t* codes,
                                void* scales, uint8_t* zeros, hipStream_t s);

}  // namespace mok
