// Launchers of the low-rank adapters beside a projection (include/mok.h:
// mok_lora_rows and its backward pass).  Internal to libmok.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mok {

constexpr int kLoraMaxRank = 128;

// The groups' rows: group g (0..G-1) has the sorted rows [offsets[g], offsets[g + 1])
// cut to [0, rows); row q is token pair_of_row[q] of [0, rows), or row q itself
// where pair_of_row is NULL.
struct LoraMap {
  const int32_t* offsets;  // at the first local group
  const int32_t* pair_of_row;
  const int32_t* row_of_pair;
  int rows, G;
};

// part[s][row][r] = the s-th share of K of A_g in_row (fp32); s < splits.
struct LoraRank {
  LoraMap map;
  const void* in;  // [rows, K]
  const void* A;   // [G, r, K]
  float* part;     // [splits, rows, r]
  int K, r, dtype, splits;
};

// out_row = base_row + scale_g B_g (sum_s part[s][row]); the sum to u where that is given.
struct LoraAdd {
  LoraMap map;
  const float* part;
  const void* B;       // [G, N, r]
  const float* scale;  // [G], NULL: 1
  const void* base;    // [rows, N], NULL: 0
  void* out;           // [rows, N]; may be base
  float* u;            // [rows, r] or NULL
  int N, r, dtype, splits;
};

// The gradients of both stacks: out[m] of group g sums scale_g v[m][row] wide[m][row] over its rows.
struct LoraGrad {
  LoraMap map;
  const void* wide[2];  // x [rows, K], dout [rows, N]
  const float* v[2];    // du, u [rows, r]
  float* out[2];        // dA [G, r, K], dB [G, N, r]
  int width[2];
  const float* scale;
  int r, dtype;
};

// K's shares of the rank product that fill the device with few rows.
int lora_splits(int rows, int G, int K, int dtype);

hipError_t launch_lora_rank(const LoraRank& a, hipStream_t s);
hipError_t launch_lora_add(const LoraAdd& a, hipStream_t s);
hipError_t launch_lora_grad(const LoraGrad& a, hipStream_t s);
// At [G, K, r] of A [G, r, K] and Bt [G, r, N] of B [G, N, r].
hipError_t launch_lora_transpose(const void* A, const void* B, int G, int r, int K, int N, int dtype, void* At,
                                 void* Bt, hipStream_t s);

}  // namespace mok
