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

// Width of a row of the rank products that the kernels hand on: whole tiles of
// the matrix instruction, zeros past r.
__host__ __device__ inline int lora_width(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

// part[s][row][lora_width(r)] = the s-th share of K of A_g in_row (fp32); s < splits.
struct LoraRank {
  LoraMap map;
  const void* in;  // [rows, K]
  const void* A;   // [G, r, K]
  float* part;
  int K, r, dtype, splits;
  int height, ranges;  // set by the launcher
};

// out_row = base_row + scale_g B_g (sum_s part[s][row]); the sum to u where that is given,
// u_width (r or lora_width(r)) floats a row.
struct LoraAdd {
  LoraMap map;
  const float* part;
  const void* B;       // [G, N, r]
  const float* scale;  // [G], NULL: 1
  const void* base;    // [rows, N], NULL: 0
  void* out;           // [rows, N]; may be base
  float* u;            // [rows, u_width] or NULL
  int N, r, dtype, splits, u_width;
};

// The gradients of both stacks: out[m] of group g sums scale_g v[m][row] wide[m][row] over its rows.
struct LoraGrad {
  LoraMap map;
  const void* wide[2];  // x [rows, K], dout [rows, N]
  const float* v[2];    // du [rows, lora_width(r)], u [rows, r]
  float* out[2];        // dA [G, r, K], dB [G, N, r]
  int width[2];
  const float* scale;
  int r, dtype;
  int ranges;   // lora_grad_plan
  float* part;  // NULL with one range
};

// Ranges of rows that the grad kernel's workgroups take, and the bytes that the sums
// of groups in several of them take.
struct LoraGradPlan {
  int ranges;
  int64_t part_bytes;
};
LoraGradPlan lora_grad_plan(int rows, int G, int r, int K, int N, int dtype);

// What the backward pass needs first: At [G, K, r] of A [G, r, K], Bt [G, r, N] of
// B [G, N, r], and dA and dB of groups without rows.
struct LoraPrepare {
  LoraMap map;
  const void *A, *B;
  void *At, *Bt;
  float *dA, *dB;
  int r, K, N, dtype;
};

// K's shares of the rank product that fill the device with few rows.
int lora_splits(int rows, int G, int r, int K, int dtype);

hipError_t launch_lora_rank(const LoraRank& a, hipStream_t s);
hipError_t launch_lora_add(const LoraAdd& a, hipStream_t s);
hipError_t launch_lora_grad(const LoraGrad& a, hipStream_t s);
hipError_t launch_lora_prepare(const LoraPrepare& a, hipStream_t s);

}  // namespace mok
