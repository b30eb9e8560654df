// Launcher of the whole layer for a few tokens (include/mok.h:
// mok_few_token_layer).  Internal to libmok.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mok {

constexpr int kFewTokens = 16;  // one 16-column tile of the matrix instruction
constexpr int kFewSlots = 64;   // most experts a token may choose
constexpr int kFewSigmoid = 1, kFewRenorm = 2;

// Low-rank adapters of one projection: A [L, E_loc, r, K], B [L, E_loc, N, r].
struct FewLora {
  const void* A;  // NULL: none
  const void* B;
  const float* scale;  // [L], NULL: 1
  int r;
};

struct FewTokens {
  const void* x;
  const float* logits;
  const void* w[3];  // W1, W3, W2
  void* out;
  int32_t* idx;
  float* gate;
  void* h;      // gate * silu(a) * b, in columns [0, F): fp32 [T k, Fp], or two bf16 parts [T k, 2, Fp]
  void* table;  // few_table_size bytes: the chosen experts and their pairs
  float* u[3];  // [T k, rp] scale * A v of each pair, zeros past r
  FewLora lora[3];
  const int32_t* adapter;  // [T], NULL: no adapters
  int T, d, F, Fp, E, eb, E_loc, k, L, dtype, gating;
};

// Width of an h row, of four bytes an element: whole lines of 128 bytes for fp32, whole
// 16 bytes for the two parts of the 16-bit types.
inline int few_h_width(int F, int dtype) { return dtype == 0 ? (F + 31) / 32 * 32 : (F + 3) / 4 * 4; }
// Width of a u row: whole 16-byte loads.
__host__ __device__ inline int few_u_width(int r) { return (r + 7) / 8 * 8; }

size_t few_table_size(int T, int k, int E_loc);
hipError_t launch_few_tokens(const FewTokens& a, hipStream_t s);

}  // namespace mok
