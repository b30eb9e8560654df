// C ABI of the separate expert operators (include/mok.h): argument checks on
// the host, then the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/mok.h"
#include "int4_matvec.h"
#include "pair_ops.h"

using namespace mok;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// a pointer to `n` elements: not null unless there are none, 16-byte aligned
bool good(const void* p, int64_t n) { return (p || n == 0) && aligned16(p); }

mok_status result(hipError_t e) { return e == hipSuccess ? MOK_OK : MOK_ERR_HIP; }

constexpr int64_t kMaxPairs = int64_t(1) << 31;

bool bad_pairs(int32_t T, int32_t k) { return T < 0 || k < 1 || k > 1024 || (int64_t)T * k >= kMaxPairs; }
bool bad_experts(int32_t E, int32_t eb, int32_t ee) { return E < 1 || E > 1024 || eb < 0 || ee <= eb || ee > E; }

mok_status pair_rows(const void* a, const void* in, void* out, float* dot, const float* gate, const int32_t* rop,
                     int32_t T, int32_t k, int32_t d, mok_dtype dtype, int64_t rows, PairRows* p) {
  if (bad_pairs(T, k) || d < 1 || d > (1 << 20) || rows < 0 || rows >= kMaxPairs) return MOK_ERR_INVALID_ARG;
  if (dtype != MOK_DTYPE_F32 && dtype != MOK_DTYPE_BF16 && dtype != MOK_DTYPE_F16) return MOK_ERR_INVALID_ARG;
  if (!good(rop, T) || !aligned16(gate) || !aligned16(dot)) return MOK_ERR_INVALID_ARG;
  *p = PairRows{a, in, out, dot, gate, rop, T, k, d, (int)dtype, rows};
  return MOK_OK;
}

}  // namespace

extern "C" {

mok_status mok_sort_pairs_workspace_query(int32_t T, int32_t k, int32_t E, size_t* workspace_bytes) {
  if (bad_pairs(T, k) || E < 1 || E > 1024 || !workspace_bytes) return MOK_ERR_INVALID_ARG;
  const int64_t chunks = ((int64_t)T * k + kPairChunk - 1) / kPairChunk;
  *workspace_bytes = chunks > 1 ? (size_t)chunks * E * sizeof(int32_t) : 0;
  return MOK_OK;
}

mok_status mok_sort_pairs(const int32_t* topk_idx, int32_t T, int32_t k, int32_t E, int32_t expert_begin,
                          int32_t expert_end, int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_of_pair,
                          int32_t* pair_of_row, void* workspace, void* stream) {
  if (bad_pairs(T, k) || bad_experts(E, expert_begin, expert_end)) return MOK_ERR_INVALID_ARG;
  const int64_t P = (int64_t)T * k;
  if (!good(topk_idx, P) || !good(row_of_pair, P) || !good(pair_of_row, P) || !good(expert_counts, 1) ||
      !good(expert_offsets, 1) || !good(workspace, P > kPairChunk))
    return MOK_ERR_INVALID_ARG;
  return result(launch_sort_pairs(topk_idx, P, E, expert_begin, expert_end, expert_counts, expert_offsets, row_of_pair,
                                  pair_of_row, (int32_t*)workspace, (hipStream_t)stream));
}

mok_status mok_permute_rows(const void* x, const float* gate, const int32_t* row_of_pair, int32_t T, int32_t k,
                            int32_t d, mok_dtype dtype, int64_t rows, void* xp, void* stream) {
  PairRows p;
  const mok_status st = pair_rows(x, nullptr, xp, nullptr, gate, row_of_pair, T, k, d, dtype, rows, &p);
  if (st != MOK_OK) return st;
  if (!good(x, T) || !good(xp, rows)) return MOK_ERR_INVALID_ARG;
  return result(launch_scatter_rows(p, (hipStream_t)stream));
}

mok_status mok_permute_rows_backward(const void* dxp, const void* x, const float* gate, const int32_t* row_of_pair,
                                     int32_t T, int32_t k, int32_t d, mok_dtype dtype, int64_t rows, void* dx,
                                     float* dgate, void* stream) {
  PairRows p;
  const mok_status st = pair_rows(x, dxp, dx, dgate, gate, row_of_pair, T, k, d, dtype, rows, &p);
  if (st != MOK_OK) return st;
  if (!good(dxp, rows) || !aligned16(x) || !good(dx, T)) return MOK_ERR_INVALID_ARG;
  if (T > 0 && (x != nullptr) != (dgate != nullptr)) return MOK_ERR_INVALID_ARG;
  return result(launch_gather_rows(p, (hipStream_t)stream));
}

mok_status mok_unpermute_rows(const void* y, const float* gate, const int32_t* row_of_pair, int32_t T, int32_t k,
                              int32_t d, mok_dtype dtype, int64_t rows, void* out, void* stream) {
  PairRows p;
  const mok_status st = pair_rows(nullptr, y, out, nullptr, gate, row_of_pair, T, k, d, dtype, rows, &p);
  if (st != MOK_OK) return st;
  if (!good(y, rows) || !good(out, T)) return MOK_ERR_INVALID_ARG;
  return result(launch_gather_rows(p, (hipStream_t)stream));
}

mok_status mok_unpermute_rows_backward(const void* dout, const void* y, const float* gate, const int32_t* row_of_pair,
                                       int32_t T, int32_t k, int32_t d, mok_dtype dtype, int64_t rows, void* dy,
                                       float* dgate, void* stream) {
  PairRows p;
  const mok_status st = pair_rows(dout, y, dy, dgate, gate, row_of_pair, T, k, d, dtype, rows, &p);
  if (st != MOK_OK) return st;
  if (!good(dout, T) || !aligned16(y) || !good(dy, rows)) return MOK_ERR_INVALID_ARG;
  if (T > 0 && rows > 0 && (y != nullptr) != (dgate != nullptr)) return MOK_ERR_INVALID_ARG;
  return result(launch_scatter_rows(p, (hipStream_t)stream));
}

mok_status mok_expert_matvec_int4(const void* x, const int32_t* pair_of_row, const int32_t* expert_offsets,
                                  const mok_int4_weights* w, const mok_int4_weights* w_up,
                                  const mok_int4_config* cfg, void* out, void* stream) {
  if (!cfg || !w) return MOK_ERR_INVALID_ARG;
  const mok_int4_config& c = *cfg;
  if (c.rows < 0 || c.rows > (1 << 24) || c.x_rows < 0 || c.x_rows > (1 << 24)) return MOK_ERR_INVALID_ARG;
  if (c.k < 1 || c.N < 1 || c.K < 1) return MOK_ERR_INVALID_ARG;
  if (bad_experts(c.E, c.expert_begin, c.expert_end)) return MOK_ERR_INVALID_ARG;
  if (c.group != 32 && c.group != 64 && c.group != 128) return MOK_ERR_INVALID_ARG;
  if (c.K % c.group || c.K > (1 << 20)) return MOK_ERR_INVALID_ARG;
  if (c.dtype == MOK_DTYPE_F32) return MOK_ERR_UNSUPPORTED;
  if (c.dtype != MOK_DTYPE_BF16 && c.dtype != MOK_DTYPE_F16) return MOK_ERR_INVALID_ARG;
  // x and one expert's codes are addressed in 32 bits
  if ((int64_t)c.x_rows * c.K * 2 >= (int64_t(1) << 31) || (int64_t)c.N * (c.K / 2) >= (int64_t(1) << 31))
    return MOK_ERR_INVALID_ARG;
  const int32_t E_loc = c.expert_end - c.expert_begin;
  // units of 4 rows by 16 columns, and of an expert by 16 columns, are counted in 32 bits
  if ((int64_t)c.rows * c.N >= (int64_t(1) << 36) || (int64_t)E_loc * c.N * (c.K / 2) >= (int64_t(1) << 38))
    return MOK_ERR_INVALID_ARG;
  if (!expert_offsets && (E_loc != 1 || pair_of_row)) return MOK_ERR_INVALID_ARG;
  if (!pair_of_row && c.x_rows < c.rows) return MOK_ERR_INVALID_ARG;
  if (!good(x, c.x_rows) || !good(out, c.rows) || !aligned16(pair_of_row) || !aligned16(expert_offsets))
    return MOK_ERR_INVALID_ARG;
  const mok_int4_weights* ws[2] = {w, w_up};
  for (const mok_int4_weights* m : ws)
    if (m && (!good(m->codes, 1) || !good(m->scales, 1) || !aligned16(m->zeros))) return MOK_ERR_INVALID_ARG;
  if (w_up && (w->zeros != nullptr) != (w_up->zeros != nullptr)) return MOK_ERR_INVALID_ARG;
  if (c.rows == 0) return MOK_OK;
  Int4Args a{};
  a.x = x;
  a.pair_of_row = pair_of_row;
  a.offsets = expert_offsets;
  for (int m = 0; m < (w_up ? 2 : 1); ++m) {
    a.codes[m] = ws[m]->codes;
    a.scales[m] = ws[m]->scales;
    a.zeros[m] = ws[m]->zeros;
  }
  a.out = out;
  a.rows = c.rows;
  a.x_rows = c.x_rows;
  a.k = c.k;
  a.E = c.E;
  a.eb = c.expert_begin;
  a.E_loc = E_loc;
  a.N = c.N;
  a.K = c.K;
  a.group = c.group;
  a.pair = w_up != nullptr;
  return result(c.dtype == MOK_DTYPE_BF16 ? launch_int4_matvec_bf16(a, (hipStream_t)stream)
                                          : launch_int4_matvec_f16(a, (hipStream_t)stream));
}

mok_status mok_quantize_int4(const void* src, int64_t rows, int64_t K, int32_t group, mok_dtype dtype, uint8_t* codes,
                             void* scales, uint8_t* zeros, void* stream) {
  if (rows < 0 || K < 1 || (group != 32 && group != 64 && group != 128) || K % group) return MOK_ERR_INVALID_ARG;
  if (dtype == MOK_DTYPE_F32) return MOK_ERR_UNSUPPORTED;
  if (dtype != MOK_DTYPE_BF16 && dtype != MOK_DTYPE_F16) return MOK_ERR_INVALID_ARG;
  if (rows > (int64_t(1) << 40) / K) return MOK_ERR_INVALID_ARG;
  if (!good(src, rows) || !good(codes, rows) || !good(scales, rows) || !aligned16(zeros)) return MOK_ERR_INVALID_ARG;
  return result(launch_quantize_int4(src, rows, K, group, dtype, codes, scales, zeros, (hipStream_t)stream));
}

}  // extern "C"
