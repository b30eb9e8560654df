// C ABI of the separate expert operators (include/mok.h): argument checks on
// the host, then the launches on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/mok.h"
#include "few_tokens.h"
#include "int4_matvec.h"
#include "lora_rows.h"
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

// Parts of a workspace, one after the other on 256 bytes.
struct Parts {
  size_t total = 0;
  size_t take(int64_t n) {
    const size_t at = total;
    total += ((size_t)n + 255) & ~(size_t)255;
    return at;
  }
};

bool bad_dtype(int32_t t) { return t != MOK_DTYPE_F32 && t != MOK_DTYPE_BF16 && t != MOK_DTYPE_F16; }
int64_t elem_bytes(int32_t t) { return t == MOK_DTYPE_F32 ? 4 : 2; }
bool bad_rank(int32_t r) { return r < 1 || r > kLoraMaxRank; }

struct FewLayout {
  size_t h, table, u[3], total;
};
mok_status few_layout(const mok_few_token_config* cfg, const mok_lora_weights* lora, FewLayout* o) {
  if (!cfg) return MOK_ERR_INVALID_ARG;
  const mok_few_token_config& c = *cfg;
  if (c.T < 0 || c.T > kFewTokens || c.d < 1 || c.d > 65536 || c.ffn < 1 || c.ffn > 65536) return MOK_ERR_INVALID_ARG;
  if (bad_experts(c.E, c.expert_begin, c.expert_end) || c.k < 1 || c.k > c.E || c.k > kFewSlots)
    return MOK_ERR_INVALID_ARG;
  if (bad_dtype(c.dtype) || (c.flags & ~(MOK_FLAG_SIGMOID_GATES | MOK_FLAG_RENORM_GATES))) return MOK_ERR_INVALID_ARG;
  const int64_t P = (int64_t)c.T * c.k;
  Parts p;
  const int64_t h = P * few_h_width(c.ffn, c.dtype) * 4;  // whole 16 bytes: the tables follow at once
  o->h = p.take(h + (P ? few_table_size(c.T, c.k, c.expert_end - c.expert_begin) : 0));
  o->table = o->h + h;
  for (int m = 0; m < 3; ++m) {
    o->u[m] = p.total;
    if (!lora) continue;
    if ((lora[m].A != nullptr) != (lora[m].B != nullptr)) return MOK_ERR_INVALID_ARG;
    if (!lora[m].A) continue;
    if (bad_rank(lora[m].r) || c.L < 1) return MOK_ERR_INVALID_ARG;
    o->u[m] = p.take(P * few_u_width(lora[m].r) * 4);
  }
  o->total = p.total;
  return MOK_OK;
}

struct LoraLayout {
  size_t part, At, Bt, du, sums, total;
  int splits;
  LoraGradPlan grad;
};
mok_status lora_layout(const mok_lora_config* cfg, int32_t r, bool backward, LoraLayout* o) {
  if (!cfg) return MOK_ERR_INVALID_ARG;
  const mok_lora_config& c = *cfg;
  if (c.rows < 0 || c.rows >= (1 << 30) || bad_experts(c.E, c.expert_begin, c.expert_end)) return MOK_ERR_INVALID_ARG;
  if (c.K < 1 || c.K > (1 << 20) || c.N < 1 || c.N > (1 << 20) || bad_rank(r) || bad_dtype(c.dtype))
    return MOK_ERR_INVALID_ARG;
  // the tiles of a launch are counted in 32 bits
  if ((int64_t)c.rows * (c.K > c.N ? c.K : c.N) >= (int64_t(1) << 40)) return MOK_ERR_INVALID_ARG;
  const int G = c.expert_end - c.expert_begin;
  Parts p;
  o->splits = lora_splits(c.rows, G, r, backward ? c.N : c.K, c.dtype);
  o->part = p.take((int64_t)o->splits * c.rows * lora_width(r) * 4);
  if (backward) {
    o->At = p.take((int64_t)G * r * c.K * elem_bytes(c.dtype));
    o->Bt = p.take((int64_t)G * r * c.N * elem_bytes(c.dtype));
    o->du = o->splits > 1 ? p.take((int64_t)c.rows * lora_width(r) * 4) : o->part;
    o->grad = lora_grad_plan(c.rows, G, r, c.K, c.N, c.dtype);
    o->sums = p.take(o->grad.part_bytes);
  }
  o->total = p.total;
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

mok_status mok_few_token_workspace_query(const mok_few_token_config* cfg, const mok_lora_weights* lora,
                                         size_t* workspace_bytes) {
  FewLayout l;
  const mok_status st = few_layout(cfg, lora, &l);
  if (st != MOK_OK) return st;
  if (!workspace_bytes) return MOK_ERR_INVALID_ARG;
  *workspace_bytes = l.total;
  return MOK_OK;
}

mok_status mok_few_token_layer(const void* x, const float* router_logits, const void* W1, const void* W3,
                               const void* W2, const int32_t* adapter, const mok_lora_weights* lora,
                               const mok_few_token_config* cfg, void* out, int32_t* topk_idx, float* topk_gate,
                               void* workspace, void* stream) {
  FewLayout l;
  const mok_status st = few_layout(cfg, lora, &l);
  if (st != MOK_OK) return st;
  const mok_few_token_config& c = *cfg;
  if (!good(x, c.T) || !good(router_logits, c.T) || !good(W1, 1) || !good(W3, 1) || !good(W2, 1) || !good(out, c.T) ||
      !good(topk_idx, c.T) || !good(topk_gate, c.T) || !good(workspace, c.T))
    return MOK_ERR_INVALID_ARG;
  if ((lora != nullptr) != (adapter != nullptr) && c.T > 0) return MOK_ERR_INVALID_ARG;
  if (!aligned16(adapter)) return MOK_ERR_INVALID_ARG;
  if (c.T == 0) return MOK_OK;
  FewTokens a{};
  a.x = x;
  a.logits = router_logits;
  a.w[0] = W1;
  a.w[1] = W3;
  a.w[2] = W2;
  a.out = out;
  a.idx = topk_idx;
  a.gate = topk_gate;
  a.h = (char*)workspace + l.h;
  a.table = (char*)workspace + l.table;
  bool any = false;
  for (int m = 0; m < 3 && lora; ++m) {
    if (!aligned16(lora[m].A) || !aligned16(lora[m].B) || !aligned16(lora[m].scale)) return MOK_ERR_INVALID_ARG;
    a.lora[m] = FewLora{lora[m].A, lora[m].B, lora[m].scale, lora[m].r};
    a.u[m] = (float*)((char*)workspace + l.u[m]);
    any |= lora[m].A != nullptr;
  }
  a.adapter = any ? adapter : nullptr;
  a.T = c.T;
  a.d = c.d;
  a.F = c.ffn;
  a.Fp = few_h_width(c.ffn, c.dtype);
  a.E = c.E;
  a.eb = c.expert_begin;
  a.E_loc = c.expert_end - c.expert_begin;
  a.k = c.k;
  a.L = c.L;
  a.dtype = c.dtype;
  a.gating = (c.flags & MOK_FLAG_SIGMOID_GATES ? kFewSigmoid : 0) | (c.flags & MOK_FLAG_RENORM_GATES ? kFewRenorm : 0);
  return result(launch_few_tokens(a, (hipStream_t)stream));
}

mok_status mok_lora_workspace_query(const mok_lora_config* cfg, int32_t r, size_t* forward_bytes,
                                    size_t* backward_bytes) {
  LoraLayout f, b;
  mok_status st = lora_layout(cfg, r, false, &f);
  if (st == MOK_OK) st = lora_layout(cfg, r, true, &b);
  if (st != MOK_OK) return st;
  if (!forward_bytes || !backward_bytes) return MOK_ERR_INVALID_ARG;
  *forward_bytes = f.total;
  *backward_bytes = b.total;
  return MOK_OK;
}

mok_status mok_lora_rows(const void* x, const void* y, const int32_t* pair_of_row, const int32_t* row_of_pair,
                         const int32_t* offsets, const mok_lora_weights* w, const mok_lora_config* cfg, void* out,
                         float* u, void* workspace, void* stream) {
  if (!w) return MOK_ERR_INVALID_ARG;
  LoraLayout l;
  const mok_status st = lora_layout(cfg, w->r, false, &l);
  if (st != MOK_OK) return st;
  const mok_lora_config& c = *cfg;
  if (!good(x, c.rows) || !aligned16(y) || !good(out, c.rows) || !good(w->A, 1) || !good(w->B, 1) ||
      !aligned16(w->scale) || !good(offsets, 1) || !aligned16(u) || !good(workspace, c.rows))
    return MOK_ERR_INVALID_ARG;
  if (!aligned16(pair_of_row) || !aligned16(row_of_pair) || (pair_of_row != nullptr) != (row_of_pair != nullptr))
    return MOK_ERR_INVALID_ARG;
  if (c.rows == 0) return MOK_OK;
  const LoraMap map{offsets + c.expert_begin, pair_of_row, row_of_pair, c.rows, c.expert_end - c.expert_begin};
  float* part = (float*)((char*)workspace + l.part);
  hipError_t e = launch_lora_rank(LoraRank{map, x, w->A, part, c.K, w->r, c.dtype, l.splits}, (hipStream_t)stream);
  if (e == hipSuccess)
    e = launch_lora_add(LoraAdd{map, part, w->B, w->scale, y, out, u, c.N, w->r, c.dtype, l.splits, w->r}, (hipStream_t)stream);
  return result(e);
}

mok_status mok_lora_rows_backward(const void* dout, const void* x, const float* u, const void* base,
                                  const int32_t* pair_of_row, const int32_t* row_of_pair, const int32_t* offsets,
                                  const mok_lora_weights* w, const mok_lora_config* cfg, void* dx, float* dA,
                                  float* dB, void* workspace, void* stream) {
  if (!w) return MOK_ERR_INVALID_ARG;
  LoraLayout l;
  const mok_status st = lora_layout(cfg, w->r, true, &l);
  if (st != MOK_OK) return st;
  const mok_lora_config& c = *cfg;
  if (!good(dout, c.rows) || !good(x, c.rows) || !good(u, c.rows) || !aligned16(base) || !good(dx, c.rows) ||
      !good(dA, 1) || !good(dB, 1) || !good(w->A, 1) || !good(w->B, 1) || !aligned16(w->scale) || !good(offsets, 1) ||
      !good(workspace, 1))
    return MOK_ERR_INVALID_ARG;
  if (!aligned16(pair_of_row) || !aligned16(row_of_pair) ||
      ((pair_of_row != nullptr) != (row_of_pair != nullptr) && c.rows > 0))
    return MOK_ERR_INVALID_ARG;
  const LoraMap map{offsets + c.expert_begin, pair_of_row, row_of_pair, c.rows, c.expert_end - c.expert_begin};
  char* ws = (char*)workspace;
  float *part = (float*)(ws + l.part), *du = (float*)(ws + l.du);
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = launch_lora_prepare(LoraPrepare{map, w->A, w->B, ws + l.At, ws + l.Bt, dA, dB, w->r, c.K, c.N,
                                                 c.dtype}, s);
  if (c.rows > 0) {
    if (e == hipSuccess)
      e = launch_lora_rank(LoraRank{map, dout, ws + l.Bt, part, c.N, w->r, c.dtype, l.splits}, s);
    if (e == hipSuccess)
      e = launch_lora_add(LoraAdd{map, part, ws + l.At, w->scale, base, dx, l.splits == 1 ? nullptr : du, c.K, w->r,
                                  c.dtype, l.splits, lora_width(w->r)}, s);
    if (e == hipSuccess)
      e = launch_lora_grad(LoraGrad{map, {x, dout}, {du, u}, {dA, dB}, {c.K, c.N}, w->scale, w->r, c.dtype,
                                    l.grad.ranges, l.grad.part_bytes ? (float*)(ws + l.sums) : nullptr}, s);
  }
  return result(e);
}

}  // extern "C"
