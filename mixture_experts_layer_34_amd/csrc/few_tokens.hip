// The whole expert layer for a few tokens (a decode step of up to sixteen
// sequences) in two launches, four with adapters:
//   route   e_1..e_k of token t: its k largest logits, gates g_j
//   UP      h_p = g_j silu(W1_e x_t) * (W3_e x_t)      of each pair p = (t, j)
//   DOWN    out_t = sum_j W2_e h_p
// and, where adapter l of token t stands beside the expert's matrices, W + s_l
// B_{l,e} A_{l,e} in place of each: u = s_l A_{l,e} v of every pair first (a
// launch before UP and one before DOWN), B_{l,e} u added to the sums.
//
// Bound by reading each chosen expert's three matrices once.  What that takes:
//  - Routing needs no launch: every workgroup of UP routes the tokens itself
//    (the logits are a few KB in L2) and then takes tiles of up to sixteen columns
//    of h in turn.  Workgroup 0 writes the routing out, and the experts' pairs for
//    DOWN.
//  - No sort and no gather: an expert has a token once at most, so the sixteen
//    columns of a matrix instruction are the sixteen tokens whatever the expert.
//    Columns of tokens without the expert repeat the row of one that has it
//    (no traffic) and are not stored.
//  - No combine: with the gate applied to h in fp32, the sum over a token's
//    experts is a product whose K runs over all the chosen experts' F, zeros
//    standing in for the pairs that are not.  A workgroup of DOWN owns sixteen
//    columns of out, its waves share that K, and their fp32 sums meet in LDS in
//    wave order.
// h goes from UP to DOWN in four bytes whatever the type, for the 16-bit ones as
// two bf16 parts (store_h), so that it loses nothing next to out's own rounding
// and keeps fp32's range: in 16 bits it would be a second rounding as large as
// out's, and in fp16 an infinity past 65504 and nothing below 3e-8.  DOWN takes the
// two parts of eight tokens as the sixteen columns of a matrix instruction: all
// tokens', or those that have the expert (build_turns).  fp16 weights are two bf16
// parts there, exactly.
// All sums are fp32 in a fixed order.
// At d 4096, F 1536, 8 of 128 experts (bf16): one token 39 + 20 us (201 and 101 MB;
// 5.1 TB/s together), sixteen 540 us (3.1 GB, 5.7 TB/s; with h in 16 bits 533).
#include "few_tokens.h"
#include "frag.h"
#include "mok_internal.h"

namespace mok {
namespace {

constexpr int kUpWaves = 8;  // waves that share the K of a tile of UP
[[maybe_unused]] constexpr int kUnroll = 4;  // K steps of a chunk; one chunk is in flight while one is multiplied

// Tables of a workgroup in LDS.
struct FewTables {
  int32_t* idx;    // [P] the tokens' experts
  float* gate;     // [P]
  int16_t* expert; // [slots] local expert of each slot, ascending
  int16_t* pair;   // [slots][16] the pair of each token, -1: none
  int nslots;
};

__host__ __device__ inline int few_slots(int P, int E_loc) { return P < E_loc ? P : E_loc; }

// The local experts that the pairs name, ascending, and each one's pairs.
// bits: 32 words, base: 33.  For all threads of the workgroup.
__device__ __forceinline__ void build_slots(const FewTokens& a, FewTables& s, uint32_t* bits, int* base, int nthreads) {
  const int tid = threadIdx.x, P = a.T * a.k, most = few_slots(P, a.E_loc);
  if (tid < 32) bits[tid] = 0;
  for (int i = tid; i < most * 8; i += nthreads) reinterpret_cast<uint32_t*>(s.pair)[i] = 0xFFFFFFFFu;
  __syncthreads();
  for (int p = tid; p < P; p += nthreads) {
    const int e = s.idx[p] - a.eb;
    if (e >= 0 && e < a.E_loc) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (tid < 64) {
    const int n = tid < 32 ? __popc(bits[tid]) : 0;
    const int to = wave_prefix(n);
    if (tid < 32) base[tid] = to - n;
    if (tid == 31) base[32] = to;
  }
  __syncthreads();
  for (int p = tid; p < P; p += nthreads) {
    const int e = s.idx[p] - a.eb;
    if (e < 0 || e >= a.E_loc) continue;
    const int slot = base[e >> 5] + __popc(bits[e >> 5] & ((1u << (e & 31)) - 1u));
    s.expert[slot] = (int16_t)e;
    s.pair[slot * 16 + p / a.k] = (int16_t)p;
  }
  __syncthreads();
  s.nslots = __builtin_amdgcn_readfirstlane(base[32]);
}

// The tables as UP leaves them for DOWN: a word for their number, then the experts
// and the pairs of all `most` slots.
__host__ __device__ inline size_t few_table_bytes(int most) { return 16 + (size_t)(most + 1) / 2 * 4 + (size_t)most * 32; }
__device__ __forceinline__ int16_t* table_pairs(void* table, int most) {
  return reinterpret_cast<int16_t*>((char*)table + 16 + (size_t)(most + 1) / 2 * 4);
}

// Maximum of an unsigned word over a wave, in a scalar register.
template <int CTRL> __device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
  return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max_u32<0xb1>(v);   // quad_perm [1,0,3,2]
  v = dpp_max_u32<0x4e>(v);   // quad_perm [2,3,0,1]
  v = dpp_max_u32<0x124>(v);  // row_ror 4
  v = dpp_max_u32<0x128>(v);  // row_ror 8
  v = dpp_max_u32<0x142>(v);  // row_bcast 15
  v = dpp_max_u32<0x143>(v);  // row_bcast 31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Routing of tokens t0, t0 + step, ... below t1 by the calling wave: the layer's own
// (route_token.h), bit for bit, in fewer steps, for every workgroup does it
// before it can ask for a weight (one token of 128 experts, k 8: 3.4 -> 1.3 us).
// A round takes the largest word of the order-preserving code, six lane moves,
// and the lowest expert that holds it by ballots; the gates are computed once, by
// lane j for the j-th choice.
template <int EPL>
__device__ __forceinline__ void route_few(const FewTokens& a, int t0, int t1, int step, int32_t* idx, float* gate) {
  const int lane = lane_id(), E = a.E, k = a.k;
  float next[EPL];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      next[i] = t < t1 && e < E ? a.logits[(int64_t)t * E + e] : -INFINITY;
    }
  };
  fetch(t0);
  for (int t = t0; t < t1; t += step) {
    float v[EPL];
    uint32_t code[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] = next[i] != next[i] ? -INFINITY : next[i];  // a NaN ranks as -inf
      uint32_t u = __float_as_uint(v[i]);
      if ((u << 1) == 0) u = 0;  // -0 ties with +0
      code[i] = lane + 64 * i < E ? ((u & 0x80000000u) ? ~u : (u | 0x80000000u)) : 0u;
    }
    fetch(t + step);
    int mine = 0;        // lane j: the j-th choice and its logit
    float logit = 0.f, m = 0.f;
    for (int j = 0; j < k; ++j) {
      uint32_t best = code[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) best = code[i] > best ? code[i] : best;
      best = wave_max_u32(best);
      int e = 0;
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i) {  // the lowest index is looked for last, and stays
        const uint64_t at = __ballot(code[i] == best);
        e = at ? 64 * i + __ffsll((unsigned long long)at) - 1 : e;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 64 * i == e) code[i] = 0u;
      const float bv = __uint_as_float((best & 0x80000000u) ? (best & 0x7FFFFFFFu) : ~best);
      if (j == 0) m = bv;
      mine = lane == j ? e : mine;
      logit = lane == j ? bv : logit;
    }
    // a choice's gate is top * inv; the products enter the sum of a renormalised
    // row unrounded, as they do in the layer's router
    float top = 1.0f / (1.0f + expf(-logit)), inv = 1.0f;
    if (!(a.gating & kFewSigmoid)) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + 64 * i < E) s += expf(v[i] - m);
      top = expf(logit - m);
      inv = 1.0f / wave_sum(s);
    }
    float g = top * inv;
    if (a.gating & kFewRenorm) {
      float sum = 0.f;
      for (int j = 0; j < k; ++j) sum = fmaf(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(top), j)), inv, sum);
      g /= sum;
    }
    if (lane < k) {
      idx[t * k + lane] = mine;
      gate[t * k + lane] = g;
    }
  }
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_on2_t __attribute__((ext_vector_type(2), aligned(2)));

// h of the 16-bit types: a row of bf16 values, and a row of their bf16 rests Fp
// further on: off by 2^-16 of the value at most.  (fp16 itself has no range for h.)
// The first n of four neighbours.
template <int DT>
__device__ __forceinline__ void store_h(const FewTokens& a, int pair, int col, const float (&v)[4], int n) {
  if constexpr (DT == 0) {
    store_part<0>((char*)a.h + ((int64_t)pair * a.Fp + col) * 4, narrow<0>(v), n);
  } else {
    uint16_t* to = reinterpret_cast<uint16_t*>(a.h) + (int64_t)pair * 2 * a.Fp + col;
    u32x2_t hi, lo;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hi[i] = Elem<1>::pack(v[2 * i], v[2 * i + 1]);
      lo[i] = Elem<1>::pack(v[2 * i] - Elem<1>::lo(hi[i]), v[2 * i + 1] - Elem<1>::hi(hi[i]));
    }
    if (n >= 4) {
      *reinterpret_cast<u32x2_on2_t*>(to) = hi;
      *reinterpret_cast<u32x2_on2_t*>(to + a.Fp) = lo;
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < n) {
          to[i] = (uint16_t)(hi[i / 2] >> (16 * (i & 1)));
          to[a.Fp + i] = (uint16_t)(lo[i / 2] >> (16 * (i & 1)));
        }
    }
  }
}
// KE elements of h from `col` on, the first n of them (zeros behind).
template <int DT> __device__ __forceinline__ void load_h(const FewTokens& a, int pair, int col, int n, float* f) {
  if constexpr (DT == 0) {
    widen<0>(load_part<0>((const char*)a.h + ((int64_t)pair * a.Fp + col) * 4, n), f);
  } else {
    const char* at = (const char*)a.h + ((int64_t)pair * 2 * a.Fp + col) * 2;
    float lo[8];
    widen<1>(load_part<1>(at, n), f);
    widen<1>(load_part<1>(at + 2 * a.Fp, n), lo);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += lo[j];
  }
}

// fp16 elements as two bf16 parts whose sum they are: 8 bits of the 11 cut off, and
// the 3 that are left.
__device__ __forceinline__ void split_f16(u32x4_t v, u32x4_t* hi, u32x4_t* lo) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = Elem<2>::lo(v[j]), b = Elem<2>::hi(v[j]);
    const uint32_t ua = __float_as_uint(a) & 0xFFFF0000u, ub = __float_as_uint(b) & 0xFFFF0000u;
    const uint32_t ra = __float_as_uint(a - __uint_as_float(ua)), rb = __float_as_uint(b - __uint_as_float(ub));
    (*hi)[j] = __builtin_amdgcn_perm(ub, ua, 0x07060302);  // the high halves of both
    (*lo)[j] = __builtin_amdgcn_perm(rb, ra, 0x07060302);
  }
#endif
}

// The sum of a lane's column and of the one eight further on (mod 16).
__device__ __forceinline__ float both_parts(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x128, 0xf, 0xf, false));  // row_ror 8
}

__device__ __forceinline__ int adapter_of(const FewTokens& a, int t) {
  const int l = a.adapter[t];
  return l >= 0 && l < a.L ? l : -1;
}

// <B row, u> in fp32; u has zeros past r.
template <int DT> __device__ __forceinline__ float rank_dot(const char* b, const float* u, int r) {
  constexpr int KE = kFragElems<DT>;
  float s = 0.f;
  for (int c = 0; c < r; c += KE) {
    float f[KE];
    widen<DT>(load_part<DT>(b + (int64_t)c * Elem<DT>::kBytes, r - c), f);
#pragma unroll
    for (int j = 0; j < KE; j += 4) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(u + c + j);
#pragma unroll
      for (int q = 0; q < 4; ++q) s = fmaf(f[j + q], v[q], s);
    }
  }
  return s;
}

// LDS of UP: idx and gate [P] each, then the tables.
__host__ __device__ inline size_t up_lds(int P, int slots) { return (size_t)P * 8 + (size_t)slots * 34 + 64; }

// ODD: rows of x, W1 and W3 of an odd number of 16-bit elements.
template <int DT, int EPL, bool ODD>
__global__ __launch_bounds__(64 * kUpWaves) void few_up_kernel(FewTokens a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes, U = kUnroll;
  extern __shared__ __align__(16) char lds[];
  __shared__ f32x4_t red[2][kUpWaves - 1][2][64];
  __shared__ uint32_t bits[32];
  __shared__ int base[33];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int i16 = lane & 15, g = lane >> 4;
  const int P = a.T * a.k, most = few_slots(P, a.E_loc);
  FewTables s;
  s.idx = reinterpret_cast<int32_t*>(lds);
  s.gate = reinterpret_cast<float*>(lds + 4 * P);
  s.pair = reinterpret_cast<int16_t*>(lds + 8 * P);
  s.expert = s.pair + 16 * most;
  route_few<EPL>(a, w, a.T, kUpWaves, s.idx, s.gate);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int p = tid; p < P; p += 64 * kUpWaves) {
      a.idx[p] = s.idx[p];
      a.gate[p] = s.gate[p];
    }
  build_slots(a, s, bits, base, 64 * kUpWaves);
  if (blockIdx.x == 0) {
    if (tid == 0) *reinterpret_cast<int32_t*>(a.table) = s.nslots;
    for (int i = tid; i < s.nslots; i += 64 * kUpWaves) reinterpret_cast<int16_t*>((char*)a.table + 16)[i] = s.expert[i];
    for (int i = tid; i < s.nslots * 8; i += 64 * kUpWaves)
      reinterpret_cast<uint32_t*>(table_pairs(a.table, most))[i] = reinterpret_cast<const uint32_t*>(s.pair)[i];
  }

  // Columns of h: those of all slots one after the other, in tiles of up to
  // sixteen that the workgroups take in turn.  A compute unit with more to read
  // than another ends later by as much (they get even shares of the memory's rate),
  // so the tiles are as wide as makes every workgroup take the same number of them.
  const int64_t total = (int64_t)s.nslots * a.F;
  int64_t n = (total + 15) / 16;
  n = (n + kNumCUs - 1) / kNumCUs * kNumCUs;
  if (n > gridDim.x) n = gridDim.x;
  if (blockIdx.x >= n || total == 0) return;
  const int64_t tiles = ((total + 15) / 16 + n - 1) / n * n;
  int64_t tile = blockIdx.x, pos = total * tile / tiles, end = total * (tile + 1) / tiles;
  const int full = a.d / STEP;                                    // whole K steps
  const int all = full / U;                                      // whole chunks: the waves take them in turn
  const int chunks = all > w ? (all - w + kUpWaves - 1) / kUpWaves : 0;
  const int64_t row_bytes = (int64_t)a.d * S;
  // A tile, or its part of one expert.  A lane's row of W1 and W3, and
  // its token's row of x (of a token that has the expert, for those that have not).
  struct Tile {
    int n0, cols, e, pair;
    const char *p1, *p3, *px;
  };
  auto open = [&](int64_t at) {
    Tile t;
    const int slot = (int)(at / a.F);
    t.n0 = (int)(at - (int64_t)slot * a.F);
    t.cols = a.F - t.n0 < 16 ? a.F - t.n0 : 16;
    t.cols = end - at < t.cols ? (int)(end - at) : t.cols;
    t.e = __builtin_amdgcn_readfirstlane(s.expert[slot]);
    t.pair = s.pair[slot * 16 + i16];
    const uint64_t has = __ballot(t.pair >= 0);
    const int tx = t.pair >= 0 ? i16 : __ffsll((unsigned long long)has) - 1;
    const int n = t.n0 + (i16 < t.cols ? i16 : t.cols - 1);
    const int64_t row = ((int64_t)t.e * a.F + n) * row_bytes + (int64_t)(g * KE) * S;
    t.p1 = (const char*)a.w[0] + row;
    t.p3 = (const char*)a.w[1] + row;
    t.px = (const char*)a.x + tx * row_bytes + (int64_t)(g * KE) * S;
    return t;
  };
  Quad<DT, ODD> q1[2][U], q3[2][U], qx[2][U];
  auto load = [&](int buf, const char* p1, const char* p3, const char* px, int c) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int o = ((c * kUpWaves + w) * U + j) * STEP * S;
      q1[buf][j].load(p1 + o);
      q3[buf][j].load(p3 + o);
      qx[buf][j].load(px + o);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // the columns behind: of the same tile, or of the next that has any
  auto step = [&](int by) {
    pos += by;
    while (pos >= end && (tile += n) < tiles) {
      pos = total * tile / tiles;
      end = total * (tile + 1) / tiles;
    }
    return pos < end;
  };
  if (!step(0)) return;
  Tile t = open(pos);
  if (chunks) load(0, t.p1, t.p3, t.px, 0);
  bool more = true;
  for (int flip = 0; more; flip ^= 1) {
    more = step(t.cols);
    const Tile next = more ? open(pos) : t;
    const int n0 = t.n0, cols = t.cols, e = t.e, pair = t.pair;
    const char *p1 = t.p1, *p3 = t.p3, *px = t.px;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const uint32_t h1 = shift_of<ODD>(p1), h3 = shift_of<ODD>(p3), hx = shift_of<ODD>(px);
    auto mul = [&](int buf) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const u32x4_t vx = qx[buf][j].get(hx);
        acc[0] = mma<DT>(q1[buf][j].get(h1), vx, acc[0]);
        acc[1] = mma<DT>(q3[buf][j].get(h3), vx, acc[1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // Chunk c + 1 is in flight while chunk c is multiplied, and the next tile's
    // first chunk while this one's last is, and through what ends the tile.  No
    // load stands under a condition (where there is none to ask for, one is asked
    // for again): behind a branch the compiler can only wait for every load, and
    // the ring would run empty at each turn.  And it may not move loads to their
    // uses, where they save it registers.
    for (int c = 0; c < chunks; c += 2) {
      load(1, p1, p3, px, c + 1 < chunks ? c + 1 : c);
      mul(0);
      const bool here = c + 2 < chunks;
      load(0, here ? p1 : next.p1, here ? p3 : next.p3, here ? px : next.px, here ? c + 2 : 0);
      if (c + 1 < chunks) mul(1);
    }
    // the steps that fill no chunk, a wave each, and the step that d ends in
    for (int i = all * U; i < full; ++i)
      if (i % kUpWaves == w) {
        const int o = i * STEP * S;
        const u32x4_t vx = load16<DT>(px + o);
        acc[0] = mma<DT>(load16<DT>(p1 + o), vx, acc[0]);
        acc[1] = mma<DT>(load16<DT>(p3 + o), vx, acc[1]);
      }
    if (full * STEP < a.d && w == 0) {
      const int k = full * STEP + g * KE;
      if (a.d >= KE) {
        const int at = tail_at<DT>(k, a.d), o = (at - g * KE) * S;  // the pointers stand at element g KE
        const u32x4_t v1 = load16<DT>(p1 + o), v3 = load16<DT>(p3 + o), vx = but_first<DT>(load16<DT>(px + o), k - at);
        acc[0] = mma<DT>(v1, vx, acc[0]);
        acc[1] = mma<DT>(v3, vx, acc[1]);
      } else {
        const int left = a.d - k, o = full * STEP * S;
        const u32x4_t vx = load_part<DT>(px + o, left);
        acc[0] = mma<DT>(load_part<DT>(p1 + o, left), vx, acc[0]);
        acc[1] = mma<DT>(load_part<DT>(p3 + o, left), vx, acc[1]);
      }
    }
    const int l = a.adapter && pair >= 0 ? adapter_of(a, i16) : -1;
    if (l >= 0 && w < 4) {  // wave w adds the adapter's share of row 4 g + w of the tile
      const int nr = n0 + 4 * g + w;
      if (4 * g + w < cols)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          if (a.lora[m].A) {
            const int r = a.lora[m].r;
            const float v = rank_dot<DT>(
                (const char*)a.lora[m].B + (((int64_t)l * a.E_loc + e) * a.F + nr) * r * S,
                a.u[m] + (int64_t)pair * few_u_width(r), r);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] += i == w ? v : 0.f;
          }
    }
    // the waves' sums in wave order; the two halves of `red` take turns, so that
    // one barrier a unit is enough
    if (w > 0) {
      red[flip][w - 1][0][lane] = acc[0];
      red[flip][w - 1][1][lane] = acc[1];
    }
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int q = 0; q < kUpWaves - 1; ++q) {
        acc[0] += red[flip][q][0][lane];
        acc[1] += red[flip][q][1][lane];
      }
      if (pair >= 0) {
        const float gt = s.gate[pair];
        float hv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) hv[i] = acc[0][i] * sigmoidf_(acc[0][i]) * acc[1][i] * gt;
        store_h<DT>(a, pair, n0 + 4 * g, hv, cols - 4 * g);
      }
    }
    t = next;
  }
#endif
}

// A workgroup owns `cols` columns of out, up to 16 NT: as many as give every
// compute unit the same share.
constexpr int kDownWaves = 8;

// More than eight tokens of a 16-bit type: each expert's tokens in turns of up to eight,
// in their order; an expert with more has two turns, one after the other, the second
// of which finds W2 in L2.  (Both parts by two matrix instructions of sixteen tokens
// each want twice the accesses of h: 16 tokens of d 4096, F 1536, 8 of 128 experts took
// 561 us so and take 540 in turns; all of 8 experts, two turns each, 95 and 99.)
struct FewTurns {
  int16_t* pair;   // [turns][8], -1: none
  int8_t* at;      // [turns][16] the place of each token, -1: none
  int16_t* expert; // [turns]
};
__host__ __device__ inline int few_turns(int P, int slots) { return slots + P / 9; }
// For all threads of the workgroup; the number of turns.  over: 16 words.
__device__ __forceinline__ int build_turns(const FewTokens& a, const FewTurns& s, int most, int turns, uint64_t* over) {
  constexpr int N = 64 * kDownWaves;
  const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
  const int nslots = *reinterpret_cast<const int32_t*>(a.table);
  const uint32_t* from = reinterpret_cast<const uint32_t*>(table_pairs(a.table, most));
  for (int i = tid; i < turns * 4; i += N) {
    reinterpret_cast<uint32_t*>(s.pair)[i] = 0xFFFFFFFFu;
    reinterpret_cast<uint32_t*>(s.at)[i] = 0xFFFFFFFFu;
  }
  uint32_t pairs[2][8];  // of slots tid and tid + N, two a word
  int n[2] = {0, 0};
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int slot = tid + r * N;
    if (64 * w + r * N >= most) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      pairs[r][i] = slot < nslots ? from[slot * 8 + i] : 0xFFFFFFFFu;
      n[r] += ((int32_t)pairs[r][i] >= 0) + ((int16_t)pairs[r][i] >= 0);
    }
    const uint64_t b = __ballot(n[r] > 8);
    if (lane == 0) over[w + r * kDownWaves] = b;
  }
  __syncthreads();
  int second = 0;  // second turns of the slots before this wave's, and of all
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int slot = tid + r * N;
    second = 0;
    for (int i = 0; i < w + r * kDownWaves && 64 * i < most; ++i) second += __popcll(over[i]);
    if (slot < nslots) {
      const uint64_t b = over[w + r * kDownWaves];
      const int v = slot + second + __popcll(b & ((1ull << lane) - 1ull));
      const int16_t e = reinterpret_cast<const int16_t*>((const char*)a.table + 16)[slot];
      s.expert[v] = e;
      if (n[r] > 8) s.expert[v + 1] = e;
      int c = 0;
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const int16_t pair = (int16_t)(pairs[r][t / 2] >> (16 * (t & 1)));
        if (pair < 0) continue;
        s.pair[v * 8 + c] = pair;  // (place 8 of a turn is place 0 of the next)
        s.at[(v + (c >> 3)) * 16 + t] = (int8_t)(c & 7);
        ++c;
      }
    }
  }
  __syncthreads();
  second = 0;
  for (int i = 0; 64 * i < most; ++i) second += __popcll(over[i]);
  return __builtin_amdgcn_readfirstlane(nslots + second);
}

// LONG: F >= KE.  ODD: rows of W2 of an odd number of 16-bit elements.  MANY: turns of
// eight tokens (16-bit types).  A 16-bit type's columns 0..7 are the first parts of h
// and 8..15 the second ones.
template <int DT, int NT, bool WHOLE, bool LONG, bool ODD, bool MANY>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(FewTokens a, int cols) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes, U = kUnroll, NW = kDownWaves;
  extern __shared__ __align__(16) char lds[];
  __shared__ f32x4_t red[NW][NT][64];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int i16 = lane & 15, g = lane >> 4, col = DT != 0 ? i16 & 7 : i16;  // col: the lane's token, or its place
  const int P = a.T * a.k, most = few_slots(P, a.E_loc);
  constexpr int COLS = MANY ? 8 : 16;  // pairs of a slot
  int nslots;  // or turns
  int16_t *s_pair = reinterpret_cast<int16_t*>(lds), *s_expert;
  int8_t* s_at = nullptr;
  if constexpr (MANY) {
    __shared__ uint64_t over[2 * NW];
    const int turns = few_turns(P, most);
    s_at = reinterpret_cast<int8_t*>(s_pair + 8 * turns);
    s_expert = reinterpret_cast<int16_t*>(s_at + 16 * turns);
    nslots = build_turns(a, FewTurns{s_pair, s_at, s_expert}, most, turns, over);
  } else {
    s_expert = s_pair + 16 * most;
    nslots = *reinterpret_cast<const int32_t*>(a.table);
    for (int i = tid; i < most * 8; i += 64 * NW)
      reinterpret_cast<uint32_t*>(s_pair)[i] = reinterpret_cast<const uint32_t*>(table_pairs(a.table, most))[i];
    for (int i = tid; i < most; i += 64 * NW)
      s_expert[i] = reinterpret_cast<const int16_t*>((const char*)a.table + 16)[i];
    __syncthreads();
  }

  const int n0 = blockIdx.x * cols, n1 = n0 + cols < a.d ? n0 + cols : a.d;
  const int64_t row_bytes = (int64_t)a.F * S;
  int64_t wrow[NT];  // the lane's rows of W2, in bytes from the expert's first
#pragma unroll
  for (int q = 0; q < NT; ++q) {
    const int n = n0 + 16 * q + i16;
    wrow[q] = (n < n1 ? n : n1 - 1) * row_bytes;
  }
  const int chunks = (a.F + STEP * U - 1) / (STEP * U);  // of one expert
  const int all = nslots * chunks;  // the waves take them in turn: what they read at a time is neighbouring
  const int mine = all > w ? (all - w + NW - 1) / NW : 0;
  // (the last row's last access may end eight bytes behind it, in the tables)
  const auto hrs = __builtin_amdgcn_make_buffer_rsrc(a.h, (short)0, (int)((int64_t)P * a.Fp * 4 + 16), 0x00020000);
  // cursor of the next chunk to load; past the last one it stays on it
  const int skip_slots = NW / chunks, skip = NW - skip_slots * chunks;
  int slot = w / chunks, ch = w - slot * chunks;
  f32x4_t acc[NT];
#pragma unroll
  for (int q = 0; q < NT; ++q) acc[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Quad<DT, ODD> qw[2][U][NT];
  u32x4_t qh[2][U];
  uint32_t odd[2];  // a bit for each access of a chunk that starts off a dword
  int at[2];        // the place of the lane's token in the chunk's columns, < 0: it has not the expert
  int left[2];  // !WHOLE: elements of F from the lane's first of the chunk
  // WHOLE: F is a multiple of KE, a lane's 16 bytes lie in F or past it; a
  // lane past it reads the row's first bytes and zeros of h.  Otherwise the lane
  // that F ends in reads the row's last 16 bytes and moves them to their places.
  auto load = [&](int buf) {
    const int e = __builtin_amdgcn_readfirstlane(s_expert[slot]);
    const int pair = s_pair[slot * COLS + col];
    // a pair that is not: an offset past the buffer, which loads zeros
    const uint32_t hoff = pair >= 0 ? (uint32_t)(pair * a.Fp) * 4 + (DT != 0 && i16 > 7 ? a.Fp * 2 : 0) : 0xC0000000u;
    const char* wp = (const char*)a.w[2] + (int64_t)e * a.d * row_bytes;
    left[buf] = a.F - ch * U * STEP - g * KE;
    odd[buf] = 0;
    at[buf] = MANY ? s_at[slot * 16 + i16] : pair;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = (ch * U + j) * STEP + g * KE;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        if constexpr (LONG) {
          const char* from = wp + wrow[q] + (WHOLE ? (k < a.F ? k : 0) : tail_at<DT>(k, a.F)) * S;
          qw[buf][j][q].load(from);
          odd[buf] |= shift_of<ODD>(from) / 16 << (j * NT + q);
        } else {
          qw[buf][j][q].v = load_part<DT>(wp + wrow[q] + k * S, k < a.F ? a.F - k : 0);
        }
      }
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(hrs, k < a.F ? hoff + k * S : 0xC0000000u, 0, 0);
      qh[buf][j] = u32x4_t{(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]};
    }
    const bool wrap = ch + skip >= chunks;
    const int next = slot + skip_slots + wrap;
    ch = next < nslots ? ch + skip - (wrap ? chunks : 0) : ch;
    slot = next < nslots ? next : slot;
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mul = [&](int buf) {
    f32x4_t sum[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) sum[q] = MANY ? f32x4_t{0.f, 0.f, 0.f, 0.f} : acc[q];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      // past F nothing was written
      if constexpr (!WHOLE) qh[buf][j] = first_elems<DT>(qh[buf][j], left[buf] - j * STEP);
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        u32x4_t vw = qw[buf][j][q].get((odd[buf] >> (j * NT + q) & 1) * 16);
        if constexpr (!WHOLE && LONG) {
          const int in = left[buf] - j * STEP;
          vw = shift_elems<DT>(vw, in < KE ? KE - in : 0);
        }
        u32x4_t rest;
        if constexpr (DT == 2) split_f16(vw, &vw, &rest);
        sum[q] = mma<DT == 0 ? 0 : 1>(vw, qh[buf][j], sum[q]);
        if constexpr (DT == 2) sum[q] = mma<1>(rest, qh[buf][j], sum[q]);
      }
    }
    // A token takes its own column's sum (MANY: both parts', from its place in the turn),
    // and one without the expert none: zeros times an infinite weight are not 0.
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = sum[q][i];
        if constexpr (MANY) {
          const int lane_of = 16 * g + (at[buf] & 7);
          v = acc[q][i] + __uint_as_float(__builtin_amdgcn_ds_bpermute(4 * lane_of, __float_as_uint(both_parts(v))));
        }
        acc[q][i] = at[buf] >= 0 ? v : acc[q][i];
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  if (mine) {  // no load under a condition, as in UP
    load(0);
    int c = 0;
    for (; c + 2 <= mine; c += 2) {
      load(1);
      mul(0);
      load(0);
      mul(1);
    }
    if (c < mine) mul(0);
  }
  // the adapters: wave w takes slots w, w + NW, ... of every token
  if (a.adapter && a.lora[2].A && i16 < a.T) {
    const int l = adapter_of(a, i16), r = a.lora[2].r;
    if (l >= 0)
      for (int j = w; j < a.k; j += NW) {
        const int p = i16 * a.k + j, el = a.idx[p] - a.eb;
        if (el < 0 || el >= a.E_loc) continue;
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = n0 + 16 * q + 4 * g + i;
            if (n < n1)
              acc[q][i] += rank_dot<DT>((const char*)a.lora[2].B + (((int64_t)l * a.E_loc + el) * a.d + n) * r * S,
                                        a.u[2] + (int64_t)p * few_u_width(r), r);
          }
      }
  }
#pragma unroll
  for (int q = 0; q < NT; ++q) red[w][q][lane] = acc[q];
  __syncthreads();
  if (w < NT) {  // a wave for each sixteen columns
    f32x4_t v = red[0][w][lane];
#pragma unroll
    for (int k = 1; k < NW; ++k) v += red[k][w][lane];
    if constexpr (DT != 0 && !MANY)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = both_parts(v[i]);
    const int n = n0 + 16 * w + 4 * g;
    const int64_t o = (int64_t)i16 * a.d + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i16 < a.T && n + i < n1) {
        if constexpr (DT == 0) reinterpret_cast<float*>(a.out)[o + i] = v[i];
        else reinterpret_cast<uint16_t*>(a.out)[o + i] = (uint16_t)Elem<DT>::pack(v[i], 0.f);
      }
  }
#endif
}

// u = s_l A_{l,e} v of a pair: v = x_t for W1's and W3's adapters (DOWN false;
// the workgroup routes its token itself), h_p for W2's.  A wave takes one rank.
// grid: (pair, ranks / 4 of the one matrix, then of the other).
template <int DT, int EPL, bool DOWN> __global__ __launch_bounds__(256) void few_rank_kernel(FewTokens a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes;
  __shared__ int32_t idx[kFewSlots];
  __shared__ float gate[kFewSlots];
  const int lane = lane_id(), w = wave_id();
  const int p = blockIdx.x, t = p / a.k, j = p - t * a.k;
  const int l = adapter_of(a, t);
  if (l < 0) return;
  int m = 2, y = blockIdx.y, e;
  if constexpr (DOWN) {
    e = a.idx[p];
  } else {
    const int q1 = a.lora[0].A ? few_u_width(a.lora[0].r) / 4 : 0;
    m = y < q1 ? 0 : 1;
    y -= m ? q1 : 0;
    if (w == 0) {  // token t alone, as token 0 of its own row
      FewTokens one = a;
      one.logits = a.logits + (int64_t)t * a.E;
      route_few<EPL>(one, 0, 1, 1, idx, gate);
    }
    __syncthreads();
    e = idx[j];
  }
  e -= a.eb;
  if (e < 0 || e >= a.E_loc) return;
  const int r = a.lora[m].r, rr = 4 * y + w, K = DOWN ? a.F : a.d;
  float* to = a.u[m] + (int64_t)p * few_u_width(r) + rr;
  float sum = 0.f;
  if (rr < r) {
    const char* x = (const char*)a.x + (int64_t)t * K * S;
    const char* row = (const char*)a.lora[m].A + (((int64_t)l * a.E_loc + e) * r + rr) * K * S;
#pragma unroll 4
    for (int c = lane * KE; c < K; c += 64 * KE) {
      float fa[KE], fv[KE];
      widen<DT>(load_part<DT>(row + (int64_t)c * S, K - c), fa);
      if constexpr (DOWN) load_h<DT>(a, p, c, K - c, fv);
      else widen<DT>(load_part<DT>(x + (int64_t)c * S, K - c), fv);
#pragma unroll
      for (int i = 0; i < KE; ++i) sum = fmaf(fa[i], fv[i], sum);
    }
    sum = wave_sum(sum) * (a.lora[m].scale ? a.lora[m].scale[l] : 1.f);
  }
  if (lane == 0) *to = sum;
#endif
}

template <int DT, int NT, bool WHOLE, bool LONG, bool ODD> void down(const FewTokens& a, int cols, int slots, hipStream_t s) {
  const dim3 grid((a.d + cols - 1) / cols), block(64 * kDownWaves);
  if (DT != 0 && a.T > 8)
    hipLaunchKernelGGL((few_down_kernel<DT, NT, WHOLE, LONG, ODD, DT != 0>), grid, block,
                       (size_t)few_turns(a.T * a.k, slots) * 34 + 64, s, a, cols);
  else
    hipLaunchKernelGGL((few_down_kernel<DT, NT, WHOLE, LONG, ODD, false>), grid, block, (size_t)slots * 34 + 64, s, a, cols);
}

template <int DT, int EPL, bool ODD> void up(const FewTokens& a, int P, int slots, hipStream_t s) {
  static const int per_cu = [] {
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, few_up_kernel<DT, EPL, ODD>, 64 * kUpWaves, 8192) !=
            hipSuccess || n < 1)
      n = 1;
    return n;
  }();
  // as many workgroups as are resident at once beside tables of 8 KB (larger ones leave
  // fewer, and the rest follow), in whole rounds of the compute units; of those the
  // kernel uses what the chosen experts' columns take
  const int64_t units = ((int64_t)slots * a.F + 15) / 16, cap = (int64_t)kNumCUs * per_cu;
  const int64_t rounds = (units + kNumCUs - 1) / kNumCUs * kNumCUs;
  hipLaunchKernelGGL((few_up_kernel<DT, EPL, ODD>), dim3((unsigned)(rounds < cap ? rounds : cap)), dim3(64 * kUpWaves),
                     up_lds(P, slots), s, a);
}

template <int DT, int EPL> hipError_t run(const FewTokens& a, hipStream_t s) {
  const int P = a.T * a.k, slots = few_slots(P, a.E_loc);
  int ranks = 0;
  for (int m = 0; m < 2; ++m)
    if (a.lora[m].A) ranks += few_u_width(a.lora[m].r) / 4;
  if (a.adapter && ranks)
    hipLaunchKernelGGL((few_rank_kernel<DT, EPL, false>), dim3(P, ranks), dim3(256), 0, s, a);
  if (DT != 0 && a.d % 2) up<DT, EPL, DT != 0>(a, P, slots, s);
  else up<DT, EPL, false>(a, P, slots, s);
  if (a.adapter && a.lora[2].A)
    hipLaunchKernelGGL((few_rank_kernel<DT, EPL, true>), dim3(P, few_u_width(a.lora[2].r) / 4), dim3(256), 0, s, a);
  // columns of a workgroup of DOWN: d shared out evenly over the compute units,
  // in as few rounds of them as 32 columns each allow
  const int share = (a.d + 32 * kNumCUs - 1) / (32 * kNumCUs) * kNumCUs, cols = (a.d + share - 1) / share;
  constexpr int KE = kFragElems<DT>;
  if (a.F % KE == 0)
    cols <= 16 ? down<DT, 1, true, true, false>(a, cols, slots, s) : down<DT, 2, true, true, false>(a, cols, slots, s);
  else if (a.F < KE)
    cols <= 16 ? down<DT, 1, false, false, false>(a, cols, slots, s) : down<DT, 2, false, false, false>(a, cols, slots, s);
  else if (DT != 0 && a.F % 2)
    cols <= 16 ? down<DT, 1, false, true, DT != 0>(a, cols, slots, s) : down<DT, 2, false, true, DT != 0>(a, cols, slots, s);
  else
    cols <= 16 ? down<DT, 1, false, true, false>(a, cols, slots, s) : down<DT, 2, false, true, false>(a, cols, slots, s);
  return hipGetLastError();
}

template <int DT> hipError_t run_e(const FewTokens& a, hipStream_t s) {
  return a.E <= 128 ? run<DT, 2>(a, s) : a.E <= 256 ? run<DT, 4>(a, s) : run<DT, 16>(a, s);
}

}  // namespace

size_t few_table_size(int T, int k, int E_loc) { return few_table_bytes(few_slots(T * k, E_loc)); }

hipError_t launch_few_tokens(const FewTokens& a, hipStream_t s) {
  return a.dtype == 0 ? run_e<0>(a, s) : a.dtype == 1 ? run_e<1>(a, s) : run_e<2>(a, s);
}

}  // namespace mok
