// The whole expert layer for a few tokens (a decode step of up to sixteen
// sequences) in two launches, four with adapters:
//   route   e_1..e_k of token t: its k largest logits, gates g_j (route_token)
//   UP      h_p = g_j silu(W1_e x_t) * (W3_e x_t)      of each pair p = (t, j)
//   DOWN    out_t = sum_j W2_e h_p
// and, where adapter l of token t stands beside the expert's matrices, W + s_l
// B_{l,e} A_{l,e} in place of each: u = s_l A_{l,e} v of every pair first (a
// launch before UP and one before DOWN), B_{l,e} u added to the sums.
//
// Bound by reading each chosen expert's three matrices once.  What that takes:
//  - Routing needs no launch: every workgroup of UP routes the tokens itself
//    (the logits are a few KB in L2) and then takes units of (expert, sixteen
//    columns of h) in turn.  Workgroup 0 writes the routing out.
//  - No sort and no gather: an expert has a token once at most, so the sixteen
//    columns of a matrix instruction are the sixteen tokens whatever the expert.
//    Columns of tokens without the expert repeat the row of one that has it
//    (no traffic) and are not stored.
//  - No combine: with the gate applied to h in fp32, before its only rounding,
//    the sum over a token's experts is a product whose K runs over all the
//    chosen experts' F, zeros standing in for the pairs that are not.  A
//    workgroup of DOWN owns sixteen columns of out, its waves share that K, and
//    their fp32 sums meet in LDS in wave order.
// h is rounded once to the type of the weights, as the layer's own H is; all
// sums are fp32 in a fixed order.
#include "few_tokens.h"
#include "frag.h"
#include "mok_internal.h"
#include "route_token.h"

namespace mok {
namespace {

constexpr int kUpWaves = 4;  // waves that share the K of a unit of UP
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

// Routing of tokens t0, t0 + step, ... by the calling wave, into LDS.
template <int EPL>
__device__ __forceinline__ void route_few(const FewTokens& a, int t0, int t1, int step, int32_t* idx, float* gate,
                                          int32_t* idx2, float* gate2, float* lse, float* graw) {
  for (int t = t0; t < t1; t += step) {
    const float* row = a.logits + (int64_t)t * a.E;
    if (a.gating == 0)
      route_token<EPL, false, false>(row, t, a.E, a.k, idx, gate, idx2, gate2, lse, nullptr, graw);
    else if (a.gating == kFewSigmoid)
      route_token<EPL, true, false>(row, t, a.E, a.k, idx, gate, idx2, gate2, lse, nullptr, graw);
    else if (a.gating == kFewRenorm)
      route_token<EPL, false, true>(row, t, a.E, a.k, idx, gate, idx2, gate2, lse, nullptr, graw);
    else
      route_token<EPL, true, true>(row, t, a.E, a.k, idx, gate, idx2, gate2, lse, nullptr, graw);
  }
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

// LDS of UP: idx, gate and the copies route_token writes [P] each, the waves'
// raw gates, then the tables.
__host__ __device__ inline size_t up_lds(int P, int slots) {
  return (size_t)P * 16 + kUpWaves * kFewSlots * 4 + (size_t)slots * 34 + 64;
}

template <int DT, int EPL>
__global__ __launch_bounds__(64 * kUpWaves) void few_up_kernel(FewTokens a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes, U = kUnroll;
  extern __shared__ __align__(16) char lds[];
  __shared__ f32x4_t red[2][kUpWaves - 1][2][64];
  __shared__ uint32_t bits[32];
  __shared__ int base[33];
  __shared__ float lse[16];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int i16 = lane & 15, g = lane >> 4;
  const int P = a.T * a.k, most = few_slots(P, a.E_loc);
  FewTables s;
  s.idx = reinterpret_cast<int32_t*>(lds);
  s.gate = reinterpret_cast<float*>(lds + 4 * P);
  float* graw = reinterpret_cast<float*>(lds + 16 * P) + w * kFewSlots;
  s.pair = reinterpret_cast<int16_t*>(lds + 16 * P + kUpWaves * kFewSlots * 4);
  s.expert = s.pair + 16 * most;
  route_few<EPL>(a, w, a.T, kUpWaves, s.idx, s.gate, reinterpret_cast<int32_t*>(lds + 8 * P),
                 reinterpret_cast<float*>(lds + 12 * P), lse, graw);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int p = tid; p < P; p += 64 * kUpWaves) {
      a.idx[p] = s.idx[p];
      a.gate[p] = s.gate[p];
    }
  build_slots(a, s, bits, base, 64 * kUpWaves);

  const int ntn = a.Fp / 16, total = s.nslots * ntn;
  const int full = a.d / STEP;                                    // whole K steps
  const int all = full / U;                                      // whole chunks: the waves take them in turn
  const int chunks = all > w ? (all - w + kUpWaves - 1) / kUpWaves : 0;
  const int64_t row_bytes = (int64_t)a.d * S;
  int flip = 0;
  for (int un = blockIdx.x; un < total; un += gridDim.x, flip ^= 1) {
    const int slot = un / ntn, n0 = (un - slot * ntn) * 16;
    const int e = __builtin_amdgcn_readfirstlane(s.expert[slot]);
    const int pair = s.pair[slot * 16 + i16];
    const uint64_t has = __ballot(pair >= 0);
    const int tx = pair >= 0 ? i16 : __ffsll((unsigned long long)has) - 1;  // a token that has the expert
    const int n = n0 + i16 < a.F ? n0 + i16 : a.F - 1;
    const int64_t at = ((int64_t)e * a.F + n) * row_bytes + (int64_t)(g * KE) * S;
    const char* p1 = (const char*)a.w[0] + at;
    const char* p3 = (const char*)a.w[1] + at;
    const char* px = (const char*)a.x + tx * row_bytes + (int64_t)(g * KE) * S;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    u32x4_t q1[2][U], q3[2][U], qx[2][U];
    auto load = [&](int buf, int c) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int o = (c + j) * STEP * S;
        q1[buf][j] = load16<DT>(p1 + o);
        q3[buf][j] = load16<DT>(p3 + o);
        qx[buf][j] = load16<DT>(px + o);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto mul = [&](int buf) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        acc[0] = mma<DT>(q1[buf][j], qx[buf][j], acc[0]);
        acc[1] = mma<DT>(q3[buf][j], qx[buf][j], acc[1]);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // Chunk c + 1 is in flight while chunk c is multiplied.  No load stands under
    // a condition (the last one is asked for again): behind a branch the compiler
    // can only wait for every load, and the ring would run empty at each turn.
    // And it may not move loads to their uses, where they save it registers.
    if (chunks) {
      load(0, w * U);
      int c = 0;
      for (; c + 2 <= chunks; c += 2) {
        load(1, ((c + 1) * kUpWaves + w) * U);
        mul(0);
        load(0, ((c + 2 < chunks ? c + 2 : chunks - 1) * kUpWaves + w) * U);
        mul(1);
      }
      if (c < chunks) mul(0);
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
      const int left = a.d - full * STEP - g * KE, o = full * STEP * S;
      const u32x4_t vx = load_part<DT>(px + o, left);
      acc[0] = mma<DT>(load_part<DT>(p1 + o, left), vx, acc[0]);
      acc[1] = mma<DT>(load_part<DT>(p3 + o, left), vx, acc[1]);
    }
    const int l = a.adapter && pair >= 0 ? adapter_of(a, i16) : -1;
    if (l >= 0) {  // wave w adds the adapter's share of row 4 g + w of the tile
      const int nr = n0 + 4 * g + w;
      if (nr < a.F)
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
        for (int i = 0; i < 4; ++i) {
          const float va = acc[0][i];
          hv[i] = n0 + 4 * g + i < a.F ? va * sigmoidf_(va) * acc[1][i] * gt : 0.f;
        }
        char* hp = (char*)a.h + ((int64_t)pair * a.Fp + n0 + 4 * g) * S;
        if constexpr (DT == 0)
          *reinterpret_cast<f32x4_t*>(hp) = f32x4_t{hv[0], hv[1], hv[2], hv[3]};
        else
          *reinterpret_cast<u32x2_t*>(hp) = u32x2_t{Elem<DT>::pack(hv[0], hv[1]), Elem<DT>::pack(hv[2], hv[3])};
      }
    }
  }
#endif
}

template <int DT, int NW, bool WHOLE>
__global__ __launch_bounds__(64 * NW) void few_down_kernel(FewTokens a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes, U = kUnroll;
  extern __shared__ __align__(16) char lds[];
  __shared__ f32x4_t red[NW][64];
  __shared__ uint32_t bits[32];
  __shared__ int base[33];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int i16 = lane & 15, g = lane >> 4;
  const int P = a.T * a.k, most = few_slots(P, a.E_loc);
  FewTables s;
  s.idx = reinterpret_cast<int32_t*>(lds);
  s.pair = reinterpret_cast<int16_t*>(lds + 4 * P);
  s.expert = s.pair + 16 * most;
  for (int p = tid; p < P; p += 64 * NW) s.idx[p] = a.idx[p];
  __syncthreads();
  build_slots(a, s, bits, base, 64 * NW);

  const int n0 = blockIdx.x * 16;
  const int n = n0 + i16 < a.d ? n0 + i16 : a.d - 1;
  const int64_t row_bytes = (int64_t)a.F * S;
  const int chunks = (a.F + STEP * U - 1) / (STEP * U);  // of one expert
  const int all = s.nslots * chunks;  // the waves take them in turn: what they read at a time is neighbouring
  const int mine = all > w ? (all - w + NW - 1) / NW : 0;
  const auto hrs = __builtin_amdgcn_make_buffer_rsrc(a.h, (short)0, (int)((int64_t)P * a.Fp * S), 0x00020000);
  // cursor of the next chunk to load; past the last one it stays on it
  const int skip_slots = NW / chunks, skip = NW - skip_slots * chunks;
  int slot = w / chunks, ch = w - slot * chunks;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  u32x4_t qw[2][U], qh[2][U];
  // WHOLE: F is a multiple of KE, a lane's 16 bytes lie in F or past it; a
  // lane past it reads the row's first bytes and zeros of h.
  auto load = [&](int buf) {
    const int e = __builtin_amdgcn_readfirstlane(s.expert[slot]);
    const int pair = s.pair[slot * 16 + i16];
    // a pair that is not: an offset past the buffer, which loads zeros
    const uint32_t hoff = pair >= 0 ? (uint32_t)(pair * a.Fp) * S : 0xC0000000u;
    const char* wp = (const char*)a.w[2] + ((int64_t)e * a.d + n) * row_bytes;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = (ch * U + j) * STEP + g * KE;
      if constexpr (WHOLE) qw[buf][j] = load16<DT>(wp + (k < a.F ? k : 0) * S);
      else qw[buf][j] = load_part<DT>(wp + k * S, k < a.F ? a.F - k : 0);
      const auto v = __builtin_amdgcn_raw_buffer_load_b128(hrs, k < a.F ? hoff + k * S : 0xC0000000u, 0, 0);
      qh[buf][j] = u32x4_t{(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]};
    }
    const bool wrap = ch + skip >= chunks;
    const int next = slot + skip_slots + wrap;
    ch = next < s.nslots ? ch + skip - (wrap ? chunks : 0) : ch;
    slot = next < s.nslots ? next : slot;
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mul = [&](int buf) {
#pragma unroll
    for (int j = 0; j < U; ++j) acc = mma<DT>(qw[buf][j], qh[buf][j], acc);
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
        const int p = i16 * a.k + j, el = s.idx[p] - a.eb;
        if (el < 0 || el >= a.E_loc) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + 4 * g + i < a.d)
            acc[i] += rank_dot<DT>((const char*)a.lora[2].B +
                                       (((int64_t)l * a.E_loc + el) * a.d + n0 + 4 * g + i) * r * S,
                                   a.u[2] + (int64_t)p * few_u_width(r), r);
      }
  }
  red[w][lane] = acc;
  __syncthreads();
  if (w == 0 && i16 < a.T) {
    f32x4_t v = red[0][lane];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += red[q][lane];
    const int64_t o = (int64_t)i16 * a.d + n0 + 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + 4 * g + i < a.d) {
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
  __shared__ int32_t idx[2][kFewSlots];
  __shared__ float gate[2][kFewSlots], graw[kFewSlots], lse[1];
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
      route_few<EPL>(one, 0, 1, 1, idx[0], gate[0], idx[1], gate[1], lse, graw);
    }
    __syncthreads();
    e = idx[0][j];
  }
  e -= a.eb;
  if (e < 0 || e >= a.E_loc) return;
  const int r = a.lora[m].r, rr = 4 * y + w, K = DOWN ? a.F : a.d;
  float* to = a.u[m] + (int64_t)p * few_u_width(r) + rr;
  float sum = 0.f;
  if (rr < r) {
    const char* v = DOWN ? (const char*)a.h + (int64_t)p * a.Fp * S : (const char*)a.x + (int64_t)t * K * S;
    const char* row = (const char*)a.lora[m].A + (((int64_t)l * a.E_loc + e) * r + rr) * K * S;
#pragma unroll 4
    for (int c = lane * KE; c < K; c += 64 * KE) {
      float fa[KE], fv[KE];
      widen<DT>(load_part<DT>(row + (int64_t)c * S, K - c), fa);
      widen<DT>(load_part<DT>(v + (int64_t)c * S, K - c), fv);
#pragma unroll
      for (int i = 0; i < KE; ++i) sum = fmaf(fa[i], fv[i], sum);
    }
    sum = wave_sum(sum) * (a.lora[m].scale ? a.lora[m].scale[l] : 1.f);
  }
  if (lane == 0) *to = sum;
#endif
}

template <int DT, int EPL> hipError_t run(const FewTokens& a, hipStream_t s) {
  const int P = a.T * a.k, slots = few_slots(P, a.E_loc);
  int ranks = 0;
  for (int m = 0; m < 2; ++m)
    if (a.lora[m].A) ranks += few_u_width(a.lora[m].r) / 4;
  if (a.adapter && ranks)
    hipLaunchKernelGGL((few_rank_kernel<DT, EPL, false>), dim3(P, ranks), dim3(256), 0, s, a);
  static const int per_cu = [] {
    int n = 0;
    if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, few_up_kernel<DT, EPL>, 64 * kUpWaves, 8192) != hipSuccess ||
        n < 1)
      n = 1;
    return n;
  }();
  const int64_t units = (int64_t)slots * (a.Fp / 16), cap = (int64_t)kNumCUs * per_cu;
  hipLaunchKernelGGL((few_up_kernel<DT, EPL>), dim3((unsigned)(units < cap ? units : cap)), dim3(64 * kUpWaves),
                     up_lds(P, slots), s, a);
  if (a.adapter && a.lora[2].A)
    hipLaunchKernelGGL((few_rank_kernel<DT, EPL, true>), dim3(P, few_u_width(a.lora[2].r) / 4), dim3(256), 0, s, a);
  const size_t lds = (size_t)P * 4 + (size_t)slots * 34 + 64;
  if (a.F % kFragElems<DT> == 0)
    hipLaunchKernelGGL((few_down_kernel<DT, 16, true>), dim3((a.d + 15) / 16), dim3(1024), lds, s, a);
  else
    hipLaunchKernelGGL((few_down_kernel<DT, 16, false>), dim3((a.d + 15) / 16), dim3(1024), lds, s, a);
  return hipGetLastError();
}

template <int DT> hipError_t run_e(const FewTokens& a, hipStream_t s) {
  return a.E <= 128 ? run<DT, 2>(a, s) : a.E <= 256 ? run<DT, 4>(a, s) : run<DT, 16>(a, s);
}

}  // namespace

hipError_t launch_few_tokens(const FewTokens& a, hipStream_t s) {
  return a.dtype == 0 ? run_e<0>(a, s) : a.dtype == 1 ? run_e<1>(a, s) : run_e<2>(a, s);
}

}  // namespace mok
