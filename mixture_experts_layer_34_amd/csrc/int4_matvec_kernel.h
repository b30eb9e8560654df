// Expert products with 4-bit integer weights and group scales, for decode
// steps (few rows per expert): with W[n, k] = s[n, k / g] (q[n, k] - z[n, k / g]),
//   out_r = W_e x_r,  or with a pair of matrices  silu(W_e x_r) * (W'_e x_r),
// over the rows of each expert (the layer's expert products in the form of
// the decode kernel that fluidifia.com, "Cursor ouvre MoK, un mégakernel qui
// accélère l'entraînement MoE", section "Quand la communication devient le
// vrai problème", names as earlier work).  Bound by reading the codes once.
//
// The matrix cores take 16-bit floats, so codes become floats exactly: with c
// the code placed just below the exponent of 16, the bits of 16 are 16 + q
// (bf16 0x4180 | q << 3, fp16 0x4c00 | q << 6), two codes at a time by a shift
// and an and-or.  Inside one group of g
//   sum_k x_k W[n, k] = s (sum_k x_k (16 + q) - (16 + z) sum_k x_k),
// where both sums are fp32 MFMA accumulations (the second against a matrix of
// ones, once for all n) and the scale is applied to the fp32 result: no weight
// is rounded.  The offset 16 costs at most log2(32 / |q - z|) bits of the
// fp32 sum, far below the rounding of the 16-bit result.
//
// v_mfma_f32_16x16x32: A = the tile's rows of x (lane: row lane % 16, K
// 8 (lane / 16) + i), B = weight rows (lane: n = lane % 16, same K), result:
// n = lane % 16, MFMA rows 4 (lane / 16) + i.  Tile row r sits on MFMA row
// 4 (r % 4) + r / 4, so that four rows fill only i = 0.  A lane loads 16 bytes
// of one weight row (32 codes; its wave 64 bytes of 16 rows, K 128 of them):
// lane quarter g then holds K [32 g, 32 g + 32) and a step of the MFMA would
// mix four groups of 32, so the 4 x 4 words of the four quarters are
// transposed by lane swaps (two per pair of words).  The eight codes of a word
// come out as the pairs (0,4) (1,5) (2,6) (3,7); x is put in the same order.
//
// A workgroup takes one (row tile, 16 NG weight rows) unit; its waves split K
// and their fp32 sums meet in LDS, added in wave order: the same bits on every
// run.
#pragma once
#include "elem.h"
#include "int4_matvec.h"
#include "pair_ops.h"

namespace mok {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kChunk = 128;  // K per round: 16 bytes of codes a lane
constexpr int kMaxExperts = 1024;
constexpr uint32_t kNowhere = 0x80000000u;  // an offset past every buffer: reads as zero

__device__ __forceinline__ rsrc_t buffer(const void* p, int64_t bytes) {
  const uint32_t n = bytes < 0 ? 0u : bytes > 0x7FFFFFFFll ? 0x7FFFFFFFu : (uint32_t)bytes;
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, n, 0x00020000);
}
__device__ __forceinline__ u32x4_t load16(rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

template <int DT> struct Mma;
template <> struct Mma<kBF16> {
  static constexpr uint32_t kMask = 0x00780078u, kSixteen = 0x41804180u, kOnes = 0x3F803F80u;
  __device__ __forceinline__ static void place(uint32_t w, uint32_t (&d)[4]) {
    d[0] = ((w << 3) & kMask) | kSixteen;
    d[1] = ((w >> 1) & kMask) | kSixteen;
    d[2] = ((w >> 5) & kMask) | kSixteen;
    d[3] = ((w >> 9) & kMask) | kSixteen;
  }
  __device__ __forceinline__ static f32x4_t mfma(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, (u32x4_t{a[0], a[1], a[2], a[3]})),
                                                   __builtin_bit_cast(bf16x8_t, (u32x4_t{b[0], b[1], b[2], b[3]})), c,
                                                   0, 0, 0);
  }
};
template <> struct Mma<kF16> {
  static constexpr uint32_t kMask = 0x03C003C0u, kSixteen = 0x4C004C00u, kOnes = 0x3C003C00u;
  __device__ __forceinline__ static void place(uint32_t w, uint32_t (&d)[4]) {
    d[0] = ((w << 6) & kMask) | kSixteen;
    d[1] = ((w << 2) & kMask) | kSixteen;
    d[2] = ((w >> 2) & kMask) | kSixteen;
    d[3] = ((w >> 6) & kMask) | kSixteen;
  }
  __device__ __forceinline__ static f32x4_t mfma(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, (u32x4_t{a[0], a[1], a[2], a[3]})),
                                                  __builtin_bit_cast(f16x8_t, (u32x4_t{b[0], b[1], b[2], b[3]})), c,
                                                  0, 0, 0);
  }
};

// Words j = 0..3 of lane quarters g = 0..3 transposed: word j of quarter g
// becomes word g of quarter j's.
__device__ __forceinline__ void transpose_quarters(u32x4_t& w) {
  const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  w = u32x4_t{c[0], d[0], c[1], d[1]};
}

// Elements (0..7) of x as the pairs (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ void order_like_codes(const u32x4_t& v, uint32_t (&d)[4]) {
  d[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
  d[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
  d[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
  d[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
}

// NM matrices (a pair for SwiGLU), MT tiles of 16 rows, groups of GS.
template <int DT, int NM, int MT, int GS>
__global__ __launch_bounds__(512) void int4_matvec_kernel(Int4Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NSC = kChunk / GS;   // groups in a chunk
  constexpr int RT = 16 * MT;        // rows per tile
  const int tid = threadIdx.x, lane = tid & 63, kr = __builtin_amdgcn_readfirstlane(tid >> 6), KS = blockDim.x >> 6;
  const int n16 = lane & 15, g4 = lane >> 4;
  const int N = a.N, K = a.K, G = K / GS, E_loc = a.E_loc;
  const int ntn = (N + 15) / 16;
  extern __shared__ f32x4_t red[];  // [KS - 1][MT][NM][64]
  __shared__ int32_t tp[kMaxExperts + 1];  // tiles of the experts before e

  // tiles of each expert's rows, and their prefix over the experts
  if (a.offsets) {
    __shared__ int32_t wsum[8];
    int carry = 0;
    for (int e0 = 0; e0 < E_loc; e0 += blockDim.x) {
      const int e = e0 + tid;
      int n = 0;
      if (e < E_loc) {
        const int lo = max(a.offsets[a.eb + e], 0), hi = min(a.offsets[a.eb + e + 1], a.rows);
        n = hi > lo ? (hi - lo + RT - 1) / RT : 0;
      }
      int s = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(s, o, 64);
        if (lane >= o) s += u;
      }
      if (lane == 63) wsum[kr] = s;
      __syncthreads();
      int base = carry;
      for (int q = 0; q < KS; ++q) {
        base += q < kr ? wsum[q] : 0;
        carry += wsum[q];
      }
      if (e < E_loc) tp[e] = base + s - n;
      __syncthreads();
    }
    if (tid == 0) tp[E_loc] = carry;
  } else if (tid == 0) {
    tp[0] = 0;
    tp[1] = (a.rows + RT - 1) / RT;
  }
  __syncthreads();
  const int64_t total = (int64_t)tp[E_loc] * ntn;

  const int nch = (K + kChunk - 1) / kChunk;
  const int c0 = nch * kr / KS, c1 = nch * (kr + 1) / KS;
  const rsrc_t rx = buffer(a.x, (int64_t)a.x_rows * K * 2);
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int q = (int)(u / ntn), n0 = (int)(u % ntn) * 16;
    int lo = 0, hi = E_loc - 1;
    while (lo < hi) {  // the expert of tile q
      const int mid = (lo + hi + 1) >> 1;
      if (tp[mid] <= q) lo = mid; else hi = mid - 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int first = a.offsets ? max(a.offsets[a.eb + lo], 0) : 0;
    const int last = a.offsets ? min(a.offsets[a.eb + lo + 1], a.rows) : a.rows;
    const int row0 = first + (q - tp[lo]) * RT;
    const int nrow = min(last - row0, RT);

    // this lane's x row (MFMA row lane % 16) and weight row n0 + lane % 16
    uint32_t xo[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = 16 * m + 4 * (n16 & 3) + (n16 >> 2);
      int64_t src = -1;
      if (r < nrow) src = a.pair_of_row ? (a.pair_of_row[row0 + r] >= 0 ? a.pair_of_row[row0 + r] / a.k : -1) : row0 + r;
      xo[m] = src >= 0 && src < a.x_rows ? (uint32_t)(src * K * 2) : kNowhere;
    }
    const int64_t wrow = (int64_t)lo * N + n0;
    rsrc_t rw[NM], rs[NM], rz[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      rw[m] = buffer(a.codes[m] + wrow * (K / 2), (int64_t)(N - n0) * (K / 2));
      rs[m] = buffer((const uint16_t*)a.scales[m] + wrow * G, (int64_t)(N - n0) * G * 2);
      rz[m] = buffer(a.zeros[m] ? a.zeros[m] + wrow * G : nullptr, a.zeros[m] ? (int64_t)(N - n0) * G : 0);
    }

    f32x4_t tot[MT][NM];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NM; ++b) tot[m][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c = c0; c < c1; ++c) {
      const int kq = c * kChunk + 32 * g4;  // the K range this lane loads
      u32x4_t wv[NM];
      uint32_t sv[NM][NSC], zv[NM][NSC];
#pragma unroll
      for (int b = 0; b < NM; ++b) {
        wv[b] = load16(rw[b], kq < K ? (uint32_t)(n16 * (K / 2) + kq / 2) : kNowhere);
#pragma unroll
        for (int i = 0; i < NSC; ++i) {
          const int gi = c * NSC + i;
          sv[b][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs[b], gi < G ? (n16 * G + gi) * 2 : kNowhere, 0, 0);
          zv[b][i] = a.zeros[b] ? (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rz[b], gi < G ? n16 * G + gi : kNowhere, 0, 0)
                                : 8;
        }
      }
      u32x4_t xv[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          const int k = c * kChunk + 32 * st + 8 * g4;
          xv[m][st] = load16(rx, k < K && xo[m] != kNowhere ? xo[m] + 2 * k : kNowhere);
        }
      uint32_t ones[4] = {Mma<DT>::kOnes, Mma<DT>::kOnes, Mma<DT>::kOnes, Mma<DT>::kOnes};
#pragma unroll
      for (int b = 0; b < NM; ++b) transpose_quarters(wv[b]);
#pragma unroll
      for (int i = 0; i < NSC; ++i) {
        f32x4_t ax[MT], aw[MT][NM];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          ax[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < NM; ++b) aw[m][b] = ax[m];
        }
#pragma unroll
        for (int st = i * (4 / NSC); st < (i + 1) * (4 / NSC); ++st) {
          uint32_t wd[NM][4];
#pragma unroll
          for (int b = 0; b < NM; ++b) Mma<DT>::place(wv[b][st], wd[b]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t xd[4];
            order_like_codes(xv[m][st], xd);
            ax[m] = Mma<DT>::mfma(xd, ones, ax[m]);
#pragma unroll
            for (int b = 0; b < NM; ++b) aw[m][b] = Mma<DT>::mfma(xd, wd[b], aw[m][b]);
          }
        }
#pragma unroll
        for (int b = 0; b < NM; ++b) {
          const float sc = Elem<DT>::lo(sv[b][i]), zz = 16.0f + (float)zv[b][i];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[m][b][e] = fmaf(sc, fmaf(-zz, ax[m][e], aw[m][b][e]), tot[m][b][e]);
        }
      }
    }

    // the waves' sums, in wave order
    if (kr > 0)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b = 0; b < NM; ++b) red[(((kr - 1) * MT + m) * NM + b) * 64 + lane] = tot[m][b];
    __syncthreads();
    if (kr == 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        for (int w = 0; w < KS - 1; ++w)
#pragma unroll
          for (int b = 0; b < NM; ++b) tot[m][b] += red[((w * MT + m) * NM + b) * 64 + lane];
        const int n = n0 + n16;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * m + 4 * e + g4;  // MFMA row 4 g4 + e holds tile row 4 e + g4
          if (r < nrow && n < N) {
            const float v = NM == 2 ? tot[m][0][e] * sigmoidf_(tot[m][0][e]) * tot[m][NM - 1][e] : tot[m][0][e];
            ((uint16_t*)a.out)[(int64_t)(row0 + r) * N + n] = (uint16_t)Elem<DT>::pack(v, 0.f);
          }
        }
      }
    }
    __syncthreads();  // the sums are read before the next unit writes them
  }
#endif
}

template <int DT, int NM, int MT, int GS> hipError_t run(const Int4Args& a, hipStream_t s) {
  constexpr int RT = 16 * MT;
  const int64_t ntn = (a.N + 15) / 16;
  const int64_t tiles = (a.rows + RT - 1) / RT + (a.offsets ? (a.E_loc < a.rows ? a.E_loc : a.rows) : 0);
  const int64_t units = tiles * ntn;
  if (units == 0) return hipSuccess;
  const int waves = 4;
  const unsigned grid = (unsigned)(units < 65536 ? units : 65536);
  hipLaunchKernelGGL((int4_matvec_kernel<DT, NM, MT, GS>), dim3(grid), dim3(64 * waves),
                     (size_t)(waves - 1) * MT * NM * 64 * sizeof(f32x4_t), s, a);
  return hipGetLastError();
}

template <int DT, int NM, int MT> hipError_t run_group(const Int4Args& a, hipStream_t s) {
  switch (a.group) {
    case 32: return run<DT, NM, MT, 32>(a, s);
    case 64: return run<DT, NM, MT, 64>(a, s);
    case 128: return run<DT, NM, MT, 128>(a, s);
  }
  return hipErrorInvalidValue;
}

template <int DT, int NM> hipError_t run_tile(const Int4Args& a, hipStream_t s) {
  return run_group<DT, NM, 1>(a, s);
}

template <int DT> hipError_t run_dtype(const Int4Args& a, hipStream_t s) {
  return a.pair ? run_tile<DT, 2>(a, s) : run_tile<DT, 1>(a, s);
}

}  // namespace

}  // namespace mok
