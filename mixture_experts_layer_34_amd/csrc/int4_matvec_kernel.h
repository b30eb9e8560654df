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
// is rounded.  The two sums cancel in 16 + z, so the fp32 error goes with
// s sum_k |x_k| (32 + q + z) 2^-24 and not with the weights: a code equal to its
// zero point leaves some too.  For x of one magnitude that is log2(32 / |q - z|)
// bits of 24, far below the rounding of the 16-bit result; an x far above the
// others shows in fp16 (6e4 on weights of 0 among x of 1, K 4096: the mean error
// 0.066 -> 0.10 to 0.15 scales, results of 380 scales; with 1000, and in bf16 with
// either, unchanged).
//
// v_mfma_f32_16x16x32: A = the tile's rows of x (lane: row lane % 16, K
// 8 (lane / 16) + i), B = weight rows (lane: n = lane % 16, same K), result:
// n = lane % 16, MFMA rows 4 (lane / 16) + i.  A lane loads 16 bytes of one
// weight row (32 codes; its wave 64 bytes of 16 rows, K 128 of them, a chunk):
// lane quarter g then holds K [32 g, 32 g + 32) and a step of the MFMA would
// mix four groups of 32, so the 4 x 4 words of the four quarters are
// transposed by lane swaps (one per word).  The eight codes of a word come out
// as the pairs (0,4) (1,5) (2,6) (3,7); x is put in the same order.
//
// Tile row r sits on MFMA row 4 (r % 4) + r / 4 % 4.  In tiles of four rows
// the quad of MFMA rows 4 r .. 4 r + 3 belongs to row r, its lanes holding x
// of the chunk's steps 0 .. 3: step st's result st is the product of step st
// with itself (the others are products of unlike steps, and dropped), so one
// load of x serves the four steps.
//
// A workgroup takes one (row tile, 16 NG NW weight rows) unit.  Its waves lie
// side by side along N, sharing the tile's x through LDS (a lane's own load of
// x touches sixteen rows, as many cache lines as its codes: with those loads
// straight from cache 128 experts' gate / up of 128 tokens took 233 us, 178
// through LDS, against 156 for the codes alone), or split K where there are
// too few units, their fp32 sums then meeting in LDS, added in wave order: the
// same bits on every run.
//
// Measured: gate / up of 128 experts (d 4096, F 1536) 171 us for 128 tokens
// (groups of 128; 4.9 TB/s of codes and scales), 129 us for 16 tokens (82
// experts, groups of 32 with zero points; 4.8 TB/s), 16.5 us for one (8
// experts; 3.1 TB/s, 6 us of it the launch and the first loads).  A ring of
// eight chunks is level at best and loses up to 37 % (one token's down product
// 11.3 -> 12.0, 8 experts' with 128 rows 46.8 -> 64 us); non-temporal loads of
// the codes gave nothing.  Past sixteen rows the vector units taking the codes
// apart are the bound, once for each tile of rows: 64 rows on one matrix (8192
// x 4096) 18.4 us where four rows take 9.2.
#pragma once
#include "elem.h"
#include "int4_rules.h"
#include "pair_ops.h"

namespace mok {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
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
  __device__ __forceinline__ static void place(uint32_t w, uint32_t mask, uint32_t sixteen, uint32_t (&d)[4]) {
    d[0] = ((w << 3) & mask) | sixteen;
    d[1] = ((w >> 1) & mask) | sixteen;
    d[2] = ((w >> 5) & mask) | sixteen;
    d[3] = ((w >> 9) & mask) | sixteen;
  }
  __device__ __forceinline__ static f32x4_t mfma(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, (u32x4_t{a[0], a[1], a[2], a[3]})),
                                                   __builtin_bit_cast(bf16x8_t, (u32x4_t{b[0], b[1], b[2], b[3]})), c,
                                                   0, 0, 0);
  }
};
template <> struct Mma<kF16> {
  static constexpr uint32_t kMask = 0x03C003C0u, kSixteen = 0x4C004C00u, kOnes = 0x3C003C00u;
  __device__ __forceinline__ static void place(uint32_t w, uint32_t mask, uint32_t sixteen, uint32_t (&d)[4]) {
    d[0] = ((w << 6) & mask) | sixteen;
    d[1] = ((w << 2) & mask) | sixteen;
    d[2] = ((w >> 2) & mask) | sixteen;
    d[3] = ((w >> 6) & mask) | sixteen;
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

// The dword v of lane quarter q in every quarter, for q = 0..3.
__device__ __forceinline__ void spread_quarters(uint32_t v, uint32_t (&o)[4]) {
  const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  o[0] = a[0];
  o[1] = a[1];
  o[2] = b[0];
  o[3] = b[1];
}

// NM matrices (a pair for SwiGLU), NG groups of 16 weight rows of each, tiles
// of RT rows, groups of GS; of a workgroup's waves KS split K and NW lie side
// by side along N; x is staged SCH chunks at a time; WHOLE: K is a whole number
// of chunks, whose scales and zeros are then one aligned access.
//
// The loop's loads, and what first takes their results, are free of branches
// (a load that is not wanted is sent past its buffer's end): where a load may
// or may not be outstanding, the compiler can no longer count those in flight
// and waits for all of them, which empties the ring once a round.
//
// A single matrix in thirty-twos whose waves do not split K is held to 128
// registers, two workgroups a compute unit (20480 x 4096, groups of 32, 64 rows
// 57.5 -> 47.3 us, nothing spilled); the others either fit or spill for it (a
// pair in sixteens loses 2 to 20 %).
template <int DT, int NM, int NG, int RT, int GS, int KS, int NW, int SCH, bool WHOLE>
__global__ __launch_bounds__(64 * KS * NW, RT == 32 && NM == 1 && KS == 1 ? 4 : 1)
void int4_matvec_kernel(Int4Args a, const int32_t* __restrict__ offsets, const int32_t* __restrict__ pair_of_row) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NB = NM * NG;
  constexpr int NSC = kChunk / GS;          // groups in a chunk
  constexpr int SW = NSC > 2 ? 2 : 1;       // dwords of a chunk's scales of one weight row
  constexpr bool QUAD = RT == 4;            // a tile row on each quad of MFMA rows
  constexpr int MT = QUAD ? 1 : RT / 16;    // MFMA tiles of rows
  constexpr int IR = QUAD ? 1 : 4;          // results of a lane that hold rows
  constexpr int JC = SCH / KS;              // chunks of a stage that are this wave's
  constexpr int XROW = SCH * 256 + 16;      // bytes of a staged row (+16: no bank conflicts)
  constexpr int XP = SCH * 16;              // 16-byte pieces of a staged row
  constexpr int NT = 64 * KS * NW;
  constexpr int XA = (RT * XP + NT - 1) / NT;  // pieces each thread stages
  constexpr int RING = 4;                   // chunks of codes in registers
  static_assert(JC >= 1 && JC * KS == SCH && (JC == 1 || JC % 2 == 0), "every wave has chunks of each stage");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kr = wave / NW, nw = wave % NW;
  const int n16 = lane & 15, g4 = lane >> 4;
  // constants kept in registers: an and-or takes one operand of another kind only
  uint32_t mask = Mma<DT>::kMask, sixteen = Mma<DT>::kSixteen;
  asm("" : "+v"(mask), "+v"(sixteen));
  const int N = a.N, K = a.K, G = K / GS, E_loc = a.E_loc;
  constexpr int NU = 16 * NG * NW;          // weight rows of a unit
  const int ntn = (N + NU - 1) / NU;
  __shared__ __align__(16) uint8_t xs[2][RT * XROW];
  __shared__ f32x4_t red[KS > 1 ? (KS - 1) * NW * MT * NB * 64 : 1];

  extern __shared__ int32_t tp[];           // [E_loc + 1] tiles of the experts before e
  int32_t *s_row = tp + E_loc + 1, *s_end = s_row + E_loc;  // and each one's rows

  if (offsets) {
    __shared__ int32_t wsum[KS * NW];
    int carry = 0;
    for (int e0 = 0; e0 < E_loc; e0 += NT) {
      const int e = e0 + tid;
      int n = 0;
      if (e < E_loc) {
        const RowRange r = cut_rows(offsets[a.eb + e], offsets[a.eb + e + 1], a.rows);
        n = (r.end - r.begin + RT - 1) / RT;
        s_row[e] = r.begin;
        s_end[e] = r.end;
      }
      const int s = wave_prefix(n);
      if (lane == 63) wsum[wave] = s;
      __syncthreads();
      int base = carry;
#pragma unroll
      for (int q = 0; q < KS * NW; ++q) {
        base += q < wave ? wsum[q] : 0;
        carry += wsum[q];
      }
      if (e < E_loc) tp[e] = base + s - n;
      __syncthreads();
    }
    if (tid == 0) tp[E_loc] = carry;
  } else if (tid == 0) {
    tp[0] = 0;
    tp[1] = (a.rows + RT - 1) / RT;
    s_row[0] = 0;
    s_end[0] = a.rows;
  }
  __syncthreads();
  // a sorted map's tiles are no more than this; overlapping offsets' are cut
  const int most = (a.rows + RT - 1) / RT + min(E_loc, a.rows);
  const int total = min(__builtin_amdgcn_readfirstlane(tp[E_loc]), most) * ntn;

  const int nch = (K + kChunk - 1) / kChunk;
  const int nst = (nch + SCH - 1) / SCH, nloc = nst * JC;  // stages, this wave's chunks
  // this wave's i-th chunk
  auto chunk_of = [&](int i) { return (i / JC) * SCH + kr * JC + i % JC; };
  const bool has_zeros = a.zeros[0] != nullptr;
  const uint32_t zbias = has_zeros ? 0x10101010u : 0x18181818u;  // 16 + z byte by byte, z = 8 without zeros
  const rsrc_t rx = buffer(a.x, (int64_t)a.x_rows * K * 2);
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int q = u / ntn, n0 = (u % ntn) * NU + 16 * NG * nw;
    // the expert of tile q, the last one whose tiles start at or before it: 64
    // prefixes at a time, every share'th and then those of the share
    int lo = 0;
    if (E_loc > 1) {
      const int share = (E_loc + 63) / 64;
      lo = share * (__popcll(__ballot(lane * share < E_loc && tp[min(lane * share, E_loc)] <= q)) - 1);
      if (share > 1) lo += __popcll(__ballot(lane < share && lo + lane < E_loc && tp[min(lo + lane, E_loc)] <= q)) - 1;
    }
    const int row0 = __builtin_amdgcn_readfirstlane(s_row[lo] + (q - tp[lo]) * RT);
    const int nrow = min(__builtin_amdgcn_readfirstlane(s_end[lo]) - row0, RT);

    const int64_t wrow = (int64_t)lo * N + n0;
    rsrc_t rw[NM], rs[NM], rz[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      rw[m] = buffer(a.codes[m] + wrow * (K / 2), (int64_t)(N - n0) * (K / 2));
      rs[m] = buffer((const uint16_t*)a.scales[m] + wrow * G, (int64_t)(N - n0) * G * 2);
      rz[m] = buffer(has_zeros ? a.zeros[m] + wrow * G : nullptr, has_zeros ? (int64_t)(N - n0) * G : 0);
    }

    // A ring of chunks of codes, all but two of them on their way while two (a
    // whole cache line of each weight row) are multiplied.  Loads past K read
    // zeros.
    u32x4_t wv[RING][NB];
    uint32_t sv[NB][SW], zv[NB];  // of four chunks, lane quarter q holding chunk q's
    auto load_codes = [&](int buf, int i) {
      const int k = chunk_of(i) * kChunk + 32 * g4;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        wv[buf][b] = load16(rw[b / NG],
                            i < nloc && k < K ? (uint32_t)((16 * (b % NG) + n16) * (K / 2) + k / 2) : kNowhere);
    };
    auto load_scales = [&](int i0) {
      const int c = chunk_of(i0 + g4);
      const bool in_c = i0 + g4 < nloc && c < nch;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int row = (16 * (b % NG) + n16) * G;
        const rsrc_t r = rs[b / NG], z = rz[b / NG];
        if constexpr (WHOLE) {
          const uint32_t at = in_c ? (uint32_t)(row + c * NSC) : kNowhere;
          const uint32_t o = in_c ? 2 * at : kNowhere;
          if constexpr (NSC == 4) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0);
            sv[b][0] = v[0];
            sv[b][SW - 1] = v[1];
            zv[b] = __builtin_amdgcn_raw_buffer_load_b32(z, at, 0, 0);
          } else if constexpr (NSC == 2) {
            sv[b][0] = __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
            zv[b] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(z, at, 0, 0);
          } else {
            sv[b][0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0);
            zv[b] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(z, at, 0, 0);
          }
        } else {
#pragma unroll
          for (int w = 0; w < SW; ++w) sv[b][w] = 0;
          zv[b] = 0;
#pragma unroll
          for (int i = 0; i < NSC; ++i) {
            const int gi = c * NSC + i;
            const bool in = in_c && gi < G;
            const uint32_t v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, in ? 2 * (row + gi) : kNowhere, 0, 0);
            sv[b][i / 2] |= v << (16 * (i % 2));
            const uint8_t zi = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(z, in ? row + gi : kNowhere, 0, 0);
            zv[b] |= (uint32_t)zi << (8 * i);
          }
        }
      }
    };
#pragma unroll
    for (int i = 0; i < RING - 2; ++i) load_codes(i, i);
    load_scales(0);
    // x by stages of SCH chunks through LDS: a wave takes 64 pieces of 16
    // bytes of one row at a time, puts them in the codes' order and the row
    // where the MFMA takes it.  Rows past the tile's are zeros.
    auto row_at = [&](int i) { return (i * (KS * NW) + wave) * 64 / XP; };
    auto piece_at = [&](int i) { return (i * (KS * NW) + wave) * 64 % XP + lane; };
    uint32_t xo[XA];
#pragma unroll
    for (int i = 0; i < XA; ++i) {
      const int r = row_at(i);
      int src = -1;
      if (r < nrow) {
        src = row0 + r;
        if (pair_of_row) {
          const int p = pair_of_row[src];
          src = p < 0 ? -1 : (int)((uint32_t)p / (uint32_t)a.k);
        }
      }
      src = __builtin_amdgcn_readfirstlane(src);
      xo[i] = src >= 0 && src < a.x_rows ? (uint32_t)src * (uint32_t)(K * 2) : kNowhere;
    }
    u32x4_t xr[XA];
    auto load_x = [&](int st) {
#pragma unroll
      for (int i = 0; i < XA; ++i) {
        const int k = st * SCH * kChunk + 8 * piece_at(i);
        xr[i] = load16(rx, st < nst && k < K && xo[i] != kNowhere ? xo[i] + 2 * k : kNowhere);
      }
    };
    auto store_x = [&](int buf) {
#pragma unroll
      for (int i = 0; i < XA; ++i) {
        const int r = row_at(i);
        // MFMA row of tile row r: 4 (r % 4) + r / 4 % 4 within its sixteen
        const int p = QUAD ? r : (r & ~15) + 4 * (r & 3) + ((r >> 2) & 3);
        uint32_t d[4];
        order_like_codes(xr[i], d);
        *reinterpret_cast<u32x4_t*>(&xs[buf][p * XROW + 16 * piece_at(i)]) = u32x4_t{d[0], d[1], d[2], d[3]};
      }
    };
    load_x(0);
    store_x(0);
    __syncthreads();

    f32x4_t tot[MT][NB];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < NB; ++b) tot[m][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    const uint32_t ones[4] = {Mma<DT>::kOnes, Mma<DT>::kOnes, Mma<DT>::kOnes, Mma<DT>::kOnes};
    int cur = 0;
    for (int i0 = 0; i0 < nloc; i0 += RING) {
      uint32_t sc[NB][SW][4], zc[NB][4];  // four chunks' scales and 16 + zeros, in every lane quarter
#pragma unroll
      for (int j = 0; j < RING; ++j) {
        if (j > 0 && j % JC == 0 && i0 + j >= nloc) break;  // whole stages
        if (j % 4 == 0) {
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int w = 0; w < SW; ++w) spread_quarters(sv[b][w], sc[b][w]);
            spread_quarters(zv[b] + zbias, zc[b]);
          }
          load_scales(i0 + j + 4);
        }
        if (j % JC == 0) load_x((i0 + j) / JC + 1);
        if (j % 2 == 0) {
          load_codes((j + RING - 2) % RING, i0 + j + RING - 2);
          load_codes((j + RING - 1) % RING, i0 + j + RING - 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (chunk_of(i0 + j) < nch) {
          // this lane's pieces of x: its MFMA row, K 32 st + 8 g4 of the chunk
          const int cs = kr * JC + j % JC;  // chunk of the stage
          const uint8_t* xb = &xs[cur][cs * 256 + 16 * g4];
          u32x4_t xq;
          if constexpr (QUAD) xq = *reinterpret_cast<const u32x4_t*>(xb + (n16 >> 2) * XROW + 64 * (n16 & 3));
#pragma unroll
          for (int b = 0; b < NB; ++b) transpose_quarters(wv[j][b]);
#pragma unroll
          for (int i = 0; i < NSC; ++i) {
            float sf[NB], zz[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const uint32_t sw = sc[b][i / 2][j % 4];
              sf[b] = i % 2 ? Elem<DT>::hi(sw) : Elem<DT>::lo(sw);
              zz[b] = (float)((zc[b][j % 4] >> (8 * i)) & 255u);
            }
            constexpr int GST = 4 / NSC;  // MFMA steps of a group
            const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
            f32x4_t ax[MT], aw[MT][NB];
#pragma unroll
            for (int st = i * GST; st < (i + 1) * GST; ++st) {
              const bool first = QUAD || st == i * GST;
              uint32_t wd[NB][4];
#pragma unroll
              for (int b = 0; b < NB; ++b) Mma<DT>::place(wv[j][b][st], mask, sixteen, wd[b]);
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                if constexpr (!QUAD) xq = *reinterpret_cast<const u32x4_t*>(xb + (16 * m + n16) * XROW + 64 * st);
                const uint32_t xd[4] = {xq[0], xq[1], xq[2], xq[3]};
                ax[m] = Mma<DT>::mfma(xd, ones, first ? zero : ax[m]);
#pragma unroll
                for (int b = 0; b < NB; ++b) aw[m][b] = Mma<DT>::mfma(xd, wd[b], first ? zero : aw[m][b]);
              }
              if constexpr (QUAD) {
                // the lanes of a quad hold x of the steps 0..3: result st is step st's
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  tot[0][b][0] = fmaf(sf[b], fmaf(-zz[b], ax[0][st], aw[0][b][st]), tot[0][b][0]);
              }
            }
            if constexpr (!QUAD) {
#pragma unroll
              for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    tot[m][b][e] = fmaf(sf[b], fmaf(-zz[b], ax[m][e], aw[m][b][e]), tot[m][b][e]);
              }
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (j % JC == JC - 1) {  // the next stage of x is in place before anyone reads it
          if (i0 + j + 1 < nloc) store_x(cur ^ 1);
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
          cur ^= 1;
        }
      }
    }

    // the sums of the waves that split K, in wave order
    if (KS > 1) {
      if (kr > 0)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int b = 0; b < NB; ++b) red[((((kr - 1) * NW + nw) * MT + m) * NB + b) * 64 + lane] = tot[m][b];
      __syncthreads();
    }
    if (kr == 0) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int w = 0; w < KS - 1; ++w)
#pragma unroll
          for (int b = 0; b < NB; ++b) tot[m][b] += red[(((w * NW + nw) * MT + m) * NB + b) * 64 + lane];
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          const int n = n0 + 16 * gi + n16;
#pragma unroll
          for (int e = 0; e < IR; ++e) {
            const int r = 16 * m + 4 * e + g4;  // MFMA row 4 g4 + e holds tile row 4 e + g4 (QUAD: g4)
            if (r < nrow && n < N) {
              const float p = tot[m][gi][e];
              const float v = NM == 2 ? p * sigmoidf_(p) * tot[m][NB - NG + gi][e] : p;
              ((uint16_t*)a.out)[(int64_t)(row0 + r) * N + n] = (uint16_t)Elem<DT>::pack(v, 0.f);
            }
          }
        }
      }
    }
    // the stage's last barrier lets the next unit stage x; with a split K the
    // sums have to be read before they are written again, which that unit's
    // barriers see to
  }
#endif
}

// One configuration's launch (int4_rules.h says which).
template <int DT> struct Launch {
  hipStream_t s;
  template <int NM, int NG, int RT, int GS, int KS, int NW, int SCH, bool WHOLE>
  hipError_t run(const Int4Args& a) const {
    constexpr int64_t NU = 16 * NG * NW;
    const int64_t ntn = (a.N + NU - 1) / NU;
    const int64_t tiles = (a.rows + RT - 1) / RT + (a.offsets ? (a.E_loc < a.rows ? a.E_loc : a.rows) : 0);
    const int64_t units = tiles * ntn;
    if (units == 0) return hipSuccess;
    // a share's expected units twice (workgroups take what is over in turn): those
    // of the whole map would find none, up to 5 us of them (two tokens' down
    // product, 32 of 256 experts 12.4 -> 7.4 us)
    const int64_t local = local_rows(a);
    const int64_t twice = 2 * ((local + RT - 1) / RT + (a.E_loc < local ? a.E_loc : local)) * ntn;
    const int64_t some = twice > 1024 ? twice : 1024, most = units < some ? units : some;
    const unsigned grid = (unsigned)(most < 65536 ? most : 65536);
    hipLaunchKernelGGL((int4_matvec_kernel<DT, NM, NG, RT, GS, KS, NW, SCH, WHOLE>), dim3(grid), dim3(64 * KS * NW),
                       (3 * a.E_loc + 1) * sizeof(int32_t), s, a, a.offsets, a.pair_of_row);
    return hipGetLastError();
  }
};

}  // namespace

}  // namespace mok
