// Low-rank adapters of many requests beside a projection, forward and
// backward.  Rows are sorted by adapter (a pair map whose experts are the
// adapters), or are the experts' sorted rows with one adapter pair each:
//   u_q = A_g x_q,      out_q = y_q + s_g B_g u_q
//   du_q = B_g^T dout_q, dx_q = base_q + s_g A_g^T du_q,
//   dA_g = s_g sum_q du_q x_q^T,  dB_g = s_g sum_q dout_q u_q^T
// over the rows q of adapter g.
//
// All of it is bound by moving the rows once: with ranks of 8 to 128 beside
// widths of thousands the products are a few percent of what the matrix cores
// do in that time.  Four kernels:
//  - rank (u and du): a workgroup takes a tile of one adapter's rows, its waves
//    share K and meet in LDS; with few rows K is split over workgroups too, whose
//    fp32 parts the next kernel adds in order (no atomics).
//  - add (out and dx): the transposed product B u^T, so that a lane holds sixteen
//    neighbouring columns of one row: 128 bytes a row and wave, y in, out back.  A
//    wave keeps its 64 rows of B in registers and runs over its rows.  u enters
//    16-bit matrix instructions as a high and a low part (a K of 2 r), so that it
//    loses nothing next to out's own rounding.
//  - grad (dA and dB): K is the rows there.  v_mfma_f32_16x16x4 takes one value
//    of each operand a lane, so the j-th elements of sixteen lanes' 16-byte loads
//    are an operand as they are: no transposing, and u and du keep their 32 bits.
//  - prepare: A^T and B^T for the backward pass, which then runs the first two
//    kernels on them (du: rank with B^T; dx: add with A^T).
#include "frag.h"
#include "lora_rows.h"
#include "mok_internal.h"

namespace mok {
namespace {

struct Tile {
  int g, row0, row1;    // rows [row0, row1) of group g; g < 0: none
  int first, row_first; // the group's first tile and row
  int n;                // the group's tiles
};

__device__ __forceinline__ int cut(int v, int rows) { return v < 0 ? 0 : v > rows ? rows : v; }

// The t-th tile of mt rows, the groups' tiles counted one after the other.
__device__ __forceinline__ Tile find_tile(const LoraMap& m, int t, int mt) {
  const int lane = lane_id();
  int before = 0;
  for (int g0 = 0; g0 < m.G; g0 += 64) {
    const int g = g0 + lane;
    const int lo = cut(m.offsets[g < m.G ? g : m.G], m.rows);
    const int hi = cut(m.offsets[g < m.G ? g + 1 : m.G], m.rows);
    const int n = hi > lo ? (hi - lo + mt - 1) / mt : 0;
    const int to = wave_prefix(n) + before;
    const uint64_t hit = __ballot(t >= to - n && t < to);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int num = __builtin_amdgcn_readlane(n, l), first = __builtin_amdgcn_readlane(to, l) - num,
                a = __builtin_amdgcn_readlane(lo, l), b = __builtin_amdgcn_readlane(hi, l);
      const int row0 = a + (t - first) * mt;
      return Tile{g0 + l, row0, row0 + mt < b ? row0 + mt : b, first, a, num};
    }
    before = __builtin_amdgcn_readlane(to, 63);
  }
  return Tile{-1, 0, 0, 0, 0, 0};
}

// The token of a sorted row; -1: none.  No branch, so that several are in flight
// at once: without a map a word of the offsets is read in its place.
__device__ __forceinline__ int token_word(const LoraMap& m, int row) {
  return (m.pair_of_row ? m.pair_of_row : m.offsets)[m.pair_of_row ? row : 0];
}
__device__ __forceinline__ int token_in(const LoraMap& m, int row, int word) {
  return !m.pair_of_row ? row : word >= 0 && word < m.rows ? word : -1;
}
__device__ __forceinline__ int token_of(const LoraMap& m, int row) { return token_in(m, row, token_word(m, row)); }

// ------------------------------------------------------------------ rank
constexpr int kRankWaves = 4;

template <int DT, int RT, int M> __global__ __launch_bounds__(64 * kRankWaves) void lora_rank_kernel(LoraRank a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes;
  constexpr int U = RT >= 4 ? 1 : RT == 2 || M == 4 ? 2 : 4;  // K steps of a chunk
  __shared__ f32x4_t red[kRankWaves - 1][M][RT][64];
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const Tile t = find_tile(a.map, blockIdx.x, 16 * M);
  if (t.g < 0) return;
  const int full = a.K / STEP, steps = (a.K + STEP - 1) / STEP;
  // this workgroup's K steps, [s0, s1): its waves take chunks in turn, so that
  // what they read at a time is neighbouring
  const int s0 = (int)((int64_t)steps * blockIdx.y / a.splits), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / a.splits);
  const int ns = (s1 < full ? s1 : full) - s0;  // whole steps
  const int64_t at = (int64_t)(s0 * STEP + g4 * KE) * S;
  const char *px[M], *pa[RT];
  int tok[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int row = t.row0 + 16 * m + i16;
    tok[m] = token_of(a.map, row < t.row1 ? row : t.row1 - 1);
    px[m] = (const char*)a.in + (int64_t)(tok[m] < 0 ? 0 : tok[m]) * a.K * S + at;
  }
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    const int rr = 16 * q + i16 < a.r ? 16 * q + i16 : a.r - 1;
    pa[q] = (const char*)a.A + ((int64_t)t.g * a.r + rr) * a.K * S + at;
  }
  f32x4_t acc[M][RT];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[m][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t qx[2][U][M], qa[2][U][RT];
  auto load = [&](int buf, int j, int step) {
    const int o = step * STEP * S;
#pragma unroll
    for (int m = 0; m < M; ++m) qx[buf][j][m] = load16<DT>(px[m] + o);
#pragma unroll
    for (int q = 0; q < RT; ++q) qa[buf][j][q] = load16<DT>(pa[q] + o);
  };
  auto mul = [&](int buf, int j) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int q = 0; q < RT; ++q) acc[m][q] = mma<DT>(qa[buf][j][q], qx[buf][j][m], acc[m][q]);
  };
  // Chunk c + 1 is in flight while chunk c is multiplied.  No load stands under a
  // condition (the last one is asked for again): behind a branch the compiler
  // can only wait for every load, and the ring would run empty at each turn.  And
  // it may not move loads to their uses, where they save it registers.
  const int all = ns / U, chunks = all > w ? (all - w + kRankWaves - 1) / kRankWaves : 0;
  auto load_chunk = [&](int buf, int c) {
#pragma unroll
    for (int j = 0; j < U; ++j) load(buf, j, (c * kRankWaves + w) * U + j);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mul_chunk = [&](int buf) {
#pragma unroll
    for (int j = 0; j < U; ++j) mul(buf, j);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (chunks) {
    load_chunk(0, 0);
    int c = 0;
    for (; c + 2 <= chunks; c += 2) {
      load_chunk(1, c + 1);
      mul_chunk(0);
      load_chunk(0, c + 2 < chunks ? c + 2 : chunks - 1);
      mul_chunk(1);
    }
    if (c < chunks) mul_chunk(0);
  }
  // the steps that fill no chunk, a wave each, and the step that K ends in
  for (int i = all * U; i < ns; ++i)
    if (i % kRankWaves == w) {
      load(0, 0, i);
      mul(0, 0);
    }
  if (s1 > full && w == 0) {
    const int left = a.K - full * STEP - g4 * KE, o = (full - s0) * STEP * S;
#pragma unroll
    for (int m = 0; m < M; ++m) qx[0][0][m] = load_part<DT>(px[m] + o, left);
#pragma unroll
    for (int q = 0; q < RT; ++q) qa[0][0][q] = load_part<DT>(pa[q] + o, left);
    mul(0, 0);
  }
  if (w > 0)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int q = 0; q < RT; ++q) red[w - 1][m][q][lane] = acc[m][q];
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int row = t.row0 + 16 * m + i16;
    if (row >= t.row1) continue;
    float* to = a.part + ((int64_t)blockIdx.y * a.map.rows + row) * (16 * RT);
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      f32x4_t v = acc[m][q];
#pragma unroll
      for (int k = 0; k < kRankWaves - 1; ++k) v += red[k][m][q][lane];
      const int r0 = 16 * q + 4 * g4;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = tok[m] < 0 || r0 + i >= a.r ? 0.f : v[i];
      *reinterpret_cast<f32x4_t*>(to + r0) = v;
    }
  }
#endif
}

// ------------------------------------------------------------------ add
constexpr int kAddWaves = 4;
constexpr int kAddCols = 64 * kAddWaves;  // columns of a workgroup
constexpr int kBareTokens = 256;          // tokens a workgroup looks over for rows of no adapter

// Rows of no adapter: out = base, or 0.  A wave looks over kBareTokens / kAddWaves
// tokens at once.
template <int DT> __device__ __forceinline__ void bare_rows(const LoraAdd& a, int slab, int block) {
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, LPR = kAddCols / KE, RPW = 64 / LPR;
  constexpr int TOKENS = kBareTokens / kAddWaves;
  const int lane = lane_id(), w = wave_id();
  const int64_t t0 = (int64_t)block * kBareTokens + w * TOKENS;
  const int col = slab * kAddCols + (lane % LPR) * KE;
  bool bare = false;
  if (lane < TOKENS && t0 + lane < a.map.rows) {
    const int row = a.map.row_of_pair[t0 + lane];
    bare = row < 0 || row >= a.map.rows;
  }
  uint64_t left = __ballot(bare);
  while (left) {
    // the next RPW such rows, one for each LPR lanes
    int t = -1;
#pragma unroll
    for (int i = 0; i < RPW; ++i)
      if (left) {
        const int at = __ffsll((unsigned long long)left) - 1;
        left &= left - 1;
        t = lane / LPR == i ? at : t;
      }
    if (t < 0 || col >= a.N) continue;
    const int64_t at = ((t0 + t) * a.N + col) * S;
    const u32x4_t v = a.base ? load_part<DT>((const char*)a.base + at, a.N - col) : u32x4_t{0, 0, 0, 0};
    store_part<DT>((char*)a.out + at, v, a.N - col);
  }
}

// slabs: workgroups beside each other along N, each of kAddCols columns, the
// fastest in the grid (neighbours then write neighbouring bytes of the same rows).
// tiles: workgroups of a slab that take tiles of MT rows; those behind them look
// for rows of no adapter.
template <int DT, int RT, int MT>
__global__ __launch_bounds__(64 * kAddWaves) void lora_add_kernel(LoraAdd a, int slabs, int tiles) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, Q = 16 / KE;  // Q: accesses of a lane's sixteen columns
  constexpr int SUB = MT / 16, W = 16 * RT;
  const int slab = blockIdx.x % slabs, tile = blockIdx.x / slabs;
  if (tile >= tiles) {
    bare_rows<DT>(a, slab, tile - tiles);
    return;
  }
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const int base = slab * kAddCols + w * 64;
  const Tile t = find_tile(a.map, tile, MT);
  if (t.g < 0 || base >= a.N) return;
  const bool keeps = a.u && slab == 0 && w == 0;
  const bool whole = base + 64 <= a.N;  // every lane has all of its columns
  // 16-bit types: virtual K of 2 * 16 RT, the high parts, then the low ones
  auto rank_of = [&](int s) { const int c = 4 * s + g4; return DT == 0 ? 4 * c : 8 * (c % (2 * RT)); };
  // Columns: access j of a lane is KE neighbours from column base + 4 KE j + KE g4
  // on (64 bytes a row and access), results q = j KE / 4 + h its elements 4 h + 0..3.
  const char* rows_b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = base + 4 * KE * (4 * q / KE) + KE * (i16 >> 2) + 4 * q % KE + (i16 & 3);
    rows_b[q] = (const char*)a.B + ((int64_t)t.g * a.N + (n < a.N ? n : a.N - 1)) * a.r * S;
  }
  u32x4_t qb[4][RT];
  if (a.r % KE == 0) {  // no branch between the loads
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int s = 0; s < RT; ++s) {
        const int r0 = rank_of(s);
        const u32x4_t v = load16<DT>(rows_b[q] + (r0 < a.r ? r0 : 0) * S);
#pragma unroll
        for (int j = 0; j < 4; ++j) qb[q][s][j] = r0 < a.r ? v[j] : 0u;
      }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int s = 0; s < RT; ++s) {
        const int r0 = rank_of(s);
        qb[q][s] = load_part<DT>(rows_b[q] + r0 * S, r0 < a.r ? a.r - r0 : 0);
      }
  }
  const float scale = a.scale ? a.scale[t.g] : 1.f;
  const int col = base + KE * g4;
  int row[SUB], tok[SUB];
#pragma unroll
  for (int b = 0; b < SUB; ++b) {
    const int at = t.row0 + 16 * b + i16;
    row[b] = at < t.row1 ? at : t.row1 - 1;
    tok[b] = token_of(a.map, row[b]);
  }
  // all rows of the tile in flight at once
  u32x4_t y[SUB][Q];
#pragma unroll
  for (int b = 0; b < SUB; ++b) {
    const char* from = (const char*)a.base + ((int64_t)(tok[b] < 0 ? 0 : tok[b]) * a.N + col) * S;
    if (!a.base) {
#pragma unroll
      for (int j = 0; j < Q; ++j) y[b][j] = u32x4_t{0, 0, 0, 0};
    } else if (whole) {
#pragma unroll
      for (int j = 0; j < Q; ++j) y[b][j] = load16<DT>(from + 64 * j);
    } else {
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const int left = a.N - col - j * 4 * KE;
        y[b][j] = load_part<DT>(from + 64 * j, left < 0 ? 0 : left);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < SUB; ++b) {
    if (t.row0 + 16 * b >= t.row1) break;
    const bool live = t.row0 + 16 * b + i16 < t.row1 && tok[b] >= 0;
    float v[RT][KE];
    float big = 0.f;
#pragma unroll
    for (int s = 0; s < RT; ++s) {
      const int r0 = rank_of(s);
      const float* from = a.part + (int64_t)row[b] * W + r0;
#pragma unroll
      for (int j = 0; j < KE; j += 4) {
        f32x4_t sum = *reinterpret_cast<const f32x4_t*>(from + j);
#pragma unroll 4
        for (int p = 1; p < a.splits; ++p)
          sum += *reinterpret_cast<const f32x4_t*>(from + (int64_t)p * a.map.rows * W + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[s][j + i] = sum[i];
      }
      if (keeps && t.row0 + 16 * b + i16 < t.row1 && (DT == 0 || 4 * s + g4 < 2 * RT))
#pragma unroll
        for (int j = 0; j < KE; ++j)
          if (r0 + j < a.u_width) a.u[(int64_t)row[b] * a.u_width + r0 + j] = v[s][j];
#pragma unroll
      for (int j = 0; j < KE; ++j) {
        v[s][j] *= scale;
        big = fmaxf(big, fabsf(v[s][j]));
      }
    }
    float up = 1.f;  // fp16: the row's sums brought to [1, 2) by a power of two, exactly, and back at the end
    if constexpr (DT == 2) {
      big = fmaxf(big, __shfl_xor(big, 16, 64));
      big = fmaxf(big, __shfl_xor(big, 32, 64));
      const int e = big > 0.f && big < INFINITY ? (big < 0x1p-126f ? -126 : ilogbf(big)) : 0;
      up = ldexpf(1.f, e);
      const float down = ldexpf(1.f, -e);
#pragma unroll
      for (int s = 0; s < RT; ++s)
#pragma unroll
        for (int j = 0; j < KE; ++j) v[s][j] *= down;
    }
    f32x4_t acc[4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < RT; ++s) {
      u32x4_t f = narrow<DT>(v[s]);
      if constexpr (DT != 0) {
        float hi[KE];
        widen<DT>(f, hi);
#pragma unroll
        for (int j = 0; j < KE; ++j) hi[j] = v[s][j] - hi[j];
        const u32x4_t lo = narrow<DT>(hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = 4 * s + g4 < 2 * RT ? f[j] : lo[j];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = mma<DT>(qb[q][s], f, acc[q]);
    }
    if (!live) continue;
    char* to = (char*)a.out + ((int64_t)tok[b] * a.N + col) * S;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      float o[KE];
      widen<DT>(y[b][j], o);
#pragma unroll
      for (int i = 0; i < KE; ++i) o[i] = fmaf(acc[(j * KE + i) / 4][i % 4], up, o[i]);
      const u32x4_t r = narrow<DT>(o);
      if (whole) {
        store16<DT>(to + 64 * j, r);
      } else {
        const int left = a.N - col - j * 4 * KE;
        if (left > 0) store_part<DT>(to + 64 * j, r, left);
      }
    }
  }
#endif
}

// ------------------------------------------------------------------ grad
constexpr int kGradWaves = 4;

// Rows of a tile: enough tiles for three workgroups a compute unit (a compute
// unit takes no more than about 23 GB/s from HBM, so all of them have to be at
// work to the end), and no more, for a group of several tiles adds their sums.
int grad_rows(int rows, int K, int N, int cols) {
  const int64_t slabs = (K + cols - 1) / cols + (N + cols - 1) / cols;
  const int64_t n = (int64_t)rows * slabs / (3 * kNumCUs);
  return n < 128 ? 128 : n > (1 << 20) ? (1 << 20) : (int)((n + 127) / 128 * 128);
}

// Places of the tiles' sums that are still to be added: the first tiles of two
// groups of several tiles start more than a tile's height apart, and so do two
// later tiles; one place for each height's first tile and one for a later one.
__host__ __device__ inline int grad_places(int rows, int tile_rows) { return 2 * (rows / tile_rows + 1); }
__device__ __forceinline__ int64_t grad_place(const LoraGrad& a, const Tile& t, int row, int frags) {
  const int64_t unit = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  return (unit * grad_places(a.map.rows, a.tile_rows) + 2 * (row / a.tile_rows) + (row != t.row_first)) * frags * 64;
}

// A group's gradients from the sums of a wave: lane 16 g4 + i16 holds ranks
// 16 (q0 + q) + 4 g4 + 0..3 of column col + j.
template <int DT, int RT>
__device__ __forceinline__ void write_grad(const LoraGrad& a, int g, int mat, int q0, int at, int col,
                                           const f32x4_t (&acc)[RT][kFragElems<DT>]) {
  constexpr int KE = kFragElems<DT>;
  const int W = a.width[mat], g4 = lane_id() >> 4;
  if (at >= W) return;
  const float scale = a.scale ? a.scale[g] : 1.f;
  float* out = a.out[mat] + (int64_t)g * a.r * W;
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    const int r0 = 16 * (q0 + q) + 4 * g4;
    if (mat == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < a.r)
#pragma unroll
          for (int j = 0; j < KE; j += 4) {
            float* to = out + (int64_t)(r0 + i) * W + col + j;
            const f32x4_t v = f32x4_t{acc[q][j][i], acc[q][j + 1][i], acc[q][j + 2][i], acc[q][j + 3][i]} * scale;
            store_part<0>((char*)to, __builtin_bit_cast(u32x4_t, v), W - col - j);
          }
    } else {
#pragma unroll
      for (int j = 0; j < KE; ++j)
        if (col + j < W)
          store_part<0>((char*)(out + (int64_t)(col + j) * a.r + r0),
                        __builtin_bit_cast(u32x4_t, acc[q][j] * scale), a.r - r0);
    }
  }
}

// grid: (slabs of 16 KE columns of the wider matrix, tile, matrix and RT rank
// tiles).  A group of one tile is written at once; a group of several leaves its
// tiles' sums for lora_grad_sum_kernel, which adds them in the tiles' order.
template <int DT, int RT, bool FULL> __global__ __launch_bounds__(64 * kGradWaves) void lora_grad_kernel(LoraGrad a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, COLS = 16 * KE, U = 4, ROUND = 4 * kGradWaves;
  __shared__ f32x4_t red[kGradWaves / 2][RT][KE][64];
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const int mat = blockIdx.z & 1, q0 = (blockIdx.z >> 1) * RT;
  const int W = a.width[mat];
  if ((int)blockIdx.x * COLS >= W) return;
  const Tile t = find_tile(a.map, blockIdx.y, a.tile_rows);
  if (t.g < 0) return;
  const int g = t.g;
  // a lane whose columns end outside takes the last KE, its neighbour's again:
  // both write the same sums (W < KE: columns past W read one by one below)
  const int at = blockIdx.x * COLS + i16 * KE, last = W > KE ? W - KE : 0;
  const int col = at < last ? at : last;
  const int lo = t.row0, hi = t.row1;
  const char* wide = (const char*)a.wide[mat] + (int64_t)col * S;
  const float* v = a.v[mat];
  const int vw = mat == 0 ? lora_width(a.r) : a.r;  // floats of a row of v
  int rank[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) rank[q] = 16 * (q0 + q) + i16 < a.r ? 16 * (q0 + q) + i16 : a.r - 1;
  f32x4_t acc[RT][KE];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < KE; ++j) acc[q][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // wave w takes rows 4 w .. 4 w + 3 of every ROUND, U rounds a batch: a batch's
  // rows are in flight while the batch before is multiplied, and their tokens
  // were read one batch earlier.  Rows past the group read its last row and count 0.
  // Nothing that was loaded is looked at before its turn, which would wait for it.
  int word[2][U];
  bool live[2][U];
  u32x4_t x[2][U];
  float f[2][U][RT];
  auto tokens = [&](int buf, int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r0 + u * ROUND + g4;
      word[buf][u] = token_word(a.map, row < hi ? row : hi - 1);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load = [&](int buf, int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r0 + u * ROUND + g4, at_row = row < hi ? row : hi - 1;
      const int tok = token_in(a.map, at_row, word[buf][u]);
      const char* p = wide + (int64_t)(tok < 0 ? 0 : tok) * W * S;
      x[buf][u] = FULL ? load16<DT>(p) : load_part<DT>(p, W);
#pragma unroll
      for (int q = 0; q < RT; ++q) f[buf][u][q] = v[(int64_t)at_row * vw + rank[q]];
      live[buf][u] = row < hi && tok >= 0;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mul = [&](int buf) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float e[KE];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[buf][u][j] = live[buf][u] ? x[buf][u][j] : 0u;
      widen<DT>(x[buf][u], e);
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const float c = live[buf][u] ? f[buf][u][q] : 0.f;
#pragma unroll
        for (int j = 0; j < KE; ++j)
          acc[q][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(c, e[j], acc[q][j], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int BATCH = ROUND * U;
  const int first = lo + 4 * w;
  if (first < hi) {  // no load under a condition in the loop, as in the rank kernel
    tokens(0, first);
    tokens(1, first + BATCH);
    load(0, first);
    int r0 = first;
    for (; r0 + BATCH < hi; r0 += 2 * BATCH) {
      load(1, r0 + BATCH);
      tokens(0, r0 + 2 * BATCH);
      mul(0);
      load(0, r0 + 2 * BATCH);
      tokens(1, r0 + 3 * BATCH);
      mul(1);
    }
    if (r0 < hi) mul(0);
  }
  // the waves' sums, half by half
#pragma unroll
  for (int half = kGradWaves / 2; half > 0; half /= 2) {
    if (w >= half && w < 2 * half)
#pragma unroll
      for (int q = 0; q < RT; ++q)
#pragma unroll
        for (int j = 0; j < KE; ++j) red[w - half][q][j][lane] = acc[q][j];
    __syncthreads();
    if (w < half)
#pragma unroll
      for (int q = 0; q < RT; ++q)
#pragma unroll
        for (int j = 0; j < KE; ++j) acc[q][j] += red[w][q][j][lane];
    __syncthreads();
  }
  if (w > 0) return;
  if (t.n > 1) {
    f32x4_t* part = (f32x4_t*)a.part + grad_place(a, t, t.row0, RT * KE) + lane;
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int j = 0; j < KE; ++j) part[(q * KE + j) * 64] = acc[q][j];
  } else {
    write_grad<DT, RT>(a, t.g, mat, q0, at, col, acc);
  }
#endif
}

// One wave a unit of a group of several tiles; grid as above, for its first tile.
template <int DT, int RT> __global__ __launch_bounds__(64) void lora_grad_sum_kernel(LoraGrad a) {
  constexpr int KE = kFragElems<DT>, COLS = 16 * KE;
  const int lane = lane_id(), i16 = lane & 15;
  const int mat = blockIdx.z & 1, q0 = (blockIdx.z >> 1) * RT;
  const int W = a.width[mat];
  if ((int)blockIdx.x * COLS >= W) return;
  const Tile t = find_tile(a.map, blockIdx.y, a.tile_rows);
  if (t.g < 0 || t.n < 2 || t.row0 != t.row_first) return;
  const int at = blockIdx.x * COLS + i16 * KE, last = W > KE ? W - KE : 0;
  f32x4_t acc[RT][KE];
#pragma unroll 2
  for (int k = 0; k < t.n; ++k) {
    const f32x4_t* part = (const f32x4_t*)a.part + grad_place(a, t, t.row_first + k * a.tile_rows, RT * KE) + lane;
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int j = 0; j < KE; ++j) {
        const f32x4_t v = part[(q * KE + j) * 64];
        acc[q][j] = k ? acc[q][j] + v : v;
      }
  }
  write_grad<DT, RT>(a, t.g, mat, q0, at, at < last ? at : last, acc);
}

// ------------------------------------------------------------------ prepare
// What the backward pass needs first: A^T and B^T, and the gradients of groups
// without rows, which no other kernel comes to.  A workgroup takes 64 positions of K (or N) of a group: grid
// (ceil(K / 64) + ceil(N / 64), G).
template <typename E> __global__ __launch_bounds__(256) void lora_prepare_kernel(LoraPrepare a) {
  __shared__ E tile[64][kLoraMaxRank + 2];
  const int r = a.r, ka = (a.K + 63) / 64;
  const bool isA = (int)blockIdx.x < ka;
  const int at = (isA ? blockIdx.x : blockIdx.x - ka) * 64, W = isA ? a.K : a.N;
  const int n = W - at < 64 ? W - at : 64;
  const int64_t g = (int64_t)blockIdx.y * r * W;
  if (cut(a.map.offsets[blockIdx.y + 1], a.map.rows) <= cut(a.map.offsets[blockIdx.y], a.map.rows)) {
    float* out = (isA ? a.dA : a.dB) + g;
    for (int i = threadIdx.x; i < r * 64; i += 256) {
      if (!isA && i < n * r) out[(int64_t)at * r + i] = 0.f;
      if (isA && (i & 63) < n) out[(int64_t)(i >> 6) * W + at + (i & 63)] = 0.f;
    }
    return;
  }
  const E* from = (const E*)(isA ? a.A : a.B) + g;
  E* to = (E*)(isA ? a.At : a.Bt) + g;
  if (isA) {
    for (int i = threadIdx.x; i < r * 64; i += 256)
      if ((i & 63) < n) tile[i & 63][i >> 6] = from[(int64_t)(i >> 6) * W + at + (i & 63)];
  } else {
    for (int i = threadIdx.x; i < n * r; i += 256) tile[i / r][i % r] = from[(int64_t)at * r + i];
  }
  __syncthreads();
  if (isA) {
    for (int i = threadIdx.x; i < n * r; i += 256) to[(int64_t)at * r + i] = tile[i / r][i % r];
  } else {
    for (int i = threadIdx.x; i < r * 64; i += 256)
      if ((i & 63) < n) to[(int64_t)(i >> 6) * W + at + (i & 63)] = tile[i & 63][i >> 6];
  }
}

// Tiles of MT rows at most: whole ones, and one more for each group with rows.
int64_t most_tiles(int rows, int G, int mt) {
  const int64_t a = (int64_t)(rows + mt - 1) / mt + G;
  return a < rows ? a : rows;
}
int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }
// Rows of a rank tile, in sixteens: as many as a group has on average, so that
// A is read once for up to 64 rows (four tiles of rank 128 want too many registers).
int rank_m(int rows, int G, int r) {
  const int64_t each = (rows + G - 1) / G;
  return each <= 16 ? 1 : each <= 32 || r > 64 ? 2 : 4;
}
bool few_rows(int rows, int G) { return rows <= 16 * (int64_t)G; }

template <int DT, int RT, int M> hipError_t rank_tiles_of(const LoraRank& a, hipStream_t s) {
  hipLaunchKernelGGL((lora_rank_kernel<DT, RT, M>), dim3((unsigned)most_tiles(a.map.rows, a.map.G, 16 * M), a.splits),
                     dim3(64 * kRankWaves), 0, s, a);
  return hipGetLastError();
}
template <int DT, int RT> hipError_t rank_of(const LoraRank& a, hipStream_t s) {
  const int m = rank_m(a.map.rows, a.map.G, a.r);
  if constexpr (RT < 8)
    if (m == 4) return rank_tiles_of<DT, RT, 4>(a, s);
  return m == 1 ? rank_tiles_of<DT, RT, 1>(a, s) : rank_tiles_of<DT, RT, 2>(a, s);
}

template <int DT, int RT, int MT> hipError_t add_tiles(const LoraAdd& a, hipStream_t s) {
  const int tiles = (int)most_tiles(a.map.rows, a.map.G, MT);
  const int bare = a.map.row_of_pair && a.out != a.base ? (a.map.rows + kBareTokens - 1) / kBareTokens : 0;
  const int slabs = (a.N + kAddCols - 1) / kAddCols;
  hipLaunchKernelGGL((lora_add_kernel<DT, RT, MT>), dim3((tiles + bare) * slabs), dim3(64 * kAddWaves), 0, s, a, slabs,
                     tiles);
  return hipGetLastError();
}
template <int DT, int RT> hipError_t add_of(const LoraAdd& a, hipStream_t s) {
  return few_rows(a.map.rows, a.map.G) ? add_tiles<DT, RT, 16>(a, s) : add_tiles<DT, RT, 64>(a, s);
}

int grad_tiles(int r) { return r <= 16 ? 1 : 2; }  // rank tiles of a workgroup of the grad kernel
int grad_slabs(int K, int N, int dtype) {
  const int cols = dtype == 0 ? 16 * kFragElems<0> : 16 * kFragElems<1>;
  return ((K > N ? K : N) + cols - 1) / cols;
}
int grad_units(int r) { return 2 * ((r + 16 * grad_tiles(r) - 1) / (16 * grad_tiles(r))); }

template <int DT, int RT> hipError_t grad_of(const LoraGrad& a, hipStream_t s) {
  const dim3 grid(grad_slabs(a.width[0], a.width[1], DT), (unsigned)most_tiles(a.map.rows, a.map.G, a.tile_rows),
                  grad_units(a.r));
  // FULL: a row of each matrix holds a whole 16-byte access
  if (a.width[0] >= kFragElems<DT> && a.width[1] >= kFragElems<DT>)
    hipLaunchKernelGGL((lora_grad_kernel<DT, RT, true>), grid, dim3(64 * kGradWaves), 0, s, a);
  else
    hipLaunchKernelGGL((lora_grad_kernel<DT, RT, false>), grid, dim3(64 * kGradWaves), 0, s, a);
  if (a.part)
    hipLaunchKernelGGL((lora_grad_sum_kernel<DT, RT>), grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

#define MOK_BY_RANK(F, DT, a, s)          \
  switch (rank_tiles(a.r)) {              \
    case 1: return F<DT, 1>(a, s);        \
    case 2: return F<DT, 2>(a, s);        \
    case 4: return F<DT, 4>(a, s);        \
    default: return F<DT, 8>(a, s);       \
  }
template <int DT> hipError_t rank_dt(const LoraRank& a, hipStream_t s) { MOK_BY_RANK(rank_of, DT, a, s) }
template <int DT> hipError_t add_dt(const LoraAdd& a, hipStream_t s) { MOK_BY_RANK(add_of, DT, a, s) }
#undef MOK_BY_RANK
template <int DT> hipError_t grad_dt(const LoraGrad& a, hipStream_t s) {
  return a.r <= 16 ? grad_of<DT, 1>(a, s) : grad_of<DT, 2>(a, s);
}

}  // namespace

int lora_splits(int rows, int G, int r, int K, int dtype) {
  const int64_t tiles = most_tiles(rows, G, 16 * rank_m(rows, G, r));
  if (tiles == 0) return 1;
  const int steps = K / (dtype == 0 ? 16 : 32);
  // four workgroups a compute unit, for it is the compute units, each with its
  // own limit of loads in flight, that have to be kept evenly at work; eight K
  // steps a wave (four with a few tiles); and parts of no more than an eighth of
  // the bytes that they come from
  int64_t n = (4 * kNumCUs + tiles - 1) / tiles;
  const int64_t each = steps / ((tiles <= 64 ? 4 : 8) * kRankWaves);
  const int64_t bytes = (int64_t)K * (dtype == 0 ? 4 : 2) / (8 * 4 * lora_width(r));
  if (n > each) n = each;
  if (tiles > 64 && n > bytes) n = bytes;
  return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}

LoraGradPlan lora_grad_plan(int rows, int G, int r, int K, int N, int dtype) {
  LoraGradPlan p;
  const int cols = dtype == 0 ? 16 * kFragElems<0> : 16 * kFragElems<1>;
  p.tile_rows = grad_rows(rows, K, N, cols);
  // no group can have a second tile: no sums to add
  p.part_bytes = rows > p.tile_rows ? (int64_t)grad_places(rows, p.tile_rows) * grad_units(r) * grad_slabs(K, N, dtype) *
                                          grad_tiles(r) * (cols / 16) * 64 * 16
                                    : 0;
  return p;
}

hipError_t launch_lora_rank(const LoraRank& a, hipStream_t s) {
  return a.dtype == 0 ? rank_dt<0>(a, s) : a.dtype == 1 ? rank_dt<1>(a, s) : rank_dt<2>(a, s);
}
hipError_t launch_lora_add(const LoraAdd& a, hipStream_t s) {
  return a.dtype == 0 ? add_dt<0>(a, s) : a.dtype == 1 ? add_dt<1>(a, s) : add_dt<2>(a, s);
}
hipError_t launch_lora_grad(const LoraGrad& a, hipStream_t s) {
  return a.dtype == 0 ? grad_dt<0>(a, s) : a.dtype == 1 ? grad_dt<1>(a, s) : grad_dt<2>(a, s);
}
hipError_t launch_lora_prepare(const LoraPrepare& a, hipStream_t s) {
  const dim3 grid((a.K + 63) / 64 + (a.N + 63) / 64, a.map.G);
  if (a.dtype == 0) hipLaunchKernelGGL((lora_prepare_kernel<uint32_t>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((lora_prepare_kernel<uint16_t>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mok
