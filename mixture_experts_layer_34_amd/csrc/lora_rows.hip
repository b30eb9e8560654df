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
//  - transpose: A^T and B^T for the backward pass, which then runs the first two
//    kernels on them (du: rank with B^T; dx: add with A^T).
#include "frag.h"
#include "lora_rows.h"
#include "mok_internal.h"

namespace mok {
namespace {

struct Tile {
  int g, row0, row1;  // rows [row0, row1) of group g; g < 0: none
};

__device__ __forceinline__ int cut(int v, int rows) { return v < 0 ? 0 : v > rows ? rows : v; }

// The t-th tile of MT rows, the groups' tiles counted one after the other.
template <int MT> __device__ __forceinline__ Tile find_tile(const LoraMap& m, int t) {
  const int lane = lane_id();
  int before = 0;
  for (int g0 = 0; g0 < m.G; g0 += 64) {
    const int g = g0 + lane;
    const int lo = cut(m.offsets[g < m.G ? g : m.G], m.rows);
    const int hi = cut(m.offsets[g < m.G ? g + 1 : m.G], m.rows);
    const int n = hi > lo ? (hi - lo + MT - 1) / MT : 0;
    const int to = wave_prefix(n) + before;
    const uint64_t hit = __ballot(t >= to - n && t < to);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int first = __builtin_amdgcn_readlane(to - n, l), a = __builtin_amdgcn_readlane(lo, l),
                b = __builtin_amdgcn_readlane(hi, l);
      const int row0 = a + (t - first) * MT;
      return Tile{g0 + l, row0, row0 + MT < b ? row0 + MT : b};
    }
    before = __builtin_amdgcn_readlane(to, 63);
  }
  return Tile{-1, 0, 0};
}

// The token of a sorted row; -1: none.
__device__ __forceinline__ int token_of(const LoraMap& m, int row) {
  if (!m.pair_of_row) return row;
  const int t = m.pair_of_row[row];
  return t >= 0 && t < m.rows ? t : -1;
}

// ------------------------------------------------------------------ rank
constexpr int kRankWaves = 4;

template <int DT, int RT, int M> __global__ __launch_bounds__(64 * kRankWaves) void lora_rank_kernel(LoraRank a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes;
  constexpr int U = RT >= 4 ? 1 : RT == 2 ? 2 : 4;  // K steps of a chunk
  __shared__ f32x4_t red[kRankWaves - 1][M][RT][64];
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const Tile t = find_tile<16 * M>(a.map, blockIdx.x);
  if (t.g < 0) return;
  const int full = a.K / STEP, steps = (a.K + STEP - 1) / STEP;
  const int part = blockIdx.y * kRankWaves + w, parts = a.splits * kRankWaves;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
  const int e1 = s1 < full ? s1 : full;
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
  const int ns = e1 > s0 ? e1 - s0 : 0, nc = ns / U * U;
  if (nc)
#pragma unroll
    for (int j = 0; j < U; ++j) load(0, j, j);
  for (int c = 0; c < nc; c += 2 * U) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (c + b * U < nc) {
        if (c + (b + 1) * U < nc)
#pragma unroll
          for (int j = 0; j < U; ++j) load(1 - b, j, c + (b + 1) * U + j);
#pragma unroll
        for (int j = 0; j < U; ++j) mul(b, j);
      }
  }
  if constexpr (U > 1) {
#pragma unroll
    for (int j = 0; j < U - 1; ++j)
      if (nc + j < ns) load(0, j, nc + j);
#pragma unroll
    for (int j = 0; j < U - 1; ++j)
      if (nc + j < ns) mul(0, j);
  }
  if (s1 > full && s1 > s0) {  // the step that K ends in
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
    float* to = a.part + ((int64_t)blockIdx.y * a.map.rows + row) * a.r;
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      f32x4_t v = acc[m][q];
#pragma unroll
      for (int k = 0; k < kRankWaves - 1; ++k) v += red[k][m][q][lane];
      const int r0 = 16 * q + 4 * g4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < a.r) to[r0 + i] = tok[m] < 0 ? 0.f : v[i];
    }
  }
#endif
}

// ------------------------------------------------------------------ add
constexpr int kAddWaves = 4;
constexpr int kAddCols = 64 * kAddWaves;  // columns of a workgroup
constexpr int kBareTokens = 64;           // tokens a workgroup looks over for rows of no adapter

// Rows of no adapter: out = base, or 0.
template <int DT> __device__ __forceinline__ void bare_rows(const LoraAdd& a, int block) {
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, LPR = kAddCols / KE, RPW = 64 / LPR;
  const int lane = lane_id(), w = wave_id();
  const int col = blockIdx.y * kAddCols + (lane % LPR) * KE;
  for (int i = w * RPW + lane / LPR; i < kBareTokens; i += kAddWaves * RPW) {
    const int64_t t = (int64_t)block * kBareTokens + i;
    if (t >= a.map.rows || col >= a.N) continue;
    const int row = a.map.row_of_pair[t];
    if (row >= 0 && row < a.map.rows) continue;
    const int64_t at = (t * a.N + col) * S;
    const u32x4_t v = a.base ? load_part<DT>((const char*)a.base + at, a.N - col) : u32x4_t{0, 0, 0, 0};
    store_part<DT>((char*)a.out + at, v, a.N - col);
  }
}

// tiles: workgroups that take tiles; the rest look for rows of no adapter.
// Each takes MT rows and kAddCols columns.
template <int DT, int RT, int MT> __global__ __launch_bounds__(64 * kAddWaves) void lora_add_kernel(LoraAdd a, int tiles) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, Q = 16 / KE;  // Q: accesses of a lane's sixteen columns
  if ((int)blockIdx.x >= tiles) {
    bare_rows<DT>(a, blockIdx.x - tiles);
    return;
  }
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const int base = blockIdx.y * kAddCols + w * 64;
  const Tile t = find_tile<MT>(a.map, blockIdx.x);
  const bool keeps = a.u && blockIdx.y == 0 && w == 0;
  if (t.g < 0 || base >= a.N) return;
  // 16-bit types: virtual K of 2 * 16 RT, the high parts, then the low ones
  auto rank_of = [&](int s) { const int c = 4 * s + g4; return DT == 0 ? 4 * c : 8 * (c % (2 * RT)); };
  // row i16 of tile q is column base + 16 (i16 / 4) + 4 q + i16 % 4: a lane's
  // results are then sixteen neighbouring columns
  u32x4_t qb[4][RT];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = base + 16 * (i16 >> 2) + 4 * q + (i16 & 3);
    const char* row = (const char*)a.B + ((int64_t)t.g * a.N + (n < a.N ? n : a.N - 1)) * a.r * S;
#pragma unroll
    for (int s = 0; s < RT; ++s) {
      const int r0 = rank_of(s);
      qb[q][s] = load_part<DT>(row + r0 * S, r0 < a.r ? a.r - r0 : 0);
    }
  }
  const float scale = a.scale ? a.scale[t.g] : 1.f;
  const int col = base + 16 * g4;
  for (int sub = 0; sub < MT / 16; ++sub) {
    const int row = t.row0 + 16 * sub + i16;
    if (t.row0 + 16 * sub >= t.row1) break;
    const int at_row = row < t.row1 ? row : t.row1 - 1;
    const int tok = token_of(a.map, at_row);
    const bool live = row < t.row1 && tok >= 0;
    const int64_t at = ((int64_t)(tok < 0 ? 0 : tok) * a.N + col) * S;
    u32x4_t y[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int left = a.N - col - j * KE;
      y[j] = a.base && live && left > 0 ? load_part<DT>((const char*)a.base + at + j * 16, left)
                                        : u32x4_t{0, 0, 0, 0};
    }
    float v[RT][KE];
    float big = 0.f;
#pragma unroll
    for (int s = 0; s < RT; ++s) {
      const int r0 = rank_of(s);
#pragma unroll
      for (int j = 0; j < KE; ++j) v[s][j] = 0.f;
      for (int p = 0; p < a.splits; ++p) {
        const float* from = a.part + ((int64_t)p * a.map.rows + at_row) * a.r + r0;
#pragma unroll
        for (int j = 0; j < KE; ++j)
          if (r0 + j < a.r) v[s][j] += from[j];
      }
      if (keeps && row < t.row1 && (DT == 0 || 4 * s + g4 < 2 * RT))
#pragma unroll
        for (int j = 0; j < KE; ++j)
          if (r0 + j < a.r) a.u[(int64_t)row * a.r + r0 + j] = v[s][j];
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
      if (big > 0.f && big < INFINITY) {
        const int e = big < 0x1p-126f ? -126 : ilogbf(big);
        up = ldexpf(1.f, e);
        const float down = ldexpf(1.f, -e);
#pragma unroll
        for (int s = 0; s < RT; ++s)
#pragma unroll
          for (int j = 0; j < KE; ++j) v[s][j] *= down;
      }
    }
    f32x4_t acc[4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < RT; ++s) {
      u32x4_t f = narrow<DT>(v[s]);
      if constexpr (DT != 0) {
        if (4 * s + g4 >= 2 * RT) {
          float hi[KE];
          widen<DT>(f, hi);
#pragma unroll
          for (int j = 0; j < KE; ++j) hi[j] = v[s][j] - hi[j];
          f = narrow<DT>(hi);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = mma<DT>(qb[q][s], f, acc[q]);
    }
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int left = a.N - col - j * KE;
      if (left <= 0) break;
      float o[KE];
      widen<DT>(y[j], o);
#pragma unroll
      for (int i = 0; i < KE; ++i) o[i] = fmaf(acc[(j * KE + i) / 4][i % 4], up, o[i]);
      store_part<DT>((char*)a.out + at + j * 16, narrow<DT>(o), left);
    }
  }
#endif
}

// ------------------------------------------------------------------ grad
constexpr int kGradWaves = 8;

// grid: (64 KE-wide slabs of the wider matrix, group, matrix and RT rank tiles)
template <int DT, int RT> __global__ __launch_bounds__(64 * kGradWaves) void lora_grad_kernel(LoraGrad a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, COLS = 16 * KE, U = 4;
  __shared__ f32x4_t red[kGradWaves / 2][RT][KE][64];
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const int mat = blockIdx.z & 1, q0 = (blockIdx.z >> 1) * RT;
  const int W = a.width[mat], col = blockIdx.x * COLS + i16 * KE, g = blockIdx.y;
  if ((int)blockIdx.x * COLS >= W) return;
  const int lo = cut(a.map.offsets[g], a.map.rows), hi = cut(a.map.offsets[g + 1], a.map.rows);
  const char* wide = (const char*)a.wide[mat];
  const float* v = a.v[mat];
  f32x4_t acc[RT][KE];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < KE; ++j) acc[q][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // wave w takes rows 4 w .. 4 w + 3 of every 4 kGradWaves, U such rounds at a time
  for (int r0 = lo + 4 * w; r0 < hi; r0 += 4 * kGradWaves * U) {
    u32x4_t x[U];
    float f[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r0 + u * 4 * kGradWaves + g4;
      const int tok = row < hi ? token_of(a.map, row) : -1;
      x[u] = u32x4_t{0, 0, 0, 0};
      if (tok >= 0 && col < W) x[u] = load_part<DT>(wide + ((int64_t)tok * W + col) * S, W - col);
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int rr = 16 * (q0 + q) + i16;
        f[u][q] = tok >= 0 && rr < a.r ? v[(int64_t)row * a.r + rr] : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float e[KE];
      widen<DT>(x[u], e);
#pragma unroll
      for (int q = 0; q < RT; ++q)
#pragma unroll
        for (int j = 0; j < KE; ++j) acc[q][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[u][q], e[j], acc[q][j], 0, 0, 0);
    }
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
  const float scale = a.scale ? a.scale[g] : 1.f;
  float* out = a.out[mat] + (int64_t)g * a.r * W;
  // lane: ranks 16 (q0 + q) + 4 g4 + 0..3 of column col + j
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < KE; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 16 * (q0 + q) + 4 * g4 + i;
        if (rr < a.r && col + j < W) {
          if (mat == 0) out[(int64_t)rr * W + col + j] = scale * acc[q][j][i];
          else out[(int64_t)(col + j) * a.r + rr] = scale * acc[q][j][i];
        }
      }
#endif
}

// ------------------------------------------------------------------ transpose
// A workgroup turns 64 positions of K (or N) over: grid (ceil(K / 64) + ceil(N / 64), G).
template <typename E> __global__ __launch_bounds__(256) void lora_transpose_kernel(const E* A, const E* B, int r, int K,
                                                                                   int N, E* At, E* Bt) {
  __shared__ E tile[64][kLoraMaxRank + 2];
  const int ka = (K + 63) / 64;
  const bool isA = (int)blockIdx.x < ka;
  const int at = (isA ? blockIdx.x : blockIdx.x - ka) * 64, W = isA ? K : N;
  const int n = W - at < 64 ? W - at : 64;
  const int64_t g = (int64_t)blockIdx.y * r * W;
  if (isA) {
    for (int i = threadIdx.x; i < r * 64; i += 256)
      if ((i & 63) < n) tile[i & 63][i >> 6] = A[g + (int64_t)(i >> 6) * W + at + (i & 63)];
  } else {
    for (int i = threadIdx.x; i < n * r; i += 256) tile[i / r][i % r] = B[g + (int64_t)at * r + i];
  }
  __syncthreads();
  if (isA) {
    for (int i = threadIdx.x; i < n * r; i += 256) At[g + (int64_t)at * r + i] = tile[i / r][i % r];
  } else {
    for (int i = threadIdx.x; i < r * 64; i += 256)
      if ((i & 63) < n) Bt[g + (int64_t)(i >> 6) * W + at + (i & 63)] = tile[i & 63][i >> 6];
  }
}

// Tiles of MT rows at most: whole ones, and one more for each group with rows.
int64_t most_tiles(int rows, int G, int mt) {
  const int64_t a = (int64_t)(rows + mt - 1) / mt + G;
  return a < rows ? a : rows;
}
int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }
// Tiles of sixteen rows where a group has no more on average.
bool few_rows(int rows, int G) { return rows <= 16 * (int64_t)G; }

template <int DT, int RT> hipError_t rank_of(const LoraRank& a, hipStream_t s) {
  if (few_rows(a.map.rows, a.map.G))
    hipLaunchKernelGGL((lora_rank_kernel<DT, RT, 1>), dim3((unsigned)most_tiles(a.map.rows, a.map.G, 16), a.splits),
                       dim3(64 * kRankWaves), 0, s, a);
  else
    hipLaunchKernelGGL((lora_rank_kernel<DT, RT, 2>), dim3((unsigned)most_tiles(a.map.rows, a.map.G, 32), a.splits),
                       dim3(64 * kRankWaves), 0, s, a);
  return hipGetLastError();
}

template <int DT, int RT, int MT> hipError_t add_tiles(const LoraAdd& a, hipStream_t s) {
  const int tiles = (int)most_tiles(a.map.rows, a.map.G, MT);
  const int bare = a.map.row_of_pair && a.out != a.base ? (a.map.rows + kBareTokens - 1) / kBareTokens : 0;
  hipLaunchKernelGGL((lora_add_kernel<DT, RT, MT>), dim3(tiles + bare, (a.N + kAddCols - 1) / kAddCols),
                     dim3(64 * kAddWaves), 0, s, a, tiles);
  return hipGetLastError();
}
template <int DT, int RT> hipError_t add_of(const LoraAdd& a, hipStream_t s) {
  return few_rows(a.map.rows, a.map.G) ? add_tiles<DT, RT, 16>(a, s) : add_tiles<DT, RT, 64>(a, s);
}

template <int DT, int RT> hipError_t grad_of(const LoraGrad& a, hipStream_t s) {
  const int most = a.width[0] > a.width[1] ? a.width[0] : a.width[1], cols = 16 * kFragElems<DT>;
  hipLaunchKernelGGL((lora_grad_kernel<DT, RT>),
                     dim3((most + cols - 1) / cols, a.map.G, 2 * ((a.r + 16 * RT - 1) / (16 * RT))),
                     dim3(64 * kGradWaves), 0, s, a);
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

int lora_splits(int rows, int G, int K, int dtype) {
  const int mt = few_rows(rows, G) ? 16 : 32;
  const int steps = K / (dtype == 0 ? 16 : 32);
  const int64_t tiles = most_tiles(rows, G, mt);
  // one workgroup a compute unit, and four K steps or more for each of its waves
  int64_t n = tiles ? kNumCUs / tiles : 1;
  if (n > steps / (4 * kRankWaves)) n = steps / (4 * kRankWaves);
  return n < 1 ? 1 : n > 16 ? 16 : (int)n;
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
hipError_t launch_lora_transpose(const void* A, const void* B, int G, int r, int K, int N, int dtype, void* At,
                                 void* Bt, hipStream_t s) {
  const dim3 grid((K + 63) / 64 + (N + 63) / 64, G);
  if (dtype == 0)
    hipLaunchKernelGGL((lora_transpose_kernel<uint32_t>), grid, dim3(256), 0, s, (const uint32_t*)A, (const uint32_t*)B,
                       r, K, N, (uint32_t*)At, (uint32_t*)Bt);
  else
    hipLaunchKernelGGL((lora_transpose_kernel<uint16_t>), grid, dim3(256), 0, s, (const uint16_t*)A, (const uint16_t*)B,
                       r, K, N, (uint16_t*)At, (uint16_t*)Bt);
  return hipGetLastError();
}

}  // namespace mok
