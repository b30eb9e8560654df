// Low-rank adapters of many requests beside a projection, forward and
// backward.  Rows are sorted by adapter (a pair map whose experts are the
// adapters), or are the experts' sorted rows with one adapter pair each:
//   u_q = A_g x_q,      out_q = y_q + s_g B_g u_q
//   du_q = B_g^T dout_q, dx_q = base_q + s_g A_g^T du_q,
//   dA_g = s_g sum_q du_q x_q^T,  dB_g = s_g sum_q dout_q u_q^T
// over the rows q of adapter g.
//
// All of it is bound by moving the rows once: with ranks of 8 to 32 beside widths
// of thousands the products are a few percent of what the matrix cores do in that
// time.  The kernels, with what they take at 8192 rows of 4096 bf16 columns and
// rank 16 (a copy of one such matrix into another takes 24-26 us there):
//  - rank (u and du; 17.6-20.6 us): a workgroup takes a tile of one adapter's rows,
//    its waves share K and meet in LDS; with few rows K is split over workgroups too,
//    whose fp32 parts the next kernel adds in order (no atomics).
//  - add (out and dx; 37 us): the transposed product B u^T, so that a lane holds
//    neighbouring columns of one row, y in, out back.  A wave keeps the B of its
//    128 columns (64 for fp32 and for ranks past 32) in registers and runs over its
//    rows.  u enters 16-bit matrix
//    instructions as a high and a low part (a K of 2 r), so that it loses nothing
//    next to out's own rounding.
//  - grad (dA and dB; 38 us for both matrices, 3.5 TB/s): K is the rows there.
//    v_mfma_f32_16x16x4 takes one value of each operand a lane, so the j-th elements
//    of sixteen lanes' 16-byte loads are an operand as they are: no transposing, and u
//    and du keep their 32 bits.  From rank 64 on that instruction's rate bounds it.
//  - prepare (5 us): A^T and B^T for the backward pass, which then runs the first two
//    kernels on them (du: rank with B^T; dx: add with A^T).
#include "frag.h"
#include "lora_rows.h"
#include "mok_internal.h"

namespace mok {
namespace {

__device__ __forceinline__ int cut(int v, int rows) { return v < 0 ? 0 : v > rows ? rows : v; }

// All groups' rows, whatever the offsets between the first and the last are.
struct Span {
  int first, last;
  // an offset between them, cut to them: offsets that fall name no rows outside
  __device__ __forceinline__ int in(int offset) const { return offset < first ? first : offset > last ? last : offset; }
};
__device__ __forceinline__ Span span_of(const LoraMap& m, int first, int last) {
  first = cut(first, m.rows);
  last = cut(last, m.rows);
  return Span{first, last > first ? last : first};
}

// The groups' rows, shared out evenly in n ranges of `each` rows.  (A compute unit
// with more rows than another ends later by as much: they get even shares of the
// memory's rate.)  What a kernel reads before it can ask for its first row adds to
// its time in full, so one load brings all offsets of up to 63 groups, a lane each.
struct Rows : Span {
  int offset;  // of group `lane`, or the end of the last
  int each;
  __device__ __forceinline__ int begin(int i) const {
    const int64_t at = first + (int64_t)each * i;
    return at < last ? (int)at : last;
  }
  __device__ __forceinline__ int range_of(int row) const { return (row - first) / each; }
};
__device__ __forceinline__ Rows rows_of(const LoraMap& m, int n) {
  Rows r;
  const int lane = lane_id();
  r.offset = m.offsets[lane < m.G ? lane : m.G];
  static_cast<Span&>(r) = span_of(m, __builtin_amdgcn_readfirstlane(r.offset),
                                  m.G < 64 ? __builtin_amdgcn_readlane(r.offset, m.G) : m.offsets[m.G]);
  r.each = (r.last - r.first + n - 1) / n;
  r.each = r.each > 0 ? r.each : 1;
  return r;
}

// The rows of a range that are of one group: those from `row` on.
struct Part {
  int g, end;    // the group; the end of its rows in the range
  int lo, hi;    // all of the group's rows
};
__device__ __forceinline__ Part part_at(const LoraMap& m, const Rows& rows, int row, int end) {
  const int lane = lane_id();
  int g, lo, hi;
  // the offsets behind the first that are at or before row
  if (m.G < 64) {
    g = __popcll(__ballot(lane > 0 && lane < m.G && rows.offset <= row));
    lo = __builtin_amdgcn_readlane(rows.offset, g);
    hi = __builtin_amdgcn_readlane(rows.offset, g + 1);
  } else {
    g = 0;
#pragma unroll 4
    for (int g0 = 1; g0 < m.G; g0 += 64) {
      const int at = g0 + lane;
      g += __popcll(__ballot(at < m.G && m.offsets[at < m.G ? at : 0] <= row));
    }
    g = __builtin_amdgcn_readfirstlane(g);
    lo = m.offsets[g];
    hi = m.offsets[g + 1];
  }
  lo = rows.in(lo);
  hi = rows.in(hi);
  const int e = hi < end ? hi : end;
  return Part{g, e > row ? e : row + 1, lo, hi};  // (offsets that fall: a row at a time)
}

// The t-th tile of `height` rows of one group, the groups' tiles counted one after
// the other; g < 0: none.
__device__ __forceinline__ Part find_tile(const LoraMap& m, int t, int height, int* row0) {
  const int lane = lane_id();
  int before = 0;
  for (int g0 = 0; g0 < m.G; g0 += 64) {
    const int g = g0 + lane;
    const int lo = cut(m.offsets[g < m.G ? g : m.G], m.rows), hi = cut(m.offsets[g < m.G ? g + 1 : m.G], m.rows);
    const int n = hi > lo ? (int)((unsigned)(hi - lo + height - 1) / (unsigned)height) : 0;
    const int to = wave_prefix(n) + before;
    const uint64_t hit = __ballot(t >= to - n && t < to);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int first = __builtin_amdgcn_readlane(to - n, l);
      const int a = __builtin_amdgcn_readlane(lo, l), b = __builtin_amdgcn_readlane(hi, l);
      *row0 = a + (t - first) * height;
      return Part{g0 + l, *row0 + height < b ? *row0 + height : b, a, b};
    }
    before = __builtin_amdgcn_readlane(to, 63);
  }
  return Part{-1, 0, 0, 0};
}

// Workgroup b of n (a multiple of 8) on XCD b % 8: its place in the order in which
// every XCD has an eighth of the rows, so that a group's A or B comes to one or
// two of the eight L2s.
__device__ __forceinline__ int by_xcd(int b, int n) { return (b & 7) * (n >> 3) + (b >> 3); }

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

// grid: (tiles of a.height rows of one group, or ranges of rows, in eights; shares of K)
// ODD: rows of an odd number of 16-bit elements.
template <int DT, int RT, int M, bool ODD> __global__ __launch_bounds__(64 * kRankWaves) void lora_rank_kernel(LoraRank a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, STEP = kFragStep<DT>, S = Elem<DT>::kBytes;
  constexpr int U = RT >= 4 ? 1 : RT == 2 || M > 2 ? 2 : 4;  // K steps of a chunk
  __shared__ f32x4_t red[kRankWaves - 1][M][RT][64];
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const int full = a.K / STEP, steps = (a.K + STEP - 1) / STEP;
  // this workgroup's K steps, [s0, s1): its waves take chunks in turn, so that
  // what they read at a time is neighbouring
  const int s0 = (int)((int64_t)steps * blockIdx.y / a.splits), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / a.splits);
  const int ns = (s1 < full ? s1 : full) - s0;  // whole steps
  const int64_t at = (int64_t)(s0 * STEP + g4 * KE) * S;
  const int place = by_xcd(blockIdx.x, gridDim.x);
  Rows rows{};
  Part t{0, 0, 0, 0};
  int row0, end;
  if (a.height) {
    t = find_tile(a.map, place, a.height, &row0);
    if (t.g < 0) return;
    end = t.end;
  } else {
    if (place >= a.ranges) return;
    rows = rows_of(a.map, a.ranges);
    row0 = rows.begin(place);
    end = rows.begin(place + 1);
  }
  for (; row0 < end; row0 += 16 * M) {
    if (row0 >= t.end) t = part_at(a.map, rows, row0, end);
    const int row1 = row0 + 16 * M < t.end ? row0 + 16 * M : t.end;
    const char *px[M], *pa[RT];
    int word[M], tok[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int row = row0 + 16 * m + i16;
      word[m] = token_word(a.map, row < row1 ? row : row1 - 1);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int row = row0 + 16 * m + i16;
      tok[m] = token_in(a.map, row < row1 ? row : row1 - 1, word[m]);
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
    Quad<DT, ODD> qx[2][U][M], qa[2][U][RT];
    auto load = [&](int buf, int j, int step) {
      const int o = step * STEP * S;
#pragma unroll
      for (int m = 0; m < M; ++m) qx[buf][j][m].load(px[m] + o);
#pragma unroll
      for (int q = 0; q < RT; ++q) qa[buf][j][q].load(pa[q] + o);
    };
    auto mul = [&](int buf, int j) {
      u32x4_t vx[M];
#pragma unroll
      for (int m = 0; m < M; ++m) vx[m] = qx[buf][j][m].get(shift_of<ODD>(px[m]));
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const u32x4_t va = qa[buf][j][q].get(shift_of<ODD>(pa[q]));
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m][q] = mma<DT>(va, vx[m], acc[m][q]);
      }
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
      const int k = full * STEP + g4 * KE;
      u32x4_t vx[M], va[RT];
      if (a.K >= KE) {
        const int at_k = tail_at<DT>(k, a.K), o = (at_k - g4 * KE - s0 * STEP) * S;  // the pointers stand at s0 STEP + g4 KE
#pragma unroll
        for (int m = 0; m < M; ++m) vx[m] = load16<DT>(px[m] + o);
#pragma unroll
        for (int q = 0; q < RT; ++q) va[q] = load16<DT>(pa[q] + o);
#pragma unroll
        for (int m = 0; m < M; ++m) vx[m] = but_first<DT>(vx[m], k - at_k);
      } else {
#pragma unroll
        for (int m = 0; m < M; ++m) vx[m] = load_part<DT>(px[m], a.K - k);
#pragma unroll
        for (int q = 0; q < RT; ++q) va[q] = load_part<DT>(pa[q], a.K - k);
      }
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int q = 0; q < RT; ++q) acc[m][q] = mma<DT>(va[q], vx[m], acc[m][q]);
    }
    if (w > 0)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int q = 0; q < RT; ++q) red[w - 1][m][q][lane] = acc[m][q];
    __syncthreads();
    if (w == 0)
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int row = row0 + 16 * m + i16;
        float* to = a.part + ((int64_t)blockIdx.y * a.map.rows + row) * (16 * RT);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          f32x4_t v = acc[m][q];
#pragma unroll
          for (int k = 0; k < kRankWaves - 1; ++k) v += red[k][m][q][lane];
          const int r0 = 16 * q + 4 * g4;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = tok[m] < 0 || r0 + i >= a.r ? 0.f : v[i];
          if (row < row1) *reinterpret_cast<f32x4_t*>(to + r0) = v;
        }
      }
    row0 = row1 - 16 * M;  // the next rows, of this group or another
    if (row1 < end) __syncthreads();  // the sums are read before they are written again
  }
#endif
}

// ------------------------------------------------------------------ add
constexpr int kAddWaves = 4;
constexpr int kBareTokens = 16;  // tokens a wave looks over at once for rows of no adapter
// Most workgroups that look: a launch counts its threads in 32 bits, and 2^30 rows at
// kBareTokens a wave would pass them.  Each goes on to further tokens where there are more.
constexpr int kBareWorkgroups = 1 << 16;

// 64-column blocks of a wave (8192 x 4096 of rank 16: 39.4 us with two, 45.0 with
// one, 47.0 with four; 24576 x 1408 of rank 32: 65 with two, 76 with one).
template <int DT, int RT> constexpr int kAddBlocks = RT >= 4 || DT == 0 ? 1 : 2;

// Rows of no adapter: out = base, or 0.  For the kBareTokens tokens from t0 on, by a wave.
template <int DT> __device__ __forceinline__ void bare_rows(const LoraAdd& a, int64_t t0) {
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes;
  const int lane = lane_id();
  bool bare = false;
  if (lane < kBareTokens && t0 + lane < a.map.rows) {
    const int row = a.map.row_of_pair[t0 + lane];
    bare = row < 0 || row >= a.map.rows;
  }
  for (uint64_t left = __ballot(bare); left; left &= left - 1) {
    const int64_t at = (t0 + __ffsll((unsigned long long)left) - 1) * a.N;
    const char* from = (const char*)a.base + at * S;
    char* to = (char*)a.out + at * S;
    if (a.N >= KE && a.base) {  // eight accesses in flight; one that would end outside copies the last KE columns
      for (int c0 = lane * KE; c0 < a.N; c0 += 8 * 64 * KE) {
        u32x4_t v[8];
        int col[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          col[i] = c0 + i * 64 * KE;
          col[i] = col[i] < a.N - KE ? col[i] : a.N - KE;
          v[i] = load16<DT>(from + col[i] * S);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) store16<DT>(to + col[i] * S, v[i]);
      }
    } else {
      for (int col = lane * KE; col < a.N; col += 64 * KE)
        store_part<DT>(to + col * S, a.base ? load_part<DT>(from + col * S, a.N - col) : u32x4_t{0, 0, 0, 0}, a.N - col);
    }
  }
}

// A wave takes a range of the rows and a block of columns; the blocks of a range
// are neighbouring waves.  bare: workgroups that look for rows of no adapter.
template <int DT, int RT>
__global__ __launch_bounds__(64 * kAddWaves) void lora_add_kernel(LoraAdd a, int ranges, int bare) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, Q = 16 / KE;  // Q: accesses of a lane's sixteen columns
  constexpr int CT = kAddBlocks<DT, RT>, W = 16 * RT;
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  if ((int)blockIdx.x < bare) {
    const int64_t at_once = (int64_t)bare * kAddWaves * kBareTokens;
    for (int64_t t0 = (blockIdx.x * kAddWaves + w) * kBareTokens; t0 < a.map.rows; t0 += at_once) bare_rows<DT>(a, t0);
    return;
  }
  const int blocks = (a.N + 64 * CT - 1) / (64 * CT);
  const int unit = by_xcd(blockIdx.x - bare, gridDim.x - bare) * kAddWaves + w, block = unit % blocks, range = unit / blocks;
  if (range >= ranges) return;
  const Rows rows = rows_of(a.map, ranges);
  const int base = block * 64 * CT, end = rows.begin(range + 1);
  const bool keeps = a.u && block == 0;
  const bool whole = base + 64 * CT <= a.N;  // every lane has all of its columns
  // 16-bit types: virtual K of 2 * 16 RT, the high parts, then the low ones
  auto rank_of = [&](int s) { const int c = 4 * s + g4; return DT == 0 ? 4 * c : 8 * (c % (2 * RT)); };
  const int col = base + KE * g4;
  for (int row0 = rows.begin(range); row0 < end;) {
    const Part t = part_at(a.map, rows, row0, end);
    const float scale = a.scale ? a.scale[t.g] : 1.f;

    // sixteen rows at a time: the next ones are in flight, and the tokens of
    // those behind, while these are worked on (no load under a condition, none
    // moved to its use; rows past the group ask for its last one again)
    u32x4_t qb[CT][4][RT];
    int word[2], tok[2];
    u32x4_t y[2][CT][Q];
    f32x4_t u[2][RT][KE / 4];
    auto at_row = [&](int r) { return r + i16 < t.end ? r + i16 : t.end - 1; };
    auto words = [&](int buf, int r) {
      word[buf] = token_word(a.map, at_row(r));
      __builtin_amdgcn_sched_barrier(0);
    };
    auto load = [&](int buf, int r) {
      tok[buf] = token_in(a.map, at_row(r), word[buf]);
      const int64_t at = ((int64_t)(tok[buf] < 0 ? 0 : tok[buf]) * a.N + col) * S;
#pragma unroll
      for (int s = 0; s < RT; ++s)
#pragma unroll
        for (int j = 0; j < KE / 4; ++j)
          u[buf][s][j] = *reinterpret_cast<const f32x4_t*>(a.part + (int64_t)at_row(r) * W + rank_of(s) + 4 * j);
      if (whole && a.base) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int j = 0; j < Q; ++j) y[buf][c][j] = load16<DT>((const char*)a.base + at + 64 * (c * Q + j));
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto work = [&](int buf, int r) {
      const bool live = r + i16 < t.end && tok[buf] >= 0;
      const int64_t at = ((int64_t)(tok[buf] < 0 ? 0 : tok[buf]) * a.N + col) * S;
      float v[RT][KE];
      float big = 0.f;
#pragma unroll
      for (int s = 0; s < RT; ++s) {
        const int r0 = rank_of(s);
#pragma unroll
        for (int j = 0; j < KE / 4; ++j) {
          f32x4_t sum = u[buf][s][j];
          const float* from = a.part + (int64_t)at_row(r) * W + r0 + 4 * j;
#pragma unroll 8
          for (int p = 1; p < a.splits; ++p) sum += *reinterpret_cast<const f32x4_t*>(from + (int64_t)p * a.map.rows * W);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[s][4 * j + i] = sum[i];
        }
        if (keeps && r + i16 < t.end && (DT == 0 || 4 * s + g4 < 2 * RT))
#pragma unroll
          for (int j = 0; j < KE; ++j)
            if (r0 + j < a.u_width) a.u[(int64_t)(r + i16) * a.u_width + r0 + j] = v[s][j];
#pragma unroll
        for (int j = 0; j < KE; ++j) {
          v[s][j] *= scale;
          big = fmaxf(big, fabsf(v[s][j]));
        }
      }
      // fp16: the row's sums brought to [2^14, 2^15) by a power of two, exactly, and back
      // at the end: a rank 2^-22 below the largest still has its 16 bits, and what is off
      // of any is 2^-39 of the largest.  (At [1, 2) a rank lost bits from 2^-9 on.)
      float up = 1.f;
      if constexpr (DT == 2) {
        big = fmaxf(big, __shfl_xor(big, 16, 64));
        big = fmaxf(big, __shfl_xor(big, 32, 64));
        const int e = big > 0.f && big < INFINITY ? (big < 0x1p-112f ? -112 : ilogbf(big)) : 14;
        up = ldexpf(1.f, e - 14);
        const float down = ldexpf(1.f, 14 - e);
#pragma unroll
        for (int s = 0; s < RT; ++s)
#pragma unroll
          for (int j = 0; j < KE; ++j) v[s][j] *= down;
      }
      u32x4_t f[RT];
#pragma unroll
      for (int s = 0; s < RT; ++s) {
        f[s] = narrow<DT>(v[s]);
        if constexpr (DT != 0) {
          float rest[KE];
          widen<DT>(f[s], rest);
#pragma unroll
          for (int j = 0; j < KE; ++j) rest[j] = v[s][j] - rest[j];
          const u32x4_t lo = narrow<DT>(rest);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[s][j] = 4 * s + g4 < 2 * RT ? f[s][j] : lo[j];
        }
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        f32x4_t acc[4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int s = 0; s < RT; ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] = mma<DT>(qb[c][q][s], f[s], acc[q]);
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
          const int left = a.N - col - 4 * KE * (c * Q + j);
          if (!whole && left <= 0) continue;
          float o[KE];
          u32x4_t old = {0, 0, 0, 0};
          if (a.base) old = whole ? y[buf][c][j] : load_part<DT>((const char*)a.base + at + 64 * (c * Q + j), left);
          widen<DT>(old, o);
#pragma unroll
          for (int i = 0; i < KE; ++i) o[i] = fmaf(acc[(j * KE + i) / 4][i % 4], up, o[i]);
          char* to = (char*)a.out + at + 64 * (c * Q + j);
          if (whole) store16<DT>(to, narrow<DT>(o));
          else store_part<DT>(to, narrow<DT>(o), left);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    words(0, row0);
    words(1, row0 + 16);
    // Columns: access j of a lane in block c is KE neighbours from column base + 64 c
    // + 4 KE j + KE g4 on (64 bytes a row and access), results q = j KE / 4 + h its
    // elements 4 h + 0..3.
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = base + 64 * c + 4 * KE * (4 * q / KE) + KE * (i16 >> 2) + 4 * q % KE + (i16 & 3);
        const char* from = (const char*)a.B + ((int64_t)t.g * a.N + (n < a.N ? n : a.N - 1)) * a.r * S;
#pragma unroll
        for (int s = 0; s < RT; ++s) {
          const int r0 = rank_of(s);
          qb[c][q][s] = a.r % KE == 0 ? load16<DT>(from + (r0 < a.r ? r0 : 0) * S)
                                      : load_part<DT>(from + r0 * S, r0 < a.r ? a.r - r0 : 0);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
    load(0, row0);
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int s = 0; s < RT; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) qb[c][q][s][j] = rank_of(s) < a.r ? qb[c][q][s][j] : 0u;
    for (int r = row0; r < t.end; r += 32) {
      load(1, r + 16);
      words(0, r + 32);
      work(0, r);
      load(0, r + 32);
      words(1, r + 48);
      if (r + 16 < t.end) work(1, r + 16);
    }
    row0 = t.end;
  }
#endif
}

// ------------------------------------------------------------------ grad
constexpr int kGradWaves = 4;

// Where a range leaves its sum of a group that others share: in place 0 if the
// group began before it, else in place 1 (of the ranges' two each no group but
// the first and the last of a range wants one).
__device__ __forceinline__ int64_t grad_place(int ranges, int range, bool began, int frags) {
  const int64_t unit = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  return ((unit * ranges + range) * 2 + began) * frags * 64;
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

// grid: (slabs of 16 KE columns of the wider matrix, ranges of rows, matrix and RT
// rank tiles).  A group that lies in one range is written at once; of one that does
// not each range leaves its sum for lora_grad_sum_kernel, which adds them in order.
template <int DT, int RT, bool FULL> __global__ __launch_bounds__(64 * kGradWaves) void lora_grad_kernel(LoraGrad a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, S = Elem<DT>::kBytes, COLS = 16 * KE, U = 4, ROUND = 4 * kGradWaves;
  __shared__ f32x4_t red[kGradWaves / 2][RT][KE][64];
  const int lane = lane_id(), w = wave_id(), i16 = lane & 15, g4 = lane >> 4;
  const int mat = blockIdx.z & 1, q0 = (blockIdx.z >> 1) * RT;
  const int W = a.width[mat];
  if ((int)blockIdx.x * COLS >= W) return;
  const int ranges = gridDim.y;
  const Rows rows = rows_of(a.map, ranges);
  const int begin = rows.begin(blockIdx.y), end = rows.begin(blockIdx.y + 1);
  // a lane whose columns end outside takes the last KE, its neighbour's again:
  // both write the same sums (W < KE: columns past W read one by one below)
  const int at = blockIdx.x * COLS + i16 * KE, last = W > KE ? W - KE : 0;
  const int col = at < last ? at : last;
  const char* wide = (const char*)a.wide[mat] + (int64_t)col * S;
  const float* v = a.v[mat];
  const int vw = mat == 0 ? lora_width(a.r) : a.r;  // floats of a row of v
  int rank[RT];
#pragma unroll
  for (int q = 0; q < RT; ++q) rank[q] = 16 * (q0 + q) + i16 < a.r ? 16 * (q0 + q) + i16 : a.r - 1;
  for (int row0 = begin; row0 < end;) {
    const Part t = part_at(a.map, rows, row0, end);
    const int lo = row0, hi = t.end;
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
    if (w == 0) {
      if (t.lo < begin || t.hi > end) {
        f32x4_t* part = (f32x4_t*)a.part + grad_place(ranges, blockIdx.y, t.lo >= begin, RT * KE) + lane;
#pragma unroll
        for (int q = 0; q < RT; ++q)
#pragma unroll
          for (int j = 0; j < KE; ++j) part[(q * KE + j) * 64] = acc[q][j];
      } else {
        write_grad<DT, RT>(a, t.g, mat, q0, at, col, acc);
      }
    }
    row0 = hi;
  }
#endif
}

// One wave for each slab, group, matrix and rank tiles.
template <int DT, int RT> __global__ __launch_bounds__(64) void lora_grad_sum_kernel(LoraGrad a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KE = kFragElems<DT>, COLS = 16 * KE;
  const int lane = lane_id(), i16 = lane & 15;
  const int mat = blockIdx.z & 1, q0 = (blockIdx.z >> 1) * RT, g = blockIdx.y;
  const int W = a.width[mat];
  if ((int)blockIdx.x * COLS >= W) return;
  const Rows rows = rows_of(a.map, a.ranges);
  const int lo = rows.in(a.map.offsets[g]), hi = rows.in(a.map.offsets[g + 1]);
  if (hi <= lo) return;
  const int r0 = rows.range_of(lo), r1 = rows.range_of(hi - 1);
  if (r0 == r1) return;
  const int at = blockIdx.x * COLS + i16 * KE, last = W > KE ? W - KE : 0;
  f32x4_t acc[RT][KE];
#pragma unroll
  for (int q = 0; q < RT; ++q)
#pragma unroll
    for (int j = 0; j < KE; ++j) acc[q][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int r = r0; r <= r1; ++r) {
    const f32x4_t* part = (const f32x4_t*)a.part + grad_place(a.ranges, r, r == r0, RT * KE) + lane;
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int j = 0; j < KE; ++j) acc[q][j] += part[(q * KE + j) * 64];
  }
  write_grad<DT, RT>(a, g, mat, q0, at, at < last ? at : last, acc);
#endif
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
  const Span span = span_of(a.map, a.map.offsets[0], a.map.offsets[a.map.G]);
  if (span.in(a.map.offsets[blockIdx.y + 1]) <= span.in(a.map.offsets[blockIdx.y])) {
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

int rank_tiles(int r) { return r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : 8; }

// How the rank kernel shares the rows out.  A workgroup's time is mostly one pass
// over K, whatever its rows, so none should make two where others make one: tiles
// of one group, as low as leaves no compute unit a workgroup more than the others
// (one each up to 48 rows, else two), counted for the worst places of the groups'
// ends.  Where the rows want more passes anyhow, even ranges of rows across groups.
struct RankShare {
  int height, places;  // height 0: ranges
};
RankShare rank_share(int rows, int G, int r) {
  const int most = r > 64 ? 32 : 64;  // rows of a pass
  for (int n = 1; n <= 2; ++n) {
    const int free = n * kNumCUs - G;
    if (free <= 0) continue;
    int h = (int)(((int64_t)rows + free - 1) / free);
    h = h < 16 ? 16 : h;
    if (h <= (n == 1 && most > 48 ? 48 : most)) {
      const int tiles = (rows + h - 1) / h + G;
      return RankShare{h, tiles < rows ? tiles : rows};
    }
  }
  if (rows <= 16 * (int64_t)G) return RankShare{16, (rows + 15) / 16 + G < rows ? (rows + 15) / 16 + G : rows};
  return RankShare{0, 2 * kNumCUs};
}

template <int DT, int RT, int M> hipError_t rank_m(const LoraRank& a, int places, hipStream_t s) {
  const dim3 grid((places + 7) / 8 * 8, a.splits);
  if (DT != 0 && a.K % 2)
    hipLaunchKernelGGL((lora_rank_kernel<DT, RT, M, DT != 0>), grid, dim3(64 * kRankWaves), 0, s, a);
  else
    hipLaunchKernelGGL((lora_rank_kernel<DT, RT, M, false>), grid, dim3(64 * kRankWaves), 0, s, a);
  return hipGetLastError();
}
template <int DT, int RT> hipError_t rank_of(const LoraRank& b, hipStream_t s) {
  LoraRank a = b;
  const RankShare share = rank_share(a.map.rows, a.map.G, a.r);
  a.height = share.height;
  a.ranges = share.places;
  const int each = share.height ? share.height : 64;
  if (each <= 16) return rank_m<DT, RT, 1>(a, share.places, s);
  if constexpr (RT < 8) {  // more than two tiles of rank 128 want too many registers
    if (each > 48) return rank_m<DT, RT, 4>(a, share.places, s);
    if (each > 32) return rank_m<DT, RT, 3>(a, share.places, s);
  }
  return rank_m<DT, RT, 2>(a, share.places, s);
}

template <int DT, int RT> hipError_t add_of(const LoraAdd& a, hipStream_t s) {
  const int64_t blocks = (a.N + 64 * kAddBlocks<DT, RT> - 1) / (64 * kAddBlocks<DT, RT>);
  // twelve waves a compute unit (eight 39 us, sixteen 41 at 8192 x 4096 of rank 16, bf16;
  // fp16 and ranks past 16 have registers for eight or four), but no less than a row each
  int64_t ranges = (12 * kNumCUs + blocks - 1) / blocks;
  if (ranges > a.map.rows) ranges = a.map.rows;
  int bare = a.map.row_of_pair && a.out != a.base
                 ? (a.map.rows + 8 * kBareTokens * kAddWaves - 1) / (8 * kBareTokens * kAddWaves) * 8
                 : 0;
  if (bare > kBareWorkgroups) bare = kBareWorkgroups;
  hipLaunchKernelGGL((lora_add_kernel<DT, RT>), dim3((unsigned)((blocks * ranges + 8 * kAddWaves - 1) / (8 * kAddWaves) * 8 + bare)),
                     dim3(64 * kAddWaves), 0, s, a, (int)ranges, bare);
  return hipGetLastError();
}

int grad_tiles(int r) { return r <= 16 ? 1 : 2; }  // rank tiles of a workgroup of the grad kernel
int grad_slabs(int K, int N, int dtype) {
  const int cols = dtype == 0 ? 16 * kFragElems<0> : 16 * kFragElems<1>;
  return ((K > N ? K : N) + cols - 1) / cols;
}
int grad_units(int r) { return 2 * ((r + 16 * grad_tiles(r) - 1) / (16 * grad_tiles(r))); }

template <int DT, int RT> hipError_t grad_of(const LoraGrad& a, hipStream_t s) {
  const int slabs = grad_slabs(a.width[0], a.width[1], DT), units = grad_units(a.r);
  const dim3 grid(slabs, a.ranges, units);
  // FULL: a row of each matrix holds a whole 16-byte access
  if (a.width[0] >= kFragElems<DT> && a.width[1] >= kFragElems<DT>)
    hipLaunchKernelGGL((lora_grad_kernel<DT, RT, true>), grid, dim3(64 * kGradWaves), 0, s, a);
  else
    hipLaunchKernelGGL((lora_grad_kernel<DT, RT, false>), grid, dim3(64 * kGradWaves), 0, s, a);
  if (a.ranges > 1)
    hipLaunchKernelGGL((lora_grad_sum_kernel<DT, RT>), dim3(slabs, a.map.G, units), dim3(64), 0, s, a);
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
  if (rows == 0) return 1;
  // two workgroups a compute unit where the rows do not fill half of them, for each
  // share is read again by the add kernel; four K steps or more for each wave
  const int places = rank_share(rows, G, r).places;
  const int n = places > kNumCUs / 2 ? 1 : 2 * kNumCUs / places, each = K / (dtype == 0 ? 16 : 32) / (4 * kRankWaves);
  return each < 1 ? 1 : n > each ? (each > 16 ? 16 : each) : n > 16 ? 16 : n;
}

LoraGradPlan lora_grad_plan(int rows, int G, int r, int K, int N, int dtype) {
  const int cols = dtype == 0 ? 16 * kFragElems<0> : 16 * kFragElems<1>;
  // three workgroups a compute unit, but 128 rows each or more, or a group (44 rows
  // of 36 adapters, 256 to 3930 columns: 130 us by one range, for each group is a pass)
  const int64_t slabs = (K + cols - 1) / cols + (N + cols - 1) / cols;
  int64_t n = 3 * kNumCUs / slabs;
  const int64_t most = rows / 128 > G ? rows / 128 : rows < G ? rows : G;
  if (n > most) n = most;
  LoraGradPlan p;
  p.ranges = n < 1 ? 1 : (int)n;
  p.part_bytes = p.ranges > 1 ? (int64_t)p.ranges * 2 * grad_units(r) * grad_slabs(K, N, dtype) * grad_tiles(r) *
                                    (cols / 16) * 64 * 16
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
