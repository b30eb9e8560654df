// Token-expert pairs sorted by expert for a caller's own routing: the layout
// step of the layer (kucoin.com, "Cursor's MoK réalise une amélioration des
// performances de 2,37x sur NVIDIA GB300 NVL72", section 01: count each
// expert's tokens, then place them, one expert's rows together) as an operator
// of its own.  Pair p = t k + j of expert e goes to row
//   offsets[e] + #{q < p : e(q) = e},
// integers only, so the result is exact and the same on every run.
//
// A workgroup of sixteen waves walks one chunk of pairs once: lanes holding
// the same expert find each other by a ballot per expert-id bit, the lowest of
// them advances the wave's count of that expert in LDS, and a pair's rank
// inside its wave is the count before plus the lower lanes'.  The counts'
// prefix over waves, chunks and experts turns ranks into rows.  Bound by
// latency: 4 bytes read and 8 written per pair.
#include "elem.h"
#include "pair_ops.h"

namespace mok {
namespace {

__device__ __forceinline__ uint64_t same_expert(int e, bool valid, int nbits) {
  uint64_t m = __ballot(valid);
  for (int b = 0; b < nbits; ++b) {
    const bool bit = (e >> b) & 1;
    const uint64_t bm = __ballot(bit);
    m &= bit ? bm : ~bm;
  }
  return m;
}

// Orders the LDS accesses of one wave's lanes around it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct SortShared {
  int32_t cnt[16][1024];  // pairs of expert e in wave w
  int32_t wsum[16];
  int32_t total;
};

// Ranks of a chunk's pairs inside their waves and each wave's counts.  The
// pairs of wave w are the kSortIters * 64 from base + w * kSortIters * 64.
__device__ __forceinline__ void walk(SortShared& sh, const int32_t* __restrict__ idx, int64_t P, int64_t base, int E,
                                     int eb, int ee, int nbits, int (&ev)[kSortIters], int (&rank)[kSortIters]) {
  const int w = threadIdx.x >> 6, lane = lane_id();
  const uint64_t lt = lane == 0 ? 0ull : (~0ull >> (64 - lane));
#pragma unroll
  for (int it = 0; it < kSortIters; ++it) {
    const int64_t p = base + ((int64_t)w * kSortIters + it) * 64 + lane;
    ev[it] = p < P ? idx[p] : -1;
  }
  for (int e = lane; e < E; e += 64) sh.cnt[w][e] = 0;
  wave_sync();
#pragma unroll
  for (int it = 0; it < kSortIters; ++it) {
    const int e = ev[it];
    const bool valid = e >= eb && e < ee;
    const uint64_t m = same_expert(e, valid, nbits);
    const int before = valid ? sh.cnt[w][e] : 0;
    rank[it] = valid ? before + __popcll(m & lt) : -1;
    wave_sync();
    if (valid && lane == __ffsll((unsigned long long)m) - 1) sh.cnt[w][e] = before + __popcll(m);
    wave_sync();
  }
}

// Exclusive prefix over the workgroup's 1024 threads; the sum in sh.total.
__device__ __forceinline__ int block_prefix(SortShared& sh, int v) {
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const int x = wave_prefix(v);
  if (lane == 63) sh.wsum[w] = x;
  __syncthreads();
  int base = 0, tot = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int s = sh.wsum[q];
    base += q < w ? s : 0;
    tot += s;
  }
  if (threadIdx.x == 0) sh.total = tot;
  return base + x - v;
}

// Chunk c's pairs per expert into table[c, e].
__global__ __launch_bounds__(1024) void count_kernel(const int32_t* __restrict__ idx, int64_t P, int E, int eb, int ee,
                                                     int nbits, int32_t* __restrict__ table) {
  __shared__ SortShared sh;
  int ev[kSortIters], rank[kSortIters];
  walk(sh, idx, P, (int64_t)blockIdx.x * kPairChunk, E, eb, ee, nbits, ev, rank);
  __syncthreads();
  const int e = threadIdx.x;
  if (e < E) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) n += sh.cnt[w][e];
    table[(int64_t)blockIdx.x * E + e] = n;
  }
}

// Long tables: one workgroup per expert replaces its column by the column's
// exclusive prefix and writes the expert's total.
__global__ __launch_bounds__(256) void column_prefix_kernel(int32_t* __restrict__ table, int64_t nch, int E,
                                                            int32_t* __restrict__ counts) {
  __shared__ int32_t wsum[4];
  const int e = blockIdx.x, lane = lane_id(), w = threadIdx.x >> 6;
  int carry = 0;
  for (int64_t c0 = 0; c0 < nch; c0 += 256) {
    const int64_t c = c0 + threadIdx.x;
    const int v = c < nch ? table[c * E + e] : 0;
    const int x = wave_prefix(v);
    if (lane == 63) wsum[w] = x;
    __syncthreads();
    int base = carry;
    for (int q = 0; q < w; ++q) base += wsum[q];
    if (c < nch) table[c * E + e] = base + x - v;
    carry += wsum[0] + wsum[1] + wsum[2] + wsum[3];
    __syncthreads();
  }
  if (threadIdx.x == 0) counts[e] = carry;
}

// Rows of chunk c's pairs.  MODE 0: the one chunk of a small call; 1: the
// table holds every chunk's counts, summed here; 2: it holds their prefix over
// the chunks and `counts` the totals.
template <int MODE>
__global__ __launch_bounds__(1024) void place_kernel(const int32_t* __restrict__ idx, int64_t P, int E, int eb, int ee,
                                                     int nbits, const int32_t* __restrict__ table, int nch,
                                                     int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                     int32_t* __restrict__ row_of_pair,
                                                     int32_t* __restrict__ pair_of_row) {
  __shared__ SortShared sh;
  const int c = blockIdx.x, e = threadIdx.x, w = threadIdx.x >> 6, lane = lane_id();
  const int64_t base = (int64_t)c * kPairChunk;
  int ev[kSortIters], rank[kSortIters];
  // pairs of expert e in every chunk, and in the chunks before c
  int total = 0, before = 0;
  if (MODE == 1 && e < E) {
#pragma unroll 8
    for (int q = 0; q < nch; ++q) {
      const int v = table[(int64_t)q * E + e];
      total += v;
      before += q < c ? v : 0;
    }
  }
  if (MODE == 2 && e < E) {
    total = counts[e];
    before = table[(int64_t)c * E + e];
  }
  walk(sh, idx, P, base, E, eb, ee, nbits, ev, rank);
  __syncthreads();
  if (MODE == 0 && e < E) {
#pragma unroll
    for (int q = 0; q < 16; ++q) total += sh.cnt[q][e];
  }
  const int off = block_prefix(sh, total);  // a barrier: the sums above are done
  if (e < E) {
    int r = off + before;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int n = sh.cnt[q][e];
      sh.cnt[q][e] = r;  // first row of wave q's pairs of expert e
      r += n;
    }
    if (c == 0) {
      if (MODE != 2) counts[e] = total;
      offsets[e] = off;
      if (e == E - 1) offsets[E] = off + total;
    }
  }
  __syncthreads();
  const int local = sh.total;
#pragma unroll
  for (int it = 0; it < kSortIters; ++it) {
    const int64_t p = base + ((int64_t)w * kSortIters + it) * 64 + lane;
    if (p >= P) continue;
    const int row = rank[it] < 0 ? -1 : sh.cnt[w][ev[it]] + rank[it];
    row_of_pair[p] = row;
    if (row >= 0) pair_of_row[row] = (int32_t)p;
    if (p >= local) pair_of_row[p] = -1;  // rows past the last local pair
  }
}

}  // namespace

hipError_t launch_sort_pairs(const int32_t* idx, int64_t P, int E, int eb, int ee, int32_t* counts, int32_t* offsets,
                             int32_t* row_of_pair, int32_t* pair_of_row, int32_t* table, hipStream_t s) {
  int nbits = 0;
  while ((1 << nbits) < E) ++nbits;
  const int64_t nch = (P + kPairChunk - 1) / kPairChunk;
  if (nch <= 1) {
    hipLaunchKernelGGL(place_kernel<0>, dim3(1), dim3(1024), 0, s, idx, P, E, eb, ee, nbits, table, 1, counts, offsets,
                       row_of_pair, pair_of_row);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(count_kernel, dim3((unsigned)nch), dim3(1024), 0, s, idx, P, E, eb, ee, nbits, table);
  if (nch <= kSelfScanChunks) {
    hipLaunchKernelGGL(place_kernel<1>, dim3((unsigned)nch), dim3(1024), 0, s, idx, P, E, eb, ee, nbits, table,
                       (int)nch, counts, offsets, row_of_pair, pair_of_row);
  } else {
    hipLaunchKernelGGL(column_prefix_kernel, dim3(E), dim3(256), 0, s, table, nch, E, counts);
    hipLaunchKernelGGL(place_kernel<2>, dim3((unsigned)nch), dim3(1024), 0, s, idx, P, E, eb, ee, nbits, table,
                       (int)nch, counts, offsets, row_of_pair, pair_of_row);
  }
  return hipGetLastError();
}

}  // namespace mok
