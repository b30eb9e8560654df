// Token rows to their experts' rows and back, with the gates applied, as
// operators of their own (the dispatch and the weighted combine of the layer:
// kucoin.com, "Cursor's MoK réalise une amélioration des performances de 2,37x
// sur NVIDIA GB300 NVL72", sections 01 and 03), and their gradients:
//   permute    xp[row(t,j)] = w_tj x_t      unpermute  out_t = sum_j w_tj y[row(t,j)]
//   gradients  dx_t = sum_j w_tj dxp[row]              dy[row(t,j)] = w_tj dout_t
//              dw_tj = <x_t, dxp[row]>                 dw_tj = <dout_t, y[row]>
// so two passes over the tokens serve all four: `scatter` (one row read, its k
// rows written) and `gather` (k rows read, one written), each with the dot
// products on the way where a gradient of the gates is asked for.  A pair
// without a row (row -1, or outside the buffer) is skipped: it adds nothing,
// its dot product is 0, and no row but those of the map is written.  Products
// and sums in fp32, slots ascending, one rounding; dot products by a fixed
// tree.  Without a gate a scatter copies the bits.
//
// Bound by HBM: every row is read or written once.
#include "elem.h"
#include "pair_ops.h"

namespace mok {
namespace {

// A row as a buffer resource: row_bytes bytes, or none for a pair without a
// row, whose loads then return zeros and whose stores are dropped.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t row_of(const void* base, int64_t r, int row_bytes) {
  const char* p = (const char*)base + (r >= 0 ? r * row_bytes : 0);
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, r >= 0 ? row_bytes : 0, 0x00020000);
}

// The same, made again at each 16-byte access: eight rows' resources held
// across the loop do not fit the scalar registers (the way back's gradient of
// 1777 x 1411 fp32 33.0 -> 28.2 us).  A loop of narrow accesses is longer and
// keeps them (4096 x 1411 bf16 back: 32.1 us, 35.8 made again).
template <int VE> __device__ __forceinline__ rsrc_t row_here(const void* base, int32_t r, int row_bytes) {
  if constexpr (VE > 1) asm volatile("" : "+s"(r));
  return row_of(base, r, row_bytes);
}

// VE elements from element `at` of a row.  Accesses of 4 bytes and more need
// their address on 4 bytes only.
template <int AUX, int DT, int VE> __device__ __forceinline__ Vec<DT, VE> load(rsrc_t rs, int at) {
  typedef Vec<DT, VE> V;
  V o;
  const int off = at * Elem<DT>::kBytes;
  if constexpr (V::kB == 16) {
    const auto u = __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, AUX);
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = u[i];
  } else if constexpr (V::kB == 4) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, AUX);
  } else {
    o.w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, AUX);
  }
  return o;
}
template <int DT, int VE> __device__ __forceinline__ void store(rsrc_t rs, int at, const Vec<DT, VE>& o) {
  typedef Vec<DT, VE> V;
  const int off = at * Elem<DT>::kBytes;
  if constexpr (V::kB == 16) {
    __builtin_amdgcn_raw_buffer_store_b128(
        decltype(__builtin_amdgcn_raw_buffer_load_b128(rs, 0, 0, 0)){o.w[0], o.w[1], o.w[2], o.w[3]}, rs, off, 0, 0);
  } else if constexpr (V::kB == 4) {
    __builtin_amdgcn_raw_buffer_store_b32(o.w[0], rs, off, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16((unsigned short)o.w[0], rs, off, 0, 0);
  }
}

// f(at, width) over a row of d elements by TPT threads: VE elements at a time,
// then what is left of a row of whole dwords a dword at a time.  VE = 1 for
// rows of an odd number of 16-bit elements, which share dwords.
template <int N> struct Width { static constexpr int value = N; };
template <int DT, int VE, int TPT, typename F> __device__ __forceinline__ void over_row(int d, int tid, const F& f) {
  constexpr int VT = VE == 1 ? 1 : 4 / Elem<DT>::kBytes;
  const int nv = d / VE;
  for (int v = tid; v < nv; v += TPT) f(v * VE, Width<VE>{});
  if constexpr (VE > VT) {
    const int at = nv * VE + tid * VT;
    if (at < d) f(at, Width<VT>{});
  }
}

// The rows and gates of slots [j0, j0 + NS) of one token, the same for every
// thread working on it.
template <int NS> struct Slots {
  int32_t r[NS];  // -1: no row
  float w[NS];
};
template <int NS>
__device__ __forceinline__ Slots<NS> slots_of(const PairRows& p, const int32_t* __restrict__ rop,
                                              const float* __restrict__ gate, int64_t t, int j0) {
  Slots<NS> s;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int64_t q = t * p.k + (j0 + i < p.k ? j0 + i : p.k - 1);  // clamped: all loads issued at once
    const int32_t r = rop[q];
    const float g = gate ? gate[q] : 1.0f;
    const bool live = j0 + i < p.k && r >= 0 && r < p.nrows;
    s.r[i] = live ? r : -1;
    s.w[i] = live ? g : 0.f;
  }
  return s;
}

// Sum over the TPT threads of a token; valid in its first thread.
template <int TPT, int NS> __device__ __forceinline__ void token_sums(float (&part)[NS], float (*red)[NS]) {
#pragma unroll
  for (int i = 0; i < NS; ++i) part[i] = wave_sum(part[i]);
  if constexpr (TPT > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the sums of the slots before are read
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) red[w][i] = part[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) part[i] = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
  }
}

template <int TPT, int NS>
__device__ __forceinline__ void store_dots(const PairRows& p, int64_t t, int j0, const Slots<NS>& s,
                                           const float (&part)[NS]) {
  const int tid = TPT == 64 ? lane_id() : threadIdx.x;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (tid == i && j0 + i < p.k) p.dot[t * p.k + j0 + i] = s.r[i] >= 0 ? part[i] : 0.f;
}

// TPT threads per token (a wave, or the workgroup's four).
template <int DT, int VE, int TPT, int NS, bool GATED, bool DOT>
__global__ __launch_bounds__(256) void scatter_kernel(PairRows p, const int32_t* __restrict__ rop,
                                                      const float* __restrict__ gate) {
  __shared__ float red[4][NS];
  const int row_bytes = p.d * Elem<DT>::kBytes;
  const int tid = TPT == 64 ? lane_id() : threadIdx.x;
  const int sub = TPT == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  constexpr int kTok = 256 / TPT;
  for (int64_t t = (int64_t)blockIdx.x * kTok + sub; t < p.T; t += (int64_t)gridDim.x * kTok) {
    const rsrc_t ra = row_of(p.a, t, row_bytes);
    for (int j0 = 0; j0 < p.k; j0 += NS) {
      const Slots<NS> s = slots_of<NS>(p, rop, gate, t, j0);
      float part[NS] = {};
      over_row<DT, VE, TPT>(p.d, tid, [&](int at, auto width) {
        constexpr int W = decltype(width)::value;
        const Vec<DT, W> a = load<0, DT, W>(ra, at);
        Vec<DT, W> y[NS];
        if constexpr (DOT) {
#pragma unroll
          for (int i = 0; i < NS; ++i) y[i] = load<2, DT, W>(row_here<VE>(p.in, s.r[i], row_bytes), at);
        }
        float f[W];
        if constexpr (GATED || DOT) a.widen(f);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if constexpr (DOT) {
            float g[W];
            y[i].widen(g);
#pragma unroll
            for (int q = 0; q < W; ++q) part[i] = fmaf(f[q], g[q], part[i]);
          }
          if (s.r[i] < 0) continue;
          if constexpr (GATED) {
            float z[W];
#pragma unroll
            for (int q = 0; q < W; ++q) z[q] = s.w[i] * f[q];
            store(row_here<VE>(p.out, s.r[i], row_bytes), at, Vec<DT, W>::narrow(z));
          } else {
            store(row_here<VE>(p.out, s.r[i], row_bytes), at, a);
          }
        }
      });
      if constexpr (DOT) {
        token_sums<TPT>(part, red);
        store_dots<TPT>(p, t, j0, s, part);
      }
    }
  }
}

template <int DT, int VE, int TPT, int NS, bool DOT>
__global__ __launch_bounds__(256) void gather_kernel(PairRows p, const int32_t* __restrict__ rop,
                                                     const float* __restrict__ gate) {
  __shared__ float red[4][NS];
  const int row_bytes = p.d * Elem<DT>::kBytes;
  const int tid = TPT == 64 ? lane_id() : threadIdx.x;
  const int sub = TPT == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  constexpr int kTok = 256 / TPT;
  for (int64_t t = (int64_t)blockIdx.x * kTok + sub; t < p.T; t += (int64_t)gridDim.x * kTok) {
    const rsrc_t ra = row_of(p.a, DOT ? t : -1, row_bytes);
    const rsrc_t ro = row_of(p.out, t, row_bytes);
    const Slots<NS> s0 = slots_of<NS>(p, rop, gate, t, 0);
    float part[NS] = {};
    over_row<DT, VE, TPT>(p.d, tid, [&](int at, auto width) {
      constexpr int W = decltype(width)::value;
      float acc[W] = {};
      for (int j0 = 0; j0 < p.k; j0 += NS) {
        Vec<DT, W> y[NS];
        float w[NS];
        if (j0 == 0) {
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            y[i] = load<2, DT, W>(row_here<VE>(p.in, s0.r[i], row_bytes), at);
            w[i] = s0.w[i];
          }
        } else {
          const Slots<NS> s = slots_of<NS>(p, rop, gate, t, j0);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            y[i] = load<2, DT, W>(row_of(p.in, s.r[i], row_bytes), at);
            w[i] = s.w[i];
          }
        }
        float f[W];
        if constexpr (DOT)
          if (j0 == 0) load<0, DT, W>(ra, at).widen(f);
        // a slot without a row adds 0 * 0 to a sum that is never -0
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          float g[W];
          y[i].widen(g);
#pragma unroll
          for (int q = 0; q < W; ++q) acc[q] = fmaf(w[i], g[q], acc[q]);
          if constexpr (DOT)
            if (j0 == 0)
#pragma unroll
              for (int q = 0; q < W; ++q) part[i] = fmaf(f[q], g[q], part[i]);
        }
      }
      store(ro, at, Vec<DT, W>::narrow(acc));
    });
    if constexpr (DOT) {
      token_sums<TPT>(part, red);
      store_dots<TPT>(p, t, 0, s0, part);
      // the dot products of the slots past the first eight: their rows again
      for (int j0 = NS; j0 < p.k; j0 += NS) {
        const Slots<NS> s = slots_of<NS>(p, rop, gate, t, j0);
#pragma unroll
        for (int i = 0; i < NS; ++i) part[i] = 0.f;
        over_row<DT, VE, TPT>(p.d, tid, [&](int at, auto width) {
          constexpr int W = decltype(width)::value;
          float f[W];
          load<0, DT, W>(ra, at).widen(f);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            float g[W];
            load<0, DT, W>(row_of(p.in, s.r[i], row_bytes), at).widen(g);
#pragma unroll
            for (int q = 0; q < W; ++q) part[i] = fmaf(f[q], g[q], part[i]);
          }
        });
        token_sums<TPT>(part, red);
        store_dots<TPT>(p, t, j0, s, part);
      }
    }
  }
}

// Threads per token: a wave while a row is at most two accesses of it, else
// the workgroup.
template <int TPT> int grid_of(int64_t T) {
  const int64_t n = (T + 256 / TPT - 1) / (256 / TPT);
  return (int)(n < 65536 ? n : 65536);
}

template <int DT, int VE, int TPT, int NS> hipError_t scatter_t(const PairRows& p, hipStream_t s) {
  const dim3 g(grid_of<TPT>(p.T)), b(256);
#define MOK_SCATTER(GATED, DOT) \
  hipLaunchKernelGGL((scatter_kernel<DT, VE, TPT, NS, GATED, DOT>), g, b, 0, s, p, p.rop, p.gate)
  if (p.dot) {
    if (p.gate) MOK_SCATTER(true, true); else MOK_SCATTER(false, true);
  } else {
    if (p.gate) MOK_SCATTER(true, false); else MOK_SCATTER(false, false);
  }
#undef MOK_SCATTER
  return hipGetLastError();
}
template <int DT, int VE, int TPT, int NS> hipError_t gather_t(const PairRows& p, hipStream_t s) {
  const dim3 g(grid_of<TPT>(p.T)), b(256);
  if (p.dot) hipLaunchKernelGGL((gather_kernel<DT, VE, TPT, NS, true>), g, b, 0, s, p, p.rop, p.gate);
  else hipLaunchKernelGGL((gather_kernel<DT, VE, TPT, NS, false>), g, b, 0, s, p, p.rop, p.gate);
  return hipGetLastError();
}

template <int DT, int VE, int NS> hipError_t run(const PairRows& p, bool scatter, hipStream_t s) {
  const bool wave = p.d / VE <= 128;
  if (scatter) return wave ? scatter_t<DT, VE, 64, NS>(p, s) : scatter_t<DT, VE, 256, NS>(p, s);
  return wave ? gather_t<DT, VE, 64, NS>(p, s) : gather_t<DT, VE, 256, NS>(p, s);
}

// Slots whose rows are in flight together: as many as a token has, up to
// eight (one slot in eight's place, 8192 x 4096 bf16: 26 against 38 us back,
// 35 against 53 us with the gradient).
template <int DT, int VE> hipError_t run_k(const PairRows& p, bool scatter, hipStream_t s) {
  if (p.k == 1) return run<DT, VE, 1>(p, scatter, s);
  if (p.k == 2) return run<DT, VE, 2>(p, scatter, s);
  return p.k <= 4 ? run<DT, VE, 4>(p, scatter, s) : run<DT, VE, 8>(p, scatter, s);
}

// 16-byte accesses on rows of whole dwords, else (an odd number of 16-bit
// elements) single elements.
hipError_t dispatch(const PairRows& p, bool scatter, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  switch (p.dtype) {
    case kF32: return run_k<kF32, 4>(p, scatter, s);
    case kBF16: return p.d % 2 ? run_k<kBF16, 1>(p, scatter, s) : run_k<kBF16, 8>(p, scatter, s);
    case kF16: return p.d % 2 ? run_k<kF16, 1>(p, scatter, s) : run_k<kF16, 8>(p, scatter, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_scatter_rows(const PairRows& p, hipStream_t s) { return dispatch(p, true, s); }
hipError_t launch_gather_rows(const PairRows& p, hipStream_t s) { return dispatch(p, false, s); }

}  // namespace mok
