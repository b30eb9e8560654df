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

constexpr int kSlots = 8;  // slots whose rows are in flight together

// A row as a buffer resource: row_bytes bytes, or none for a pair without a
// row, whose loads then return zeros and whose stores are dropped.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t row_of(const void* base, int64_t r, int row_bytes) {
  const char* p = (const char*)base + (r >= 0 ? r * row_bytes : 0);
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, r >= 0 ? row_bytes : 0, 0x00020000);
}

template <int AUX, int DT, int VE> __device__ __forceinline__ Vec<DT, VE> load(rsrc_t rs, int v) {
  typedef Vec<DT, VE> V;
  V o;
  if constexpr (V::kB == 16) {
    const auto u = __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * v, 0, AUX);
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = u[i];
  } else if constexpr (V::kB == 4) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * v, 0, AUX);
  } else {
    o.w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, 2 * v, 0, AUX);
  }
  return o;
}
template <int DT, int VE> __device__ __forceinline__ void store(rsrc_t rs, int v, const Vec<DT, VE>& o) {
  typedef Vec<DT, VE> V;
  if constexpr (V::kB == 16) {
    __builtin_amdgcn_raw_buffer_store_b128(
        decltype(__builtin_amdgcn_raw_buffer_load_b128(rs, 0, 0, 0)){o.w[0], o.w[1], o.w[2], o.w[3]}, rs, 16 * v, 0, 0);
  } else if constexpr (V::kB == 4) {
    __builtin_amdgcn_raw_buffer_store_b32(o.w[0], rs, 4 * v, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16((unsigned short)o.w[0], rs, 2 * v, 0, 0);
  }
}

// The rows and gates of slots [j0, j0 + 8) of one token, the same for every
// thread working on it.
struct Slots {
  int64_t r[kSlots];
  float w[kSlots];
};
__device__ __forceinline__ Slots slots_of(const PairRows& p, const int32_t* __restrict__ rop,
                                          const float* __restrict__ gate, int64_t t, int j0) {
  Slots s;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
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
template <int TPT> __device__ __forceinline__ void token_sums(float (&part)[kSlots], float (*red)[kSlots]) {
#pragma unroll
  for (int i = 0; i < kSlots; ++i) part[i] = wave_sum(part[i]);
  if constexpr (TPT > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the sums of the slots before are read
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < kSlots; ++i) red[w][i] = part[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) part[i] = (red[0][i] + red[1][i]) + (red[2][i] + red[3][i]);
  }
}

template <int TPT> __device__ __forceinline__ void store_dots(const PairRows& p, int64_t t, int j0, const Slots& s,
                                                              const float (&part)[kSlots]) {
  const int tid = TPT == 64 ? lane_id() : threadIdx.x;
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (tid == i && j0 + i < p.k) p.dot[t * p.k + j0 + i] = s.r[i] >= 0 ? part[i] : 0.f;
}

// TPT threads per token (a wave, or the workgroup's four).
template <int DT, int VE, int TPT, bool GATED, bool DOT>
__global__ __launch_bounds__(256) void scatter_kernel(PairRows p, const int32_t* __restrict__ rop,
                                                      const float* __restrict__ gate) {
  __shared__ float red[4][kSlots];
  const int row_bytes = p.d * Elem<DT>::kBytes, nv = p.d / VE;
  const int tid = TPT == 64 ? lane_id() : threadIdx.x;
  const int sub = TPT == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  constexpr int kTok = 256 / TPT;
  for (int64_t t = (int64_t)blockIdx.x * kTok + sub; t < p.T; t += (int64_t)gridDim.x * kTok) {
    const rsrc_t ra = row_of(p.a, t, row_bytes);
    for (int j0 = 0; j0 < p.k; j0 += kSlots) {
      const Slots s = slots_of(p, rop, gate, t, j0);
      rsrc_t ro[kSlots], ri[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        ro[i] = row_of(p.out, s.r[i], row_bytes);
        if constexpr (DOT) ri[i] = row_of(p.in, s.r[i], row_bytes);
      }
      float part[kSlots] = {};
      for (int v = tid; v < nv; v += TPT) {
        const Vec<DT, VE> a = load<0, DT, VE>(ra, v);
        Vec<DT, VE> y[kSlots];
        if constexpr (DOT) {
#pragma unroll
          for (int i = 0; i < kSlots; ++i) y[i] = load<2, DT, VE>(ri[i], v);
        }
        float f[VE];
        if constexpr (GATED || DOT) a.widen(f);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          if constexpr (DOT) {
            float g[VE];
            y[i].widen(g);
#pragma unroll
            for (int q = 0; q < VE; ++q) part[i] = fmaf(f[q], g[q], part[i]);
          }
          if (s.r[i] < 0) continue;
          if constexpr (GATED) {
            float z[VE];
#pragma unroll
            for (int q = 0; q < VE; ++q) z[q] = s.w[i] * f[q];
            store(ro[i], v, Vec<DT, VE>::narrow(z));
          } else {
            store(ro[i], v, a);
          }
        }
      }
      if constexpr (DOT) {
        token_sums<TPT>(part, red);
        store_dots<TPT>(p, t, j0, s, part);
      }
    }
  }
}

template <int DT, int VE, int TPT, bool DOT>
__global__ __launch_bounds__(256) void gather_kernel(PairRows p, const int32_t* __restrict__ rop,
                                                     const float* __restrict__ gate) {
  __shared__ float red[4][kSlots];
  const int row_bytes = p.d * Elem<DT>::kBytes, nv = p.d / VE;
  const int tid = TPT == 64 ? lane_id() : threadIdx.x;
  const int sub = TPT == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  constexpr int kTok = 256 / TPT;
  for (int64_t t = (int64_t)blockIdx.x * kTok + sub; t < p.T; t += (int64_t)gridDim.x * kTok) {
    const rsrc_t ra = row_of(p.a, DOT ? t : -1, row_bytes);
    const rsrc_t ro = row_of(p.out, t, row_bytes);
    const Slots s0 = slots_of(p, rop, gate, t, 0);
    rsrc_t r0[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) r0[i] = row_of(p.in, s0.r[i], row_bytes);
    float part[kSlots] = {};
    for (int v = tid; v < nv; v += TPT) {
      float acc[VE] = {};
      for (int j0 = 0; j0 < p.k; j0 += kSlots) {
        Vec<DT, VE> y[kSlots], a;
        float w[kSlots];
        if (j0 == 0) {
#pragma unroll
          for (int i = 0; i < kSlots; ++i) {
            y[i] = load<2, DT, VE>(r0[i], v);
            w[i] = s0.w[i];
          }
        } else {
          const Slots s = slots_of(p, rop, gate, t, j0);
#pragma unroll
          for (int i = 0; i < kSlots; ++i) {
            y[i] = load<2, DT, VE>(row_of(p.in, s.r[i], row_bytes), v);
            w[i] = s.w[i];
          }
        }
        float f[VE];
        if constexpr (DOT)
          if (j0 == 0) {
            a = load<0, DT, VE>(ra, v);
            a.widen(f);
          }
        // a slot without a row adds 0 * 0 to a sum that is never -0
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          float g[VE];
          y[i].widen(g);
#pragma unroll
          for (int q = 0; q < VE; ++q) acc[q] = fmaf(w[i], g[q], acc[q]);
          if constexpr (DOT)
            if (j0 == 0)
#pragma unroll
              for (int q = 0; q < VE; ++q) part[i] = fmaf(f[q], g[q], part[i]);
        }
      }
      store(ro, v, Vec<DT, VE>::narrow(acc));
    }
    if constexpr (DOT) {
      token_sums<TPT>(part, red);
      store_dots<TPT>(p, t, 0, s0, part);
      // the dot products of the slots past the first eight: their rows again
      for (int j0 = kSlots; j0 < p.k; j0 += kSlots) {
        const Slots s = slots_of(p, rop, gate, t, j0);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) part[i] = 0.f;
        for (int v = tid; v < nv; v += TPT) {
          float f[VE];
          load<0, DT, VE>(ra, v).widen(f);
#pragma unroll
          for (int i = 0; i < kSlots; ++i) {
            float g[VE];
            load<0, DT, VE>(row_of(p.in, s.r[i], row_bytes), v).widen(g);
#pragma unroll
            for (int q = 0; q < VE; ++q) part[i] = fmaf(f[q], g[q], part[i]);
          }
        }
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

template <int DT, int VE, int TPT> hipError_t scatter_t(const PairRows& p, hipStream_t s) {
  const dim3 g(grid_of<TPT>(p.T)), b(256);
  if (p.dot) {
    if (p.gate) hipLaunchKernelGGL((scatter_kernel<DT, VE, TPT, true, true>), g, b, 0, s, p, p.rop, p.gate);
    else hipLaunchKernelGGL((scatter_kernel<DT, VE, TPT, false, true>), g, b, 0, s, p, p.rop, p.gate);
  } else {
    if (p.gate) hipLaunchKernelGGL((scatter_kernel<DT, VE, TPT, true, false>), g, b, 0, s, p, p.rop, p.gate);
    else hipLaunchKernelGGL((scatter_kernel<DT, VE, TPT, false, false>), g, b, 0, s, p, p.rop, p.gate);
  }
  return hipGetLastError();
}
template <int DT, int VE, int TPT> hipError_t gather_t(const PairRows& p, hipStream_t s) {
  const dim3 g(grid_of<TPT>(p.T)), b(256);
  if (p.dot) hipLaunchKernelGGL((gather_kernel<DT, VE, TPT, true>), g, b, 0, s, p, p.rop, p.gate);
  else hipLaunchKernelGGL((gather_kernel<DT, VE, TPT, false>), g, b, 0, s, p, p.rop, p.gate);
  return hipGetLastError();
}

template <int DT, int VE> hipError_t run(const PairRows& p, bool scatter, hipStream_t s) {
  const bool wave = p.d / VE <= 128;
  if (scatter) return wave ? scatter_t<DT, VE, 64>(p, s) : scatter_t<DT, VE, 256>(p, s);
  return wave ? gather_t<DT, VE, 64>(p, s) : gather_t<DT, VE, 256>(p, s);
}

// The widest access that divides a row: 16 bytes, 4, or (an odd row of 16-bit
// elements) 2.
hipError_t dispatch(const PairRows& p, bool scatter, hipStream_t s) {
  if (p.T == 0) return hipSuccess;
  const int64_t b = (int64_t)p.d * (p.dtype == kF32 ? 4 : 2);
  switch (p.dtype) {
    case kF32: return b % 16 == 0 ? run<kF32, 4>(p, scatter, s) : run<kF32, 1>(p, scatter, s);
    case kBF16:
      return b % 16 == 0 ? run<kBF16, 8>(p, scatter, s) : b % 4 == 0 ? run<kBF16, 2>(p, scatter, s)
                                                                     : run<kBF16, 1>(p, scatter, s);
    case kF16:
      return b % 16 == 0 ? run<kF16, 8>(p, scatter, s) : b % 4 == 0 ? run<kF16, 2>(p, scatter, s)
                                                                    : run<kF16, 1>(p, scatter, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_scatter_rows(const PairRows& p, hipStream_t s) { return dispatch(p, true, s); }
hipError_t launch_gather_rows(const PairRows& p, hipStream_t s) { return dispatch(p, false, s); }

}  // namespace mok
