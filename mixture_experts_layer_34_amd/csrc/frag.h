// Operand fragments of the 16x16 matrix instructions for rows of fp32, bf16 or
// fp16: 16 bytes of one row a lane, of any width and alignment.
//
// With lane = 16 g + i, the lane holds KE consecutive elements (16 bytes) of
// operand row i from element g KE of the K step on.  16-bit types: KE = 8, one
// v_mfma_f32_16x16x32 a step.  fp32: KE = 4, four v_mfma_f32_16x16x4, the j-th
// taking element j of every lane: the same order of K in both operands, so
// every product is summed once.  The result holds, in lane 16 g + i, rows
// 4 g + 0..3 (of the first operand) of column i (row i of the second).
#pragma once
#include "elem.h"

namespace mok {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

// A wave's number in its workgroup, in a scalar register: what depends on it
// branches as a whole wave.  (A matrix instruction ignores the execution mask,
// so none may stand under a condition that the compiler takes for one of lanes.)
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

template <int DT> constexpr int kFragElems = 16 / Elem<DT>::kBytes;  // KE
template <int DT> constexpr int kFragStep = 4 * kFragElems<DT>;      // elements of a K step

template <int DT> __device__ __forceinline__ f32x4_t mma(u32x4_t a, u32x4_t b, f32x4_t c) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (DT == 1) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  } else if constexpr (DT == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
    return c;
  }
#else
  return c;
#endif
}

// 16 bytes at p, which is aligned to an element only.
typedef uint32_t u32x4_on2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_on4_t __attribute__((ext_vector_type(4), aligned(4)));
template <int DT> __device__ __forceinline__ u32x4_t load16(const char* p) {
  if constexpr (Elem<DT>::kBytes == 4) return *reinterpret_cast<const u32x4_on4_t*>(p);
  else return *reinterpret_cast<const u32x4_on2_t*>(p);
}
template <int DT> __device__ __forceinline__ void store16(char* p, u32x4_t v) {
  if constexpr (Elem<DT>::kBytes == 4) *reinterpret_cast<u32x4_on4_t*>(p) = v;
  else *reinterpret_cast<u32x4_on2_t*>(p) = v;
}

// 16 bytes of a row of 16-bit elements that may start on any of them: where p is
// on no dword, the four dwords from two bytes before it and the last element on its
// own, put together at `get`: eight tokens at d 2111 198 us, with 16-byte loads off
// the dwords 271 (d 2112: 137).  Nothing outside p's sixteen bytes is read but the two
// before them, of the dword that p lies in, and their bits are shifted out.  ODD
// false: a plain load16.
template <int DT, bool ODD> struct Quad {
  u32x4_t v;
  uint32_t last;
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (ODD) {
      v = *reinterpret_cast<const u32x4_on4_t*>(p - ((uintptr_t)p & 2));
      last = *reinterpret_cast<const uint16_t*>(p + 14);
    } else {
      v = load16<DT>(p);
    }
  }
  // shift: shift_of(p)
  __device__ __forceinline__ u32x4_t get(uint32_t shift) const {
    if constexpr (!ODD) return v;
    u32x4_t o;
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_alignbit(j < 3 ? v[j < 3 ? j + 1 : 3] : last, v[j], shift);
#endif
    return o;
  }
};
template <bool ODD> __device__ __forceinline__ uint32_t shift_of(const char* p) {
  return ODD ? ((uint32_t)(uintptr_t)p & 2) * 8 : 0;
}

// The first n (0..KE) elements at p, zeros behind them.
template <int DT> __device__ __forceinline__ u32x4_t load_part(const char* p, int n) {
  constexpr int KE = kFragElems<DT>;
  if (n >= KE) return load16<DT>(p);
  u32x4_t v = {0, 0, 0, 0};
  if constexpr (Elem<DT>::kBytes == 4) {
#pragma unroll
    for (int j = 0; j < KE; ++j)
      if (j < n) v[j] = reinterpret_cast<const uint32_t*>(p)[j];
  } else {
#pragma unroll
    for (int j = 0; j < KE; ++j)
      if (j < n) v[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j & 1));
  }
  return v;
}
template <int DT> __device__ __forceinline__ void store_part(char* p, u32x4_t v, int n) {
  constexpr int KE = kFragElems<DT>;
  if (n >= KE) {
    store16<DT>(p, v);
    return;
  }
#pragma unroll
  for (int j = 0; j < KE; ++j)
    if (j < n) {
      if constexpr (Elem<DT>::kBytes == 4) reinterpret_cast<uint32_t*>(p)[j] = v[j];
      else reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
    }
}

// v with zeros in place of the elements from the n-th on (n may be negative).
template <int DT> __device__ __forceinline__ u32x4_t first_elems(u32x4_t v, int n) {
  constexpr int PER = 4 / Elem<DT>::kBytes;  // elements of a dword
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (PER == 1) v[j] = j < n ? v[j] : 0u;
    else v[j] = 2 * j + 1 < n ? v[j] : 2 * j < n ? v[j] & 0xFFFFu : 0u;
  }
  return v;
}

// v with zeros in place of its first n elements (n >= 0).
template <int DT> __device__ __forceinline__ u32x4_t but_first(u32x4_t v, int n) {
  constexpr int PER = 4 / Elem<DT>::kBytes;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (PER == 1) v[j] = j >= n ? v[j] : 0u;
    else v[j] = 2 * j >= n ? v[j] : 2 * j + 1 >= n ? v[j] & 0xFFFF0000u : 0u;
  }
  return v;
}

// The step that a row of n elements (n >= KE) ends in, a lane's elements from k
// on: both operands are read from `tail_at`, whole and inside the row, and one of
// them gets zeros for the elements that another lane or step has counted.
template <int DT> __device__ __forceinline__ int tail_at(int k, int n) {
  return k < n - kFragElems<DT> ? k : n - kFragElems<DT>;
}

// v moved down by n elements (0 <= n; zeros come in, all of it for n >= KE).
template <int DT> __device__ __forceinline__ u32x4_t shift_elems(u32x4_t v, int n) {
  constexpr int PER = 4 / Elem<DT>::kBytes;
  const int q = n / PER;
  u32x4_t t;
#pragma unroll
  for (int j = 0; j < 4; ++j) t[j] = q & 1 ? (j < 3 ? v[j < 3 ? j + 1 : 3] : 0u) : v[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = q >= 4 ? 0u : q & 2 ? (j < 2 ? t[j < 2 ? j + 2 : 3] : 0u) : t[j];
  if constexpr (PER == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = (v[j] >> 16) | (j < 3 ? v[j < 3 ? j + 1 : 3] << 16 : 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = n & 1 ? t[j] : v[j];
  }
  return v;
}

// KE elements as fp32 and back (rounded to nearest even).
template <int DT> __device__ __forceinline__ void widen(u32x4_t v, float* f) {
  Vec<DT, kFragElems<DT>> e;
#pragma unroll
  for (int j = 0; j < 4; ++j) e.w[j] = v[j];
  e.widen(f);
}
template <int DT> __device__ __forceinline__ u32x4_t narrow(const float* f) {
  const auto e = Vec<DT, kFragElems<DT>>::narrow(f);
  return u32x4_t{e.w[0], e.w[1], e.w[2], e.w[3]};
}

}  // namespace mok
