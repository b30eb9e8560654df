// Element types of the separate expert operators: storage, and vectors of VE
// consecutive elements moved as one access; and a wave's prefix sum.
#pragma once
#include "mok_device.h"

namespace mok {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// 16-bit pair <-> fp32 (round to nearest even; NaN stays NaN)
template <int DT> struct Elem;
template <> struct Elem<1> {  // bf16
  static constexpr int kBytes = 2;
  __device__ __forceinline__ static float lo(uint32_t w) { return __uint_as_float(w << 16); }
  __device__ __forceinline__ static float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
  }
};
template <> struct Elem<2> {  // fp16
  static constexpr int kBytes = 2;
  __device__ __forceinline__ static float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2_t, w)[0]; }
  __device__ __forceinline__ static float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2_t, w)[1]; }
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
  }
};
template <> struct Elem<0> {  // fp32
  static constexpr int kBytes = 4;
};

// VE elements of type DT held raw in W dwords (a lone 16-bit element in the
// low half of one dword).
template <int DT, int VE> struct Vec {
  static constexpr int kB = Elem<DT>::kBytes * VE;  // bytes of one access
  static constexpr int W = kB < 4 ? 1 : kB / 4;
  uint32_t w[W];

  __device__ __forceinline__ void widen(float* f) const {
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < VE; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (VE == 1) {
      f[0] = Elem<DT>::lo(w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        f[2 * i] = Elem<DT>::lo(w[i]);
        f[2 * i + 1] = Elem<DT>::hi(w[i]);
      }
    }
  }
  __device__ __forceinline__ static Vec narrow(const float* f) {
    Vec v;
    if constexpr (DT == 0) {
#pragma unroll
      for (int i = 0; i < VE; ++i) v.w[i] = __float_as_uint(f[i]);
    } else if constexpr (VE == 1) {
      v.w[0] = Elem<DT>::pack(f[0], 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v.w[i] = Elem<DT>::pack(f[2 * i], f[2 * i + 1]);
    }
    return v;
  }
};

// Inclusive sum over the lanes of a wave: within rows of 16 lanes by shifts,
// then the row before's and the half before's total.
template <int CTRL, int ROWS> __device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v = dpp_add<0x111, 0xf>(v);  // row_shr 1
  v = dpp_add<0x112, 0xf>(v);  // row_shr 2
  v = dpp_add<0x114, 0xf>(v);  // row_shr 4
  v = dpp_add<0x118, 0xf>(v);  // row_shr 8
  v = dpp_add<0x142, 0xa>(v);  // row_bcast 15 into rows 1 and 3
  return dpp_add<0x143, 0xc>(v);  // row_bcast 31 into rows 2 and 3
}

}  // namespace mok
