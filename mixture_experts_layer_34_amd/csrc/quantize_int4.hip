// 4-bit integer quantisation of a [rows, K] matrix along its rows, for the
// weights of mok_expert_matvec_int4 (the integer counterpart of the layer's MX
// quantisers): groups of g consecutive elements,
//   symmetric   s = amax / 7, q = clamp(rint(v / s) + 8, 0, 15), z = 8;
//   with zeros  lo = min(v, 0), hi = max(v, 0), s = (hi - lo) / 15,
//               z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(v / s) + z, 0, 15).
// s is rounded to the matrix's type before it divides; a scale of zero (a
// group of zeros, or one below the type's range) takes q = z, every weight 0.
// Eight elements per lane, g / 8 lanes to a group.  2 bytes are read and 1/2
// written an element, at 3.6-3.8 TB/s of both (128 matrices of 1536 x 4096 550-580
// us, 8192 x 4096 26 us; a copy reaches 4.9).  Once per weight, outside any decode
// step: what keeps it from a copy's rate was not looked into.
#include "elem.h"
#include "int4_matvec.h"
#include "pair_ops.h"

namespace mok {
namespace {

template <int DT, int GS>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const uint4* __restrict__ src, int64_t nvec,
                                                            uint32_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales,
                                                            uint8_t* __restrict__ zeros) {
  constexpr int LG = GS / 8;  // lanes per group
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t v0 = (int64_t)blockIdx.x * 256; v0 < nvec; v0 += stride) {
    const int64_t v = v0 + threadIdx.x;
    const bool act = v < nvec;  // nvec is a multiple of LG: a group's lanes agree
    const uint4 u = act ? src[v] : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Elem<DT>::lo(w[i]);
      f[2 * i + 1] = Elem<DT>::hi(w[i]);
    }
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, f[i]);
      hi = fmaxf(hi, f[i]);
    }
#pragma unroll
    for (int o = 1; o < LG; o <<= 1) {
      lo = fminf(lo, __shfl_xor(lo, o, 64));
      hi = fmaxf(hi, __shfl_xor(hi, o, 64));
    }
    // hi - lo, or half of it where finite values lie further apart than fp32 reaches
    const float span = hi - lo, wide = 0.5f * hi - 0.5f * lo;
    const float s15 = span <= 3.4028234e38f ? span / 15.0f : wide / 15.0f * 2.0f;
    const uint16_t sb = (uint16_t)Elem<DT>::pack(zeros ? s15 : fmaxf(hi, -lo) / 7.0f, 0.f);
    const float s = Elem<DT>::lo(sb);
    const float z = zeros ? (s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f) : 8.f;
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = s > 0.f ? fminf(fmaxf(rintf(f[i] / s) + z, 0.f), 15.f) : z;
      c |= (uint32_t)q << (4 * i);
    }
    if (act) {
      codes[v] = c;
      if (v % LG == 0) {
        scales[v / LG] = sb;
        if (zeros) zeros[v / LG] = (uint8_t)z;
      }
    }
  }
}

template <int DT> hipError_t run(const void* src, int64_t nvec, int group, uint8_t* codes, void* scales, uint8_t* zeros,
                                 hipStream_t s) {
  const int64_t n = (nvec + 255) / 256;
  const dim3 g((unsigned)(n < 65536 ? n : 65536)), b(256);
#define MOK_QUANT(GS)                                                                                             \
  hipLaunchKernelGGL((quantize_int4_kernel<DT, GS>), g, b, 0, s, (const uint4*)src, nvec, (uint32_t*)codes,        \
                     (uint16_t*)scales, zeros)
  switch (group) {
    case 32: MOK_QUANT(32); break;
    case 64: MOK_QUANT(64); break;
    case 128: MOK_QUANT(128); break;
    default: return hipErrorInvalidValue;
  }
#undef MOK_QUANT
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int4(const void* src, int64_t rows, int64_t K, int group, int dtype, uint8_t* codes,
                                void* scales, uint8_t* zeros, hipStream_t s) {
  const int64_t nvec = rows * K / 8;
  if (nvec == 0) return hipSuccess;
  if (dtype == kBF16) return run<kBF16>(src, nvec, group, codes, scales, zeros, s);
  if (dtype == kF16) return run<kF16>(src, nvec, group, codes, scales, zeros, s);
  return hipErrorInvalidValue;
}

}  // namespace mok
