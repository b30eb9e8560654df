// 4-bit integer expert products with fp16 activations and scales.
#include "int4_matvec_kernel.h"

namespace mok {
hipError_t launch_int4_matvec_f16(const Int4Args& a, hipStream_t s) { return launch_int4(a, Launch<kF16>{s}); }
}  // namespace mok
