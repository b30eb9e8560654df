// 4-bit integer expert products with bf16 activations and scales.
#include "int4_matvec_kernel.h"

namespace mok {
hipError_t launch_int4_matvec_bf16(const Int4Args& a, hipStream_t s) { return launch_int4(a, Launch<kBF16>{s}); }
}  // namespace mok
