#include "sffn_norm_kernels.h"

namespace sffn {
hipError_t launch_norm_bf16(const NormArgs& a, int y_type, hipStream_t s) { return norm_of<__bf16>(a, y_type, s); }
}  // namespace sffn
