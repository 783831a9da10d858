#include "sffn_norm_kernels.h"

namespace sffn {
hipError_t launch_norm_f16(const NormArgs& a, int y_type, hipStream_t s) { return norm_of<_Float16>(a, y_type, s); }
}  // namespace sffn
