#include "sffn_norm_kernels.h"

namespace sffn {
hipError_t launch_norm_f32(const NormArgs& a, int y_type, hipStream_t s) { return norm_of<float>(a, y_type, s); }
}  // namespace sffn
