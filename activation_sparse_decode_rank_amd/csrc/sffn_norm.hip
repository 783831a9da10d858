// Rows into 4-bit blocks and back, and the norms' dispatch by type (gfx950).
#include <algorithm>

#include "sffn_mx4.h"
#include "sffn_mx4_rows.h"

namespace sffn {
namespace {

// L lanes a row (a power of two), TPB / L rows a workgroup, and UNROLL such sets of rows at once, whose
// reads are issued together: 2048 x 12288 blocks into bf16 in 11 us so, 14 with one set; fp32 values
// are twice the bytes a lane, and gain nothing (11008 x 4096 from blocks 34.6 us, 35.7 with four).
// Bound by memory: 11008 x 4096 fp32 into blocks 35.5 us, 5.8 TB/s read and written, and back 32.6 us,
// 6.3 (in turn 50 and 34: what the second wrote then goes to memory while the first reads). Whole lines
// a load, values exchanged between lanes afterwards, take as long, and more sets of rows longer.
template <typename T>
constexpr int UNROLL = sizeof(T) == 2 ? 4 : 1;

template <typename T, int U>
__global__ __launch_bounds__(TPB) void k_quantize_mx4(Mx4QuantArgs a, int L) {
  const int64_t groups = (int64_t)a.blocks * 4;
  const int per = TPB / L;
  const int64_t step = (int64_t)gridDim.x * per;
  for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / L; row < a.rows; row += U * step) {
    for (int64_t i = (int64_t)blockIdx.y * L + threadIdx.x % L; i < groups; i += (int64_t)gridDim.y * L) {
      F8 f[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (row + k * step < a.rows) f[k] = load8(static_cast<const T*>(a.x) + (row + k * step) * a.ldx, i, a.cols);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t r = row + k * step;
        if (r >= a.rows) break;
        unsigned E;
        reinterpret_cast<unsigned*>(a.q + r * a.ldq)[i] = mx4_encode(f[k], E);
        if ((i & 3) == 0) a.scale[r * a.lds + (i >> 2)] = (uint8_t)E;
      }
    }
  }
}

template <typename T, int U>
__global__ __launch_bounds__(TPB) void k_dequantize_mx4(Mx4DequantArgs a, int L) {
  const int64_t groups = ((int64_t)a.cols + 7) / 8;
  const int per = TPB / L;
  const int64_t step = (int64_t)gridDim.x * per;
  for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / L; row < a.rows; row += U * step) {
    for (int64_t i = (int64_t)blockIdx.y * L + threadIdx.x % L; i < groups; i += (int64_t)gridDim.y * L) {
      unsigned c[U], E[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t r = row + k * step;
        if (r >= a.rows) break;
        c[k] = reinterpret_cast<const unsigned*>(a.q + r * a.ldq)[i];
        E[k] = a.scale[r * a.lds + (i >> 2)];
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t r = row + k * step;
        if (r >= a.rows) break;
        const float s = mx4_scale(E[k]);
        F8 f;
        auto two = [&](int at, auto t) {
          f.v[at] = t[0] * s;
          f.v[at + 1] = t[1] * s;
        };
        two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.f, 0));
        two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.f, 1));
        two(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.f, 2));
        two(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[k], 1.f, 3));
        put8(static_cast<T*>(a.y) + r * a.ldy, i, a.cols, f);
      }
    }
  }
}

// lanes a row, and the grid: rows down x, pieces of long rows down y, 2^20 workgroups (2^28 threads)
// at most: the kernels go on from there. A workgroup takes several sets of rows from LEAST workgroups of
// one set on, so that every compute unit still has some. bf16 from blocks: 2866 x 1703 5.3 us so and
// 5.6 with one set, 4096 x 4096 8.7 and 10.8, but 1500 x 1703 4.2 and 3.9. Into blocks it decides little:
// 4096 x 4096 10.0 and 10.3, 2048 x 12288 13.7 both ways, 2866 x 1703 6.0 and 5.6, 1500 x 1703 4.5 and 3.9.
constexpr int64_t LEAST = 2048;
struct RowGrid {
  int L;
  bool sets;
  dim3 grid;
  RowGrid(int rows, int64_t groups, int unroll) {
    L = 4;
    while (L < TPB && L < groups) L *= 2;
    const int64_t y = std::min<int64_t>((groups + L - 1) / L, 64);
    int64_t x = ((int64_t)rows + TPB / L - 1) / (TPB / L);
    sets = unroll > 1 && x * y >= LEAST;
    if (sets) x = (x + unroll - 1) / unroll;
    grid = dim3((unsigned)std::min<int64_t>(x, (1 << 20) / y), (unsigned)y);
  }
};

}  // namespace

hipError_t launch_norm(const NormArgs& a, int x_type, int y_type, hipStream_t s) {
  if (x_type == T_F32) return launch_norm_f32(a, y_type, s);
  if (x_type == T_F16) return launch_norm_f16(a, y_type, s);
  return launch_norm_bf16(a, y_type, s);
}

namespace {
template <typename T>
hipError_t quantize_launch(const Mx4QuantArgs& a, hipStream_t s) {
  const RowGrid g(a.rows, (int64_t)a.blocks * 4, UNROLL<T>);
  if (g.sets) k_quantize_mx4<T, UNROLL<T>><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  else k_quantize_mx4<T, 1><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  return hipGetLastError();
}
template <typename T>
hipError_t dequantize_launch(const Mx4DequantArgs& a, hipStream_t s) {
  const RowGrid g(a.rows, ((int64_t)a.cols + 7) / 8, UNROLL<T>);
  if (g.sets) k_dequantize_mx4<T, UNROLL<T>><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  else k_dequantize_mx4<T, 1><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_quantize_mx4(const Mx4QuantArgs& a, int x_type, hipStream_t s) {
  if (x_type == T_F32) return quantize_launch<float>(a, s);
  if (x_type == T_F16) return quantize_launch<_Float16>(a, s);
  return quantize_launch<__bf16>(a, s);
}

hipError_t launch_dequantize_mx4(const Mx4DequantArgs& a, int y_type, hipStream_t s) {
  if (y_type == T_F32) return dequantize_launch<float>(a, s);
  if (y_type == T_F16) return dequantize_launch<_Float16>(a, s);
  return dequantize_launch<__bf16>(a, s);
}

}  // namespace sffn
