// Root-mean-square norm with the residual's addition, into float rows, 8-bit rows or 4-bit blocks,
// and rows into 4-bit blocks and back (gfx950).
#include <algorithm>

#include "sffn_mx4.h"
#include "sffn_mx4_rows.h"

namespace sffn {
namespace {

typedef unsigned long long u64;

__device__ __forceinline__ double xor_lane(double v, int o) { return __shfl_xor(v, o); }

// Eight weights from element 8 i on (1 where there are none; past cols 0)
__device__ __forceinline__ F8 weights8(const NormArgs& a, int64_t i) {
  if (!a.w) {
    F8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = 1.f;
    return f;
  }
  if (a.w_type == T_F32) return load8(static_cast<const float*>(a.w), i, a.cols);
  if (a.w_type == T_F16) return load8(static_cast<const _Float16*>(a.w), i, a.cols);
  return load8(static_cast<const __bf16*>(a.w), i, a.cols);
}

// A workgroup of W waves takes a row, eight values a thread and NV such groups (NV = 0: any number,
// read again for the second pass). The sum of squares and the products v w r are 64-bit (exact
// products; 64-bit multiply-adds are as fast as 32-bit ones here, and the rows wait for memory):
// nothing overflows, and a row's one rounding is the same whatever it is held in afterwards. The
// largest |y| of an 8-bit row is the rounded product of the largest |v w|, so that it meets the sum
// at the same barrier.
template <typename T, int OUT, int W, int NV>
__global__ __launch_bounds__(W * 64) void k_norm(NormArgs a) {
  constexpr int TH = W * 64;
  constexpr bool KEPT = NV > 0;
  __shared__ double s_sum[W];
  __shared__ u64 s_max[W];
  const int cols = a.cols;
  // groups that are written: whole 16 bytes of 8-bit rows, whole blocks
  const int groups = OUT == T_MX4 ? (int)(((int64_t)cols + 31) / 32 * 4)
                     : OUT == T_I8 ? (int)(((int64_t)cols + 15) / 16 * 2) : (int)(((int64_t)cols + 7) / 8);
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
    T* sum = a.res ? static_cast<T*>(a.sum) + row * a.ldsum : nullptr;
    auto value = [&](int i) {
      F8 f = load8(x, i, cols);
      if (res) {
        const F8 g = load8(res, i, cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = (float)(T)(f.v[e] + g.v[e]);
        put8(sum, i, cols, f);
      }
      return f;
    };
    double ss = 0.0;
    u64 big = 0;
    auto take = [&](const F8& v, const F8& w) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fma((double)v.v[e], (double)v.v[e], ss);
        if (OUT == T_I8)
          big = max(big, __builtin_bit_cast(u64, (double)v.v[e] * (double)w.v[e]) & 0x7fffffffffffffffull);
      }
    };
    F8 v[KEPT ? NV : 1], w[KEPT ? NV : 1];
    if constexpr (KEPT) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = tid + u * TH;
        if (i < groups) {
          v[u] = value(i);
          w[u] = weights8(a, i);
        }
      }
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (tid + u * TH < groups) take(v[u], w[u]);
    } else {
      for (int i = tid; i < groups; i += TH) take(value(i), weights8(a, i));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      ss += xor_lane(ss, o);
      if (OUT == T_I8) big = max(big, (u64)__shfl_xor(big, o));
    }
    if constexpr (W > 1) {
      if ((tid & 63) == 0) {
        s_sum[tid >> 6] = ss;
        s_max[tid >> 6] = big;
      }
      __syncthreads();
      ss = 0.0;
      big = 0;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        ss += s_sum[q];
        big = max(big, s_max[q]);
      }
      __syncthreads();
    }
    const double r = 1.0 / sqrt(ss / (double)cols + a.eps);
    float s = 0.f, rs = 0.f;
    if (OUT == T_I8) {
      s = row_scale(mag((float)(__builtin_bit_cast(double, big) * r)), rs);
      if (tid == 0) static_cast<float*>(a.scale)[row] = s;
    }
    auto write = [&](int i, const F8& v, const F8& w) {
      F8 y;
#pragma unroll
      for (int e = 0; e < 8; ++e) y.v[e] = (float)((double)v.v[e] * (double)w.v[e] * r);
      if constexpr (OUT == T_I8) {
        const float4_t lo = {y.v[0], y.v[1], y.v[2], y.v[3]}, hi = {y.v[4], y.v[5], y.v[6], y.v[7]};
        int2 q = {0, 0};
        if (s > 0.f) q = int2{quantize4(lo, s, rs), quantize4(hi, s, rs)};
        reinterpret_cast<int2*>(static_cast<int8_t*>(a.y) + row * a.ldy)[i] = q;
      } else if constexpr (OUT == T_MX4) {
        unsigned E;
        const unsigned q = mx4_encode(y, E);
        reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.y) + row * a.ldy)[i] = q;
        if ((i & 3) == 0) (static_cast<uint8_t*>(a.scale) + row * a.lds)[i >> 2] = (uint8_t)E;
      } else if constexpr (OUT == T_F32) {
        put8(static_cast<float*>(a.y) + row * a.ldy, i, cols, y);
      } else if constexpr (OUT == T_F16) {
        put8(static_cast<_Float16*>(a.y) + row * a.ldy, i, cols, y);
      } else {
        put8(static_cast<__bf16*>(a.y) + row * a.ldy, i, cols, y);
      }
    };
    if constexpr (KEPT) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (tid + u * TH < groups) write(tid + u * TH, v[u], w[u]);
    } else {
      const T* held = res ? sum : x;  // what this thread itself has written
      for (int i = tid; i < groups; i += TH) write(i, load8(held, i, cols), weights8(a, i));
    }
  }
}

template <typename T, int OUT>
void norm_launch(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)std::min(a.rows, 1 << 20));
  const int64_t groups = ((int64_t)a.cols + 31) / 32 * 4;
  if (groups <= 2 * 64) k_norm<T, OUT, 1, 2><<<grid, dim3(64), 0, s>>>(a);
  else if (groups <= 2 * 256) k_norm<T, OUT, 4, 2><<<grid, dim3(256), 0, s>>>(a);
  else if (groups <= 2 * 1024) k_norm<T, OUT, 16, 2><<<grid, dim3(1024), 0, s>>>(a);
  else k_norm<T, OUT, 16, 0><<<grid, dim3(1024), 0, s>>>(a);
}

template <typename T>
void norm_launch(const NormArgs& a, int y_type, hipStream_t s) {
  switch (y_type) {
    case T_F32: norm_launch<T, T_F32>(a, s); break;
    case T_F16: norm_launch<T, T_F16>(a, s); break;
    case T_BF16: norm_launch<T, T_BF16>(a, s); break;
    case T_I8: norm_launch<T, T_I8>(a, s); break;
    default: norm_launch<T, T_MX4>(a, s); break;
  }
}

// L lanes a row (a power of two), TPB / L rows a workgroup
template <typename T>
__global__ __launch_bounds__(TPB) void k_quantize_mx4(Mx4QuantArgs a, int L) {
  const int groups = a.blocks * 4;
  const int per = TPB / L;
  const int64_t step = (int64_t)gridDim.x * per;
  for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / L; row < a.rows; row += step) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    unsigned* q = reinterpret_cast<unsigned*>(a.q + row * a.ldq);
    uint8_t* scale = a.scale + row * a.lds;
    for (int64_t i = (int64_t)blockIdx.y * L + threadIdx.x % L; i < groups; i += (int64_t)gridDim.y * L) {
      unsigned E;
      q[i] = mx4_encode(load8(x, i, a.cols), E);
      if ((i & 3) == 0) scale[i >> 2] = (uint8_t)E;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(TPB) void k_dequantize_mx4(Mx4DequantArgs a, int L) {
  const int groups = (int)(((int64_t)a.cols + 7) / 8);
  const int per = TPB / L;
  const int64_t step = (int64_t)gridDim.x * per;
  for (int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / L; row < a.rows; row += step) {
    const unsigned* q = reinterpret_cast<const unsigned*>(a.q + row * a.ldq);
    const uint8_t* scale = a.scale + row * a.lds;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    for (int64_t i = (int64_t)blockIdx.y * L + threadIdx.x % L; i < groups; i += (int64_t)gridDim.y * L) {
      const unsigned c = q[i];
      const float s = mx4_scale(scale[i >> 2]);
      F8 f;
      auto two = [&](int at, auto t) {
        f.v[at] = t[0] * s;
        f.v[at + 1] = t[1] * s;
      };
      two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0));
      two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1));
      two(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2));
      two(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3));
      put8(y, i, a.cols, f);
    }
  }
}

// lanes a row, and the grid: rows down x, pieces of long rows down y
struct RowGrid {
  int L;
  dim3 grid;
  RowGrid(int rows, int64_t groups) {
    L = 4;
    while (L < TPB && L < groups) L *= 2;
    const int64_t at = ((int64_t)rows + TPB / L - 1) / (TPB / L);
    grid = dim3((unsigned)std::min<int64_t>(at, 1 << 20),
                (unsigned)std::min<int64_t>((groups + L - 1) / L, 64));
  }
};

}  // namespace

hipError_t launch_norm(const NormArgs& a, int x_type, int y_type, hipStream_t s) {
  if (x_type == T_F32) norm_launch<float>(a, y_type, s);
  else if (x_type == T_F16) norm_launch<_Float16>(a, y_type, s);
  else norm_launch<__bf16>(a, y_type, s);
  return hipGetLastError();
}

hipError_t launch_quantize_mx4(const Mx4QuantArgs& a, int x_type, hipStream_t s) {
  const RowGrid g(a.rows, (int64_t)a.blocks * 4);
  if (x_type == T_F32) k_quantize_mx4<float><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  else if (x_type == T_F16) k_quantize_mx4<_Float16><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  else k_quantize_mx4<__bf16><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const Mx4DequantArgs& a, int y_type, hipStream_t s) {
  const RowGrid g(a.rows, ((int64_t)a.cols + 7) / 8);
  if (y_type == T_F32) k_dequantize_mx4<float><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  else if (y_type == T_F16) k_dequantize_mx4<_Float16><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  else k_dequantize_mx4<__bf16><<<g.grid, dim3(TPB), 0, s>>>(a, g.L);
  return hipGetLastError();
}

}  // namespace sffn
