// Root-mean-square norm with the residual's addition, into float rows, 8-bit rows or 4-bit blocks: the
// kernels, for rows of one type. Each type has a source of its own, so that they build in parallel.
#pragma once
#include <algorithm>

#include "sffn_mx4.h"
#include "sffn_mx4_rows.h"
#include "sffn_pipeline.h"

namespace sffn {
namespace {

// v plus the same value of the lane that DPP pattern CTRL names
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp_add_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, ROW_MASK, 0xF, true);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, ROW_MASK, 0xF, true);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// the larger of v and that lane's
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ unsigned dpp_max(unsigned v) {
  return max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, true));
}

// Sum, and largest, over the threads of a workgroup of W waves, in the waves' order. at: a word for
// each wave; not written again before every wave has met another barrier.
template <int W>
__device__ __forceinline__ double wg_sum(double v, double* at) {
  v = dpp_add_f64<DPP_QP_XOR1>(v);
  v = dpp_add_f64<DPP_QP_XOR2>(v);
  v = dpp_add_f64<DPP_HALF_MIRROR>(v);
  v = dpp_add_f64<DPP_MIRROR>(v);
  v = dpp_add_f64<DPP_BCAST15, 0xA>(v);
  v = dpp_add_f64<DPP_BCAST31, 0xC>(v);  // complete in the last lane
  if constexpr (W == 1) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)b, 63);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(b >> 32), 63);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  } else {
    if ((threadIdx.x & 63) == 63) at[threadIdx.x >> 6] = v;
    lds_barrier();
    v = 0.0;
#pragma unroll
    for (int q = 0; q < W; ++q) v += at[q];
    return v;
  }
}
template <int W>
__device__ __forceinline__ unsigned wg_largest(unsigned v, unsigned* at) {
  v = dpp_max<DPP_QP_XOR1>(v);
  v = dpp_max<DPP_QP_XOR2>(v);
  v = dpp_max<DPP_HALF_MIRROR>(v);
  v = dpp_max<DPP_MIRROR>(v);
  v = dpp_max<DPP_BCAST15, 0xA>(v);
  v = dpp_max<DPP_BCAST31, 0xC>(v);
  if constexpr (W == 1) {
    return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
  } else {
    if ((threadIdx.x & 63) == 63) at[threadIdx.x >> 6] = v;
    lds_barrier();
    v = 0;
#pragma unroll
    for (int q = 0; q < W; ++q) v = max(v, at[q]);
    return v;
  }
}

template <typename T>
__device__ __forceinline__ void put_raw8(T* y, int64_t i, int64_t cols, const vec8<T>& v) {
  typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  if (8 * i + 8 <= cols) {
    *reinterpret_cast<vec*>(y + 8 * i) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * i + e < cols) y[8 * i + e] = v[e];
  }
}

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

// groups of eight of a row that are written: whole 16 bytes of 8-bit rows, whole blocks
template <int OUT>
__host__ __device__ constexpr int64_t norm_groups(int64_t cols) {
  return OUT == T_MX4 ? (cols + 31) / 32 * 4 : OUT == T_I8 ? (cols + 15) / 16 * 2 : (cols + 7) / 8;
}

// 1 / sqrt(x) of a number that is not negative: the instruction's value, good to some 2^-26, made
// better twice (a few 2^-53 off). An eighth of the instructions of a root and a quotient, which
// every wave of a row would do.
__device__ __forceinline__ double inverse_root(double x) {
  double r = __builtin_amdgcn_rsq(x);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-x * r, r, 1.0), r);
  return x < __builtin_inf() ? r : x == __builtin_inf() ? 0.0 : x;
}

// Eight 64-bit values as floats on their way into OUT: the nearest ones for fp32 rows and for what is held
// in fewer bits afterwards. 16-bit rows take what the 64-bit value itself rounds to, and the nearest float
// rounds to something else only where it is the middle of two of them and the 64-bit value is not (of
// normal values one in 16000 for fp16, one in 90000 for bf16). Floats whose last 12 bits (bf16: 15) are
// zero, all such middles among them, are therefore made again: 13 bits of the 64-bit value, the last one
// set where anything behind it is. fp16 keeps 11 of those and bf16 8 (fewer below the normal numbers), so
// the bit after them and whether anything follows still decide; values below 2^-137, of which floats hold
// fewer than 13 bits, are zero in either type. 4096 x 4096 bf16 rows without a residual take 14.3 us so,
// 15.0 with every value made again, 13.3 with two roundings (with a residual 25.2, 25.2, 24.9).
template <int OUT>
__device__ __forceinline__ F8 on_their_way(const double (&v)[8]) {
  F8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = (float)v[e];
  if constexpr (OUT == T_F16 || OUT == T_BF16) {
    constexpr unsigned LAST = OUT == T_F16 ? 0xfffu : 0x7fffu;
    unsigned least = LAST;
#pragma unroll
    for (int e = 0; e < 8; ++e) least = min(least, __builtin_bit_cast(unsigned, f.v[e]) & LAST);
    if (least == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v[e]);
        unsigned hi = (unsigned)(b >> 32);
        const unsigned rest = (hi & 0xffu) | (unsigned)b;
        hi = (hi & ~0xffu) | (rest ? 0x100u : 0u);
        f.v[e] = (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
      }
    }
  }
  return f;
}

// Writes eight values y of row `row` as the call's outputs. s, rs: the scale of an 8-bit row.
template <int OUT>
__device__ __forceinline__ void write8(const NormArgs& a, int64_t row, int64_t i, const F8& y, float s, float rs) {
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
    put8(static_cast<float*>(a.y) + row * a.ldy, i, a.cols, y);
  } else if constexpr (OUT == T_F16) {
    put8(static_cast<_Float16*>(a.y) + row * a.ldy, i, a.cols, y);
  } else {
    put8(static_cast<__bf16*>(a.y) + row * a.ldy, i, a.cols, y);
  }
}

// A workgroup of W waves takes row after row, eight values a thread and NV such groups; the next row
// is on its way while one is summed and written, and the weights stay in registers. The sum of
// squares and the products v w r are 64-bit (exact products): nothing overflows, and a row's one rounding
// is the same whatever it is held in afterwards. 64-bit multiply-adds are as fast as 32-bit ones here, but
// the conversions around them are not: rows with a residual and fp32 rows have enough bytes to hide them,
// 16-bit rows without one do not.
template <typename T, int OUT, int W, int NV>
__global__ __launch_bounds__(W * 64) void k_norm(NormArgs a) {
  constexpr int TH = W * 64;
  __shared__ double s_sum[2][W];
  __shared__ unsigned s_max[2][W];
  const int cols = a.cols;
  const int groups = (int)norm_groups<OUT>(cols);
  const int tid = threadIdx.x;
  const int64_t step = gridDim.x;
  struct Row {
    vec8<T> x[NV], r[NV];
  };
  auto load = [&](Row& R, int64_t row) {
    if (row >= a.rows) return;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (tid + u * TH < groups) R.x[u] = raw8(x, tid + u * TH, cols);
    if (a.res) {
      const T* res = static_cast<const T*>(a.res) + row * a.ldr;
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (tid + u * TH < groups) R.r[u] = raw8(res, tid + u * TH, cols);
    }
  };
  Row R, next;
  load(R, blockIdx.x);
  F8 w[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (tid + u * TH < groups) w[u] = weights8(a, tid + u * TH);
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += step) {
    load(next, row + step);
    double ss = 0.0;
    F8 y[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (tid + u * TH >= groups) continue;
      if (a.res) {
#pragma unroll
        for (int e = 0; e < 8; ++e) R.x[u][e] = (T)((float)R.x[u][e] + (float)R.r[u][e]);
        put_raw8(static_cast<T*>(a.sum) + row * a.ldsum, tid + u * TH, cols, R.x[u]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double v = (double)(float)R.x[u][e];
        ss = fma(v, v, ss);
      }
    }
    const double r = inverse_root(wg_sum<W>(ss, s_sum[par]) * a.per_col + a.eps);
    unsigned big = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (tid + u * TH >= groups) continue;
      double v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (double)(float)R.x[u][e] * (double)w[u].v[e] * r;
      y[u] = on_their_way<OUT>(v);
      if (OUT == T_I8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) big = max(big, mag(y[u].v[e]));
      }
    }
    float s = 0.f, rs = 0.f;
    if (OUT == T_I8) {
      s = row_scale(wg_largest<W>(big, s_max[par]), rs);
      if (tid == 0) static_cast<float*>(a.scale)[row] = s;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (tid + u * TH < groups) write8<OUT>(a, row, tid + u * TH, y[u], s, rs);
    // the next row's sums are written beside these, the ones after them past a barrier
    par ^= 1;
    R = next;
  }
}

// Longer rows: read, summed, and read again to be written (for 8-bit rows twice). 1024 x 20000 bf16 with a
// residual take 43 us into bf16 (3.8 TB/s of what has to be read and written), 46.5 into 8 bits (3.1);
// without one 22.8 into bf16 (3.6); fp32 rows 43 (3.8); 1024 x 40000 with one into blocks 71 (3.8).
template <typename T, int OUT>
__global__ __launch_bounds__(1024) void k_norm_long(NormArgs a) {
  constexpr int W = 16, TH = W * 64;
  __shared__ double s_sum[2][W];
  __shared__ unsigned s_max[2][W];
  const int64_t groups = norm_groups<OUT>(a.cols);
  int par = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* res = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
    T* sum = a.res ? static_cast<T*>(a.sum) + row * a.ldsum : nullptr;
    double ss = 0.0;
    for (int64_t i = threadIdx.x; i < groups; i += TH) {
      F8 f = load8(x, i, a.cols);
      if (res) {
        const F8 g = load8(res, i, a.cols);
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = (float)(T)(f.v[e] + g.v[e]);
        put8(sum, i, a.cols, f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fma((double)f.v[e], (double)f.v[e], ss);
    }
    const double r = inverse_root(wg_sum<W>(ss, s_sum[par]) * a.per_col + a.eps);
    const T* held = res ? sum : x;  // what this thread itself has written
    auto again = [&](int64_t i) {
      const F8 f = load8(held, i, a.cols), w = weights8(a, i);
      double v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (double)f.v[e] * (double)w.v[e] * r;
      return on_their_way<OUT>(v);
    };
    float s = 0.f, rs = 0.f;
    if (OUT == T_I8) {
      unsigned big = 0;
      for (int64_t i = threadIdx.x; i < groups; i += TH) {
        const F8 y = again(i);
#pragma unroll
        for (int e = 0; e < 8; ++e) big = max(big, mag(y.v[e]));
      }
      s = row_scale(wg_largest<W>(big, s_max[par]), rs);
      if (threadIdx.x == 0) static_cast<float*>(a.scale)[row] = s;
    }
    for (int64_t i = threadIdx.x; i < groups; i += TH) write8<OUT>(a, row, i, again(i), s, rs);
    par ^= 1;
  }
}

template <typename T, int OUT, int W, int NV>
void norm_launch(const NormArgs& a, hipStream_t s) {
  const int at_once = resident<k_norm<T, OUT, W, NV>>(W * 64, 0);
  k_norm<T, OUT, W, NV><<<dim3((unsigned)std::min(a.rows, at_once)), dim3(W * 64), 0, s>>>(a);
}

// As many waves as hold a row with eight values a thread, sixteen at most, so that a compute unit has
// several workgroups whose reads, barriers and writes overlap: 4096 rows of 4096 bf16 with a residual
// into 8 bits take 26.7 us with eight waves, 28.2 with four of sixteen values (and into blocks 21.7
// and 22.4); of 8192, 53.5 with sixteen and 54.3 with eight; one row 3.2 us with eight, 4.0 with four.
// Bound by memory: 4.4 TB/s read and written into 8 bits where another operator's writes stand before it
// (5.1 alone; a second barrier, and the remainders), 5.0 into blocks (5.9), 5.3 into bf16 and in fp32;
// 2048 rows of 12288 into blocks 31 to 33 us. 16-bit rows without a residual are bound by the arithmetic:
// 4096 x 4096 bf16 into blocks 13.3 us (3.2 TB/s), into bf16 14.3 (4.7).
template <typename T, int OUT>
void norm_launch(const NormArgs& a, hipStream_t s) {
  const int64_t groups = ((int64_t)a.cols + 31) / 32 * 4;
  if (groups <= 64) norm_launch<T, OUT, 1, 1>(a, s);
  else if (groups <= 128) norm_launch<T, OUT, 2, 1>(a, s);
  else if (groups <= 256) norm_launch<T, OUT, 4, 1>(a, s);
  else if (groups <= 512) norm_launch<T, OUT, 8, 1>(a, s);
  else if (groups <= 1024) norm_launch<T, OUT, 16, 1>(a, s);
  else if (groups <= 2048) norm_launch<T, OUT, 16, 2>(a, s);
  else k_norm_long<T, OUT><<<dim3((unsigned)std::min(a.rows, 1 << 20)), dim3(1024), 0, s>>>(a);
}

template <typename T>
hipError_t norm_of(const NormArgs& a, int y_type, hipStream_t s) {
  switch (y_type) {
    case T_F32: norm_launch<T, T_F32>(a, s); break;
    case T_F16: norm_launch<T, T_F16>(a, s); break;
    case T_BF16: norm_launch<T, T_BF16>(a, s); break;
    case T_I8: norm_launch<T, T_I8>(a, s); break;
    default: norm_launch<T, T_MX4>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace sffn
