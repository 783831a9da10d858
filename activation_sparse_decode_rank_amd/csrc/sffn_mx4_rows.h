// Numbers in 4-bit blocks on the device: a block of 32 is held by four neighbouring lanes, eight
// numbers each.
#pragma once
#include "sffn_rows.h"

namespace sffn {
namespace {

struct F8 {
  float v[8];
};

// Eight values of a row from element 8 i on, as they lie in memory, and past `cols` zeros
template <typename T>
using vec8 = T __attribute__((ext_vector_type(8)));

template <typename T>
__device__ __forceinline__ vec8<T> raw8(const T* x, int64_t i, int64_t cols) {
  typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  vec8<T> v;
  if (8 * i + 8 <= cols) {
    v = *reinterpret_cast<const vec*>(x + 8 * i);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 8 * i + e < cols ? x[8 * i + e] : (T)0.f;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ F8 floats8(const vec8<T>& v) {
  F8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = (float)v[e];
  return f;
}

template <typename T>
__device__ __forceinline__ F8 load8(const T* x, int64_t i, int64_t cols) {
  return floats8(raw8(x, i, cols));
}

// Eight values of a row to element 8 i on, and none past `cols`
template <typename T>
__device__ __forceinline__ void put8(T* y, int64_t i, int64_t cols, const F8& f) {
  typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  if (8 * i + 8 <= cols) {
    vec t;
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = (T)f.v[e];
    *reinterpret_cast<vec*>(y + 8 * i) = t;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * i + e < cols) y[8 * i + e] = (T)f.v[e];
  }
}

// the float 2^(E - 127), NaN for 255
__device__ __forceinline__ float mx4_scale(unsigned E) {
  const unsigned bits = E == 255 ? 0x7fc00000u : E == 0 ? 0x00400000u : E << 23;
  return __builtin_bit_cast(float, bits);
}

// The codes of this lane's eight numbers, the first in the lowest four bits, and the scale of the
// block of the four lanes that it is in (all four hold it). The largest magnitude m has the scale
// 2^e with 3.5 * 2^e <= m < 7 * 2^e: m's exponent - 2, one more where its mantissa is 1.75 or
// above, which is what adding 1/4 to the mantissa carries. Under 2^e m rounds to 4 or 6, where
// 2^(e + 1) would give it no smaller error and the others larger ones; from 7 * 2^e on 6 would be
// further off than 8.
__device__ __forceinline__ unsigned mx4_encode(const F8& f, unsigned& E) {
  unsigned m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, mag(f.v[e]));
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, DPP_QP_XOR1, 0xF, 0xF, true));
  m = max(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, DPP_QP_XOR2, 0xF, 0xF, true));
  const int x = (int)((m + 0x200000u) >> 23) - 2;
  const bool bad = m >= 0x7f800000u;
  E = bad ? 255u : (unsigned)max(x, 0);
  const float s = mx4_scale(bad ? 127u : E);
  unsigned q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f.v[0], f.v[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f.v[2], f.v[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f.v[4], f.v[5], s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f.v[6], f.v[7], s, 3);
  return bad ? 0u : q;
}

}  // namespace
}  // namespace sffn
