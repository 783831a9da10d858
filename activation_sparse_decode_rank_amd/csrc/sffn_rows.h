// Rows of numbers on the device: loads and stores of neighbouring values of any float type, and
// rows held in 8 bits. Shared by the kernels that hold rows in fewer bits and those that multiply
// them.
#pragma once
#include "sffn_device.h"

namespace sffn {
namespace {

constexpr float SMALLEST_ROW = 0x1p-100f;  // rows below this are held as zeros

// The whole number nearest to x / s, ties to even, decided exactly: x * r (r about 1 / s)
// is within one of it; the remainder x - q s is exact in 32 bits (a multiple of s's last
// place, below 2^24 of them), and where it is past half of s the neighbour is nearer.
__device__ __forceinline__ int quantize(float x, float s, float r) {
#pragma clang fp contract(off)
  float q = rintf(x * r);
  const float e = __builtin_fmaf(-q, s, x);
  const float half = 0.5f * s;
  const int qi = (int)q;
  if (e > half || (e == half && (qi & 1))) return qi + 1;
  if (e < -half || (e == -half && (qi & 1))) return qi - 1;
  return qi;
}

// scale of a row from the bits of its largest magnitude; r: 1 / scale but for its last places, which
// decide nothing (0: a row of zeros)
__device__ __forceinline__ float row_scale(unsigned bits, float& r) {
  const float a = __builtin_bit_cast(float, bits);
  r = 0.f;
  if (bits >= 0x7f800000u) return __builtin_nanf("");
  if (a < SMALLEST_ROW) return 0.f;
  const float s = a * (1.f / 127.f);
  r = __builtin_amdgcn_rcpf(s);
  return s;
}

__device__ __forceinline__ unsigned mag(float v) {
  return __builtin_bit_cast(unsigned, v) & 0x7fffffffu;
}

// largest of v over the workgroup (s_max: one word per wave)
template <int WAVES>
__device__ __forceinline__ unsigned wg_max(unsigned v, unsigned* s_max) {
  for (int o = 32; o; o >>= 1) v = max(v, (unsigned)__shfl_xor((int)v, o));
  if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) v = max(v, s_max[w]);
  __syncthreads();
  return v;
}

// Four values of a row from element 4 i on, and past `cols` zeros
template <typename T>
__device__ __forceinline__ float4_t load4(const T* x, int i, int cols) {
  typedef T vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  float4_t v = {0.f, 0.f, 0.f, 0.f};
  if (4 * i + 4 <= cols) {
    const vec t = *reinterpret_cast<const vec*>(x + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * i + e < cols) v[e] = (float)x[4 * i + e];
  }
  return v;
}

// Four values of a row, packed. Almost always every remainder is clearly inside half a step and
// q stands; the neighbours are looked at only where one is not. x r + 1.5 * 2^23 is rounded to a
// whole number, and holds q in its lowest byte: four operations a value, and three permutations.
__device__ __forceinline__ int quantize4(const float4_t& v, float s, float r) {
#pragma clang fp contract(off)
  constexpr float MAGIC = 12582912.f;
  const float lim = 0.4999f * s;
  unsigned q[4];
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = __builtin_fmaf(v[e], r, MAGIC);
    q[e] = __builtin_bit_cast(unsigned, f);
    far = fmaxf(far, fabsf(__builtin_fmaf(-(f - MAGIC), s, v[e])));
  }
  if (far > lim) {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = (unsigned)quantize(v[e], s, r);
  }
  const unsigned lo = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u);
  const unsigned hi = __builtin_amdgcn_perm(q[3], q[2], 0x0c0c0400u);
  return (int)__builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Four neighbouring values of a row as T, the first `left` of them
template <typename T>
__device__ __forceinline__ void store4(void* p, size_t i, const float4_t& v, int left) {
  typedef T vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  T* o = static_cast<T*>(p) + i;
  if (left >= 4) {
    vec t;
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = (T)v[j];
    *reinterpret_cast<vec*>(o) = t;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) o[j] = (T)v[j];
  }
}

// Eight neighbouring values of a row as T, the first `left` of them
template <typename T>
__device__ __forceinline__ void store8(void* p, size_t i, const float4_t& a, const float4_t& b, int left) {
  typedef T vec __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  if (left >= 8) {
    vec t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      t[j] = (T)a[j];
      t[4 + j] = (T)b[j];
    }
    *reinterpret_cast<vec*>(static_cast<T*>(p) + i) = t;
  } else {
    store4<T>(p, i, a, left);
    store4<T>(p, i + 4, b, left - 4);
  }
}

}  // namespace
}  // namespace sffn
