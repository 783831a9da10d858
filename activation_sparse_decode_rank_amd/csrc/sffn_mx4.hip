// Products of rows in 4-bit blocks on the matrix cores (gfx950).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes a block of 32 codes (16 bytes) and its scale byte from
// each lane: lane (r16 = lane % 16, g = lane / 16) holds block g of row r16 of either operand.
#include <algorithm>

#include "sffn_mx4.h"
#include "sffn_mx4_rows.h"

namespace sffn {
namespace {

typedef int int4_t __attribute__((ext_vector_type(4)));
typedef int int8_vec __attribute__((ext_vector_type(8)));

constexpr int FMT_FP4 = 4;  // the instruction's operand format

// acc += the products of 16 rows of w and 16 rows of x, four blocks long
template <int SW, int SX>
__device__ __forceinline__ float4_t mfma16(const int4_t& w, const int4_t& x, const float4_t& acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      int8_vec{w[0], w[1], w[2], w[3], 0, 0, 0, 0}, int8_vec{x[0], x[1], x[2], x[3], 0, 0, 0, 0}, acc,
      FMT_FP4, FMT_FP4, SW, sw, SX, sx);
}

// Four neighbouring sums of a row as outputs
__device__ __forceinline__ void emit4(const Mx4ProductArgs& a, int64_t r, int c, float4_t v) {
  if (c >= a.n) return;
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < a.n) v[j] += a.bias[c + j];
  }
  const size_t o = (size_t)r * a.ldo + c;
  if (a.out_type == T_F32) store4<float>(a.out, o, v, a.n - c);
  else if (a.out_type == T_F16) store4<_Float16>(a.out, o, v, a.n - c);
  else store4<__bf16>(a.out, o, v, a.n - c);
}

// 64 channels x 64 rows of x a workgroup, 16 channels a wave, operands straight from memory.
__global__ __launch_bounds__(TPB) void k_mx4_product(Mx4ProductArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int nnt = (a.n + 63) / 64;
  const int n0 = (blockIdx.x % nnt) * 64 + wave * 16;
  const int r0 = (int)(blockIdx.x / nnt) * 64;
  const int wr = min(n0 + r16, a.n - 1);
  const uint8_t* w = a.w + (size_t)wr * a.ldw;
  const uint8_t* ws = a.ws + (size_t)wr * a.ldws;
  const uint8_t *x[4], *xs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = min(r0 + 16 * j + r16, a.rows - 1);
    x[j] = a.x + (size_t)r * a.ldx;
    xs[j] = a.xs + (size_t)r * a.ldxs;
  }
  float4_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
  for (int b0 = 0; b0 < a.nb; b0 += 4) {
    const int b = b0 + g;
    int4_t f = {0, 0, 0, 0}, v[4];
    int s = 127, vs[4];
    if (b < a.nb) {
      f = *reinterpret_cast<const int4_t*>(w + 16 * b);
      s = ws[b];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = int4_t{0, 0, 0, 0};
      vs[j] = 127;
      if (b < a.nb) {
        v[j] = *reinterpret_cast<const int4_t*>(x[j] + 16 * b);
        vs[j] = xs[j][b];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = mfma16<0, 0>(f, v[j], acc[j], s, vs[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 16 * j + r16;
    if (r < a.rows) emit4(a, r, n0 + 4 * g, acc[j]);
  }
}

}  // namespace

hipError_t launch_mx4_product(const Mx4ProductArgs& a, hipStream_t s) {
  const int64_t tiles = ((int64_t)a.n + 63) / 64 * (((int64_t)a.rows + 63) / 64);
  k_mx4_product<<<dim3((unsigned)tiles), dim3(TPB), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace sffn
