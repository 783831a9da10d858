// Rows held in 8 bits, and products of such rows on the matrix cores (gfx950).
//
// A row r is held as s = max|r| / 127 and q_j = the whole number nearest to r_j / s. A product
// of two such rows is the exact whole-number sum of q_j w_j (at most 131071 products of two
// 8-bit values fit 32 bits), times the two rows' scales.
#include <algorithm>

#include "sffn_device.h"
#include "sffn_i8.h"

namespace sffn {
namespace {

typedef int int4_t __attribute__((ext_vector_type(4)));

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

// scale of a row from the bits of its largest magnitude; r = 1 / scale (0: a row of zeros)
__device__ __forceinline__ float row_scale(unsigned bits, float& r) {
  const float a = __builtin_bit_cast(float, bits);
  r = 0.f;
  if (bits >= 0x7f800000u) return __builtin_nanf("");
  if (a < SMALLEST_ROW) return 0.f;
  const float s = a / 127.f;
  r = 1.f / s;
  return s;
}

template <typename T>
__global__ __launch_bounds__(TPB) void k_quantize(QuantArgs a) {
  __shared__ unsigned s_max[TPB / 64];
  const int rows = a.rows_dev ? min(*a.rows_dev, a.rows) : a.rows;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (size_t)row * a.ldx;
    unsigned m = 0;
    for (int j = threadIdx.x; j < a.cols; j += TPB)
      m = max(m, __builtin_bit_cast(unsigned, (float)x[j]) & 0x7fffffffu);
    for (int o = 32; o; o >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, o));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPB / 64; ++w) m = max(m, s_max[w]);
    __syncthreads();
    float r;
    const float s = row_scale(m, r);
    if (threadIdx.x == 0) a.scale[row] = s;
    int8_t* q = a.q + (size_t)row * a.ldq;
    for (int j = threadIdx.x; j < a.kpad; j += TPB)
      q[j] = j < a.cols && s > 0.f ? (int8_t)quantize((float)x[j], s, r) : 0;
  }
}

__global__ __launch_bounds__(TPB) void k_pad_rows(const int8_t* __restrict__ x, int64_t ldx,
                                                  int rows, int cols, int8_t* __restrict__ q,
                                                  int kpad) {
  for (int row = blockIdx.x; row < rows; row += gridDim.x)
    for (int j = threadIdx.x; j < kpad; j += TPB)
      q[(size_t)row * kpad + j] = j < cols ? x[(size_t)row * ldx + j] : 0;
}

template <typename T>
__device__ __forceinline__ void store_as(void* p, size_t i, float v) {
  static_cast<T*>(p)[i] = (T)v;
}

// Tile of 64 rows x 64 channels over the whole length, steps of 128 bytes. Wave w takes the
// 16 tokens 16 w .. +16 and all 64 channels (four 16 x 16 tiles); the gated form's channels
// are 32 neurons, gate and up rows of 16 neurons in neighbouring tiles.
constexpr int LDT = 128 + 16;  // LDS row: 128 bytes and a 16-byte pad against bank conflicts

template <int MODE>
__global__ __launch_bounds__(TPB) void k_product(ProductArgs a) {
  constexpr bool GROUPED = MODE != MODE_LINEAR;
  constexpr int NT = MODE == MODE_ACT_GATED ? 32 : 64;  // channels (neurons) per tile
  __shared__ __attribute__((aligned(16))) int8_t s_w[64 * LDT];
  __shared__ __attribute__((aligned(16))) int8_t s_x[64 * LDT];
  const int nnt = (a.n + NT - 1) / NT;
  const int nt = blockIdx.x % nnt, mt = blockIdx.x / nnt;
  int e = 0, r0 = mt * host::kI8Tile, r1 = a.rows;
  if (GROUPED) {
    if (mt >= *a.n_tiles) return;
    e = a.tiles[2 * mt];
    r0 = a.tiles[2 * mt + 1];
    r1 = a.offs[e + 1];
  }
  const int8_t* w = a.w + (size_t)e * a.w_group;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int n0 = nt * NT;
  const int nw = MODE == MODE_ACT_GATED ? 2 * a.n : a.n;  // rows of w
  // row of w that row i of the tile stands for
  auto wrow = [&](int i) {
    if (MODE == MODE_ACT_GATED) return 2 * (n0 + (i >> 5) * 16 + (i & 15)) + ((i >> 4) & 1);
    return n0 + i;
  };
  // row of x behind tile row i
  auto xrow = [&](int i) {
    const int r = min(r0 + i, r1 - 1);
    if (MODE == MODE_ACT || MODE == MODE_ACT_GATED) return a.src[r] / a.k;
    return r;
  };
  int4_t acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = int4_t{0, 0, 0, 0};
  // each thread stages two 16-byte chunks of each operand
  const int c8 = tid & 7;
  const int8_t *pw[2], *px[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = (tid >> 3) + 32 * u;
    pw[u] = w + (size_t)min(wrow(i), nw - 1) * a.ldw;
    px[u] = a.x + (size_t)xrow(i) * a.ldx;
  }
  for (int k0 = 0; k0 < a.kch; k0 += 8) {
    // past the row's end x holds zeros (its rows are padded), so any chunk of w will do
    const int cw = min(k0 + c8, a.kch - 1);
    int4_t vw[2], vx[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      vw[u] = *reinterpret_cast<const int4_t*>(pw[u] + (size_t)cw * 16);
      vx[u] = *reinterpret_cast<const int4_t*>(px[u] + (size_t)(k0 + c8) * 16);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = (tid >> 3) + 32 * u;
      *reinterpret_cast<int4_t*>(s_w + i * LDT + c8 * 16) = vw[u];
      *reinterpret_cast<int4_t*>(s_x + i * LDT + c8 * 16) = vx[u];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int4_t b =
          *reinterpret_cast<const int4_t*>(s_x + (wave * 16 + r16) * LDT + h * 64 + g * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int4_t m =
            *reinterpret_cast<const int4_t*>(s_w + (i * 16 + r16) * LDT + h * 64 + g * 16);
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(m, b, acc[i], 0, 0, 0);
      }
    }
  }
  // lane holds token row r16 of its wave and channels 16 i + 4 g .. +3
  const int r = r0 + wave * 16 + r16;
  if (r >= r1) return;
  const float xs = a.xs[xrow(wave * 16 + r16)];
  const float* ws = a.ws + (size_t)e * nw;
  if (MODE == MODE_ACT || MODE == MODE_ACT_GATED) {
    float* out = static_cast<float*>(a.out) + (size_t)r * a.ldo;
    const float* bias = a.bias ? a.bias + (size_t)e * a.n : nullptr;
    for (int i = 0; i < 4; i += MODE == MODE_ACT_GATED ? 2 : 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n0 + (MODE == MODE_ACT_GATED ? (i >> 1) : i) * 16 + 4 * g + j;
        if (c >= a.n) continue;
        double h;
        if (MODE == MODE_ACT_GATED)
          h = (double)acc[i][j] * ((double)xs * (double)ws[2 * c]);
        else
          h = (double)acc[i][j] * ((double)xs * (double)ws[c]);
        if (bias) h += (double)bias[c];
        h = h < 0.0 ? 0.0 : h;  // NaN stays
        if (MODE == MODE_ACT_GATED)
          h *= (double)acc[(i + 1) & 3][j] * ((double)xs * (double)ws[2 * c + 1]);
        out[c] = (float)h;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + i * 16 + 4 * g + j;
      if (c >= a.n) continue;
      float v = (float)acc[i][j] * (xs * ws[c]);
      if (MODE == MODE_DOWN) {
        static_cast<float*>(a.out)[(size_t)a.src[r] * a.ldo + c] = v;
      } else {
        if (a.bias) v += a.bias[c];
        const size_t o = (size_t)r * a.ldo + c;
        if (a.out_type == T_F32) store_as<float>(a.out, o, v);
        else if (a.out_type == T_F16) store_as<_Float16>(a.out, o, v);
        else store_as<__bf16>(a.out, o, v);
      }
    }
}

}  // namespace

hipError_t launch_quantize(const QuantArgs& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)std::min(a.rows, 1 << 20)), block(TPB);
  if (dtype == T_F32) k_quantize<float><<<grid, block, 0, s>>>(a);
  else if (dtype == T_F16) k_quantize<_Float16><<<grid, block, 0, s>>>(a);
  else k_quantize<__bf16><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const int8_t* x, int64_t ldx, int rows, int cols, int8_t* q, int kpad,
                           hipStream_t s) {
  k_pad_rows<<<dim3((unsigned)std::min(rows, 1 << 20)), dim3(TPB), 0, s>>>(x, ldx, rows, cols, q,
                                                                          kpad);
  return hipGetLastError();
}

hipError_t launch_product(const ProductArgs& a, ProductMode mode, hipStream_t s) {
  const int nt = mode == MODE_ACT_GATED ? 32 : 64;
  const int64_t tiles = mode == MODE_LINEAR
                            ? ((int64_t)a.rows + host::kI8Tile - 1) / host::kI8Tile
                            : (int64_t)a.max_tiles;
  const dim3 grid((unsigned)(tiles * (((int64_t)a.n + nt - 1) / nt))), block(TPB);
  switch (mode) {
    case MODE_LINEAR: k_product<MODE_LINEAR><<<grid, block, 0, s>>>(a); break;
    case MODE_ACT: k_product<MODE_ACT><<<grid, block, 0, s>>>(a); break;
    case MODE_ACT_GATED: k_product<MODE_ACT_GATED><<<grid, block, 0, s>>>(a); break;
    case MODE_DOWN: k_product<MODE_DOWN><<<grid, block, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace sffn
