// Rows held in 8 bits, and products of such rows on the matrix cores (gfx950).
//
// A row r is held as s = max|r| * (1 / 127) and q_j = the whole number nearest to r_j / s. A product
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
  const float s = a * (1.f / 127.f);
  r = 1.f / s;
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

// Four values of a row from element 4 i on, and past `cols` zeros. VEC: the row starts at a
// multiple of four elements' size.
template <typename T, bool VEC>
__device__ __forceinline__ float4_t load4(const T* x, int i, int cols) {
  typedef T vec __attribute__((ext_vector_type(4)));
  float4_t v = {0.f, 0.f, 0.f, 0.f};
  if (VEC && 4 * i + 4 <= cols) {
    const vec t = reinterpret_cast<const vec*>(x)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * i + e < cols) v[e] = (float)x[4 * i + e];
  }
  return v;
}

__device__ __forceinline__ int quantize4(const float4_t& v, float s, float r) {
  int p = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) p |= (quantize(v[e], s, r) & 0xff) << (8 * e);
  return p;
}

// A workgroup takes a row. NV groups of four values per thread stay in registers between the
// maximum and the rounding, so the row is read once (NV = 0: longer rows, read twice).
template <typename T, bool VEC, int NV>
__global__ __launch_bounds__(TPB) void k_quantize(QuantArgs a) {
  __shared__ unsigned s_max[TPB / 64];
  const int rows = a.rows_dev ? min(*a.rows_dev, a.rows) : a.rows;
  const int nq = a.kpad / 4;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (size_t)row * a.ldx;
    int* q = reinterpret_cast<int*>(a.q + (size_t)row * a.ldq);
    unsigned m = 0;
    float r;
    if constexpr (NV > 0) {
      float4_t v[NV];
#pragma unroll
      for (int u = 0; u < NV; ++u) v[u] = load4<T, VEC>(x, threadIdx.x + u * TPB, a.cols);
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, mag(v[u][e]));
      m = wg_max<TPB / 64>(m, s_max);
      const float s = row_scale(m, r);
      if (threadIdx.x == 0) a.scale[row] = s;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = threadIdx.x + u * TPB;
        if (i < nq) q[i] = s > 0.f ? quantize4(v[u], s, r) : 0;
      }
    } else {
      for (int i = threadIdx.x; i < nq; i += TPB) {
        const float4_t v = load4<T, VEC>(x, i, a.cols);
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, mag(v[e]));
      }
      m = wg_max<TPB / 64>(m, s_max);
      const float s = row_scale(m, r);
      if (threadIdx.x == 0) a.scale[row] = s;
      for (int i = threadIdx.x; i < nq; i += TPB)
        q[i] = s > 0.f ? quantize4(load4<T, VEC>(x, i, a.cols), s, r) : 0;
    }
  }
}

__global__ __launch_bounds__(TPB) void k_pad_rows(const int8_t* __restrict__ x, int64_t ldx,
                                                  int rows, int cols, int8_t* __restrict__ q,
                                                  int kpad) {
  for (int row = blockIdx.x; row < rows; row += gridDim.x)
    for (int j = threadIdx.x; j < kpad; j += TPB)
      q[(size_t)row * kpad + j] = j < cols ? x[(size_t)row * ldx + j] : 0;
}

// Four neighbouring values of a row as T; whole: all four are inside the row and the row's
// places are multiples of four elements.
template <typename T>
__device__ __forceinline__ void store4(void* p, size_t i, const float4_t& v, int left, bool whole) {
  typedef T vec __attribute__((ext_vector_type(4)));
  T* o = static_cast<T*>(p) + i;
  if (whole) {
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

// What becomes of the sums of sorted row (or row) r at channels (neurons) c .. c + 3 of expert
// e: v, and in the gated form u of the up rows. xs: the scale of the row of x behind r.
template <int MODE>
__device__ __forceinline__ void emit(const ProductArgs& a, int e, int r, float xs, int c,
                                     const int4_t& v, const int4_t& u) {
  if (c >= a.n) return;
  const int left = a.n - c;
  const bool whole = left >= 4 && a.vec_out;
  float4_t y;
  if constexpr (MODE == MODE_ACT || MODE == MODE_ACT_GATED) {
    // h in 64 bits up to its one rounding: it decides between whole numbers afterwards
    constexpr int M = MODE == MODE_ACT_GATED ? 2 : 1;
    const float* ws = a.ws + ((size_t)e * a.n + c) * M;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= left) break;
      double h = (double)v[j] * ((double)xs * (double)ws[M * j]);
      if (a.bias) h += (double)a.bias[(size_t)e * a.n + c + j];
      h = h < 0.0 ? 0.0 : h;  // NaN stays
      if (M == 2) h *= (double)u[j] * ((double)xs * (double)ws[M * j + 1]);
      y[j] = (float)h;
    }
    store4<float>(a.out, (size_t)r * a.ldo + c, y, left, whole);
  } else {
    const float* ws = a.ws + (size_t)e * a.n + c;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= left) break;
      y[j] = (float)v[j] * (xs * ws[j]);
      if (MODE == MODE_LINEAR && a.bias) y[j] += a.bias[c + j];
    }
    if (MODE == MODE_DOWN) {
      store4<float>(a.out, (size_t)a.src[r] * a.ldo + c, y, left, whole);
    } else {
      const size_t o = (size_t)r * a.ldo + c;
      if (a.out_type == T_F32) store4<float>(a.out, o, y, left, whole);
      else if (a.out_type == T_F16) store4<_Float16>(a.out, o, y, left, whole);
      else store4<__bf16>(a.out, o, y, left, whole);
    }
  }
}

// The rows that tile mt stands for: [r0, r1) of expert e; false: no such tile.
template <int MODE>
__device__ __forceinline__ bool tile_rows(const ProductArgs& a, int mt, int& e, int& r0, int& r1) {
  e = 0;
  r0 = mt * a.tile;
  r1 = a.rows;
  if (MODE != MODE_LINEAR) {
    if (mt >= *a.n_tiles) return false;
    e = a.tiles[2 * mt];
    r0 = a.tiles[2 * mt + 1];
    r1 = a.offs[e + 1];
  }
  return true;
}

// row of x behind (sorted) row r
template <int MODE>
__device__ __forceinline__ int row_of_x(const ProductArgs& a, int r) {
  return MODE == MODE_ACT || MODE == MODE_ACT_GATED ? a.src[r] / a.k : r;
}

// Few rows: the weights are streamed from memory once, straight into the matrix cores'
// registers. A workgroup of 8 waves takes 16 NC channels (gated: 8 NC neurons, gate and up rows
// in tiles 2 i and 2 i + 1) and up to 16 NR rows; its waves take blocks of 256 bytes of the
// length in turn (each lane 16 bytes of 4 steps; the next block's loads are issued before the
// current block's products) and add their sums through LDS at the end, whole numbers, so the
// split changes nothing. x comes from the caches.
constexpr int SK_W = 8;          // waves
constexpr int SK_BLK = 16;       // 16-byte chunks of a block

template <int MODE, int NC, int NR>
__global__ __launch_bounds__(SK_W * 64) void k_product_few(ProductArgs a) {
  constexpr bool G = MODE == MODE_ACT_GATED;
  constexpr int NT = G ? 8 * NC : 16 * NC;
  __shared__ __attribute__((aligned(16))) int4_t s_acc[SK_W][NC * NR][64];
  const int nnt = (a.n + NT - 1) / NT;
  const int nt = blockIdx.x % nnt;
  int e, r0, r1;
  if (!tile_rows<MODE>(a, blockIdx.x / nnt, e, r0, r1)) return;
  r1 = min(r1, r0 + 16 * NR);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, g = lane >> 4;
  const int n0 = nt * NT;
  const int nw = G ? 2 * a.n : a.n;
  const int8_t* pw[NC];
  const int8_t* px[NR];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int row = G ? 2 * (n0 + (i >> 1) * 16 + r16) + (i & 1) : n0 + i * 16 + r16;
    pw[i] = a.w + (size_t)e * a.w_group + (size_t)min(row, nw - 1) * a.ldw + g * 16;
  }
#pragma unroll
  for (int t = 0; t < NR; ++t)
    px[t] = a.x + (size_t)row_of_x<MODE>(a, min(r0 + t * 16 + r16, r1 - 1)) * a.ldx + g * 16;

  int4_t acc[NC][NR];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int t = 0; t < NR; ++t) acc[i][t] = int4_t{0, 0, 0, 0};
  struct Block {
    int4_t w[4][NC], x[4][NR];
  };
  auto load = [&](Block& B, int b) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const size_t o = (size_t)b * (SK_BLK * 16) + s * 64;
#pragma unroll
      for (int i = 0; i < NC; ++i)
        B.w[s][i] = __builtin_nontemporal_load(reinterpret_cast<const int4_t*>(pw[i] + o));
#pragma unroll
      for (int t = 0; t < NR; ++t) B.x[s][t] = *reinterpret_cast<const int4_t*>(px[t] + o);
    }
  };
  auto products = [&](const Block& B) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int t = 0; t < NR; ++t)
          acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(B.w[s][i], B.x[s][t], acc[i][t], 0, 0, 0);
  };
  const int nb = a.kch / SK_BLK;  // whole blocks
  Block B0, B1;
  int b = wave;
  if (b < nb) load(B0, b);
  while (b < nb) {
    if (b + SK_W < nb) load(B1, b + SK_W);
    products(B0);
    b += SK_W;
    if (b >= nb) break;
    if (b + SK_W < nb) load(B0, b + SK_W);
    products(B1);
    b += SK_W;
  }
  // the last, part block: one wave, chunk by chunk
  if (nb * SK_BLK < a.kch && wave == nb % SK_W) {
    for (int c = nb * SK_BLK; c < a.kch; c += 4) {
      const int4_t z = {0, 0, 0, 0};
      const bool in = c + g < a.kch;
      int4_t w[NC], x[NR];
#pragma unroll
      for (int i = 0; i < NC; ++i)
        w[i] = in ? *reinterpret_cast<const int4_t*>(pw[i] + (size_t)c * 16) : z;
#pragma unroll
      for (int t = 0; t < NR; ++t)
        x[t] = in ? *reinterpret_cast<const int4_t*>(px[t] + (size_t)c * 16) : z;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int t = 0; t < NR; ++t)
          acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i], x[t], acc[i][t], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int t = 0; t < NR; ++t) s_acc[wave][i * NR + t][lane] = acc[i][t];
  __syncthreads();
  auto total = [&](int q) {
    int4_t v = s_acc[0][q][lane];
#pragma unroll
    for (int w = 1; w < SK_W; ++w) v += s_acc[w][q][lane];
    return v;
  };
  // wave w: tiles w, w + 8, ... (gated: pairs of tiles); lane: row r16, channels 4 g .. +3
  for (int q = wave; q < (G ? NC / 2 : NC) * NR; q += SK_W) {
    const int i = q / NR, t = q % NR;
    const int r = r0 + t * 16 + r16;
    if (r >= r1) continue;
    const float xs = a.xs[row_of_x<MODE>(a, r)];
    if (G)
      emit<MODE>(a, e, r, xs, n0 + i * 16 + 4 * g, total(2 * i * NR + t), total((2 * i + 1) * NR + t));
    else
      emit<MODE>(a, e, r, xs, n0 + i * 16 + 4 * g, total(q), int4_t{0, 0, 0, 0});
  }
}

// Tile of 64 rows x 64 channels over the whole length, steps of 128 bytes. Wave w takes the
// 16 tokens 16 w .. +16 and all 64 channels (four 16 x 16 tiles); the gated form's channels
// are 32 neurons, gate and up rows of 16 neurons in neighbouring tiles.
constexpr int LDT = 128 + 16;  // LDS row: 128 bytes and a 16-byte pad against bank conflicts

template <int MODE>
__global__ __launch_bounds__(TPB) void k_product(ProductArgs a) {
  constexpr int NT = MODE == MODE_ACT_GATED ? 32 : 64;  // channels (neurons) per tile
  __shared__ __attribute__((aligned(16))) int8_t s_w[64 * LDT];
  __shared__ __attribute__((aligned(16))) int8_t s_x[64 * LDT];
  const int nnt = (a.n + NT - 1) / NT;
  const int nt = blockIdx.x % nnt, mt = blockIdx.x / nnt;
  int e, r0, r1;
  if (!tile_rows<MODE>(a, mt, e, r0, r1)) return;
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
  auto xrow = [&](int i) { return row_of_x<MODE>(a, min(r0 + i, r1 - 1)); };
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
  // lane holds row r16 of its wave and channels 16 i + 4 g .. +3
  const int r = r0 + wave * 16 + r16;
  if (r >= r1) return;
  const float xs = a.xs[xrow(wave * 16 + r16)];
#pragma unroll
  for (int i = 0; i < 4; i += MODE == MODE_ACT_GATED ? 2 : 1)
    emit<MODE>(a, e, r, xs, n0 + (MODE == MODE_ACT_GATED ? (i >> 1) : i) * 16 + 4 * g, acc[i],
               acc[(i + 1) & 3]);
}

template <int MODE, int NC, int NR>
void few_launch(const ProductArgs& a, int64_t tiles, hipStream_t s) {
  constexpr int NT = MODE == MODE_ACT_GATED ? 8 * NC : 16 * NC;
  const dim3 grid((unsigned)(tiles * ((a.n + NT - 1) / NT)));
  k_product_few<MODE, NC, NR><<<grid, dim3(SK_W * 64), 0, s>>>(a);
}

template <int MODE>
void product_launch(ProductArgs a, hipStream_t s) {
  a.vec_out = a.ldo % 4 == 0 &&
              reinterpret_cast<uintptr_t>(a.out) % (a.out_type == T_F32 ? 16 : 8) == 0;
  const int64_t tiles = MODE == MODE_LINEAR ? ((int64_t)a.rows + a.tile - 1) / a.tile : a.max_tiles;
  if (a.tile == 16) {
    few_launch<MODE, MODE == MODE_ACT_GATED ? 2 : 1, 1>(a, tiles, s);
  } else if (a.tile == 32) {
    few_launch<MODE, MODE == MODE_ACT_GATED ? 2 : 1, 2>(a, tiles, s);
  } else {
    constexpr int NT = MODE == MODE_ACT_GATED ? 32 : 64;
    k_product<MODE><<<dim3((unsigned)(tiles * ((a.n + NT - 1) / NT))), dim3(TPB), 0, s>>>(a);
  }
}

template <typename T, bool VEC>
void quantize_rows(const QuantArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)std::min(a.rows, 1 << 20)), block(TPB);
  const int nv = (a.kpad / 4 + TPB - 1) / TPB;
  if (nv <= 2) k_quantize<T, VEC, 2><<<grid, block, 0, s>>>(a);
  else if (nv <= 4) k_quantize<T, VEC, 4><<<grid, block, 0, s>>>(a);
  else if (nv <= 12) k_quantize<T, VEC, 12><<<grid, block, 0, s>>>(a);
  else k_quantize<T, VEC, 0><<<grid, block, 0, s>>>(a);
}

template <typename T>
void quantize_launch(const QuantArgs& a, hipStream_t s) {
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % (4 * sizeof(T)) == 0 && a.ldx % 4 == 0;
  if (vec) quantize_rows<T, true>(a, s);
  else quantize_rows<T, false>(a, s);
}

}  // namespace

hipError_t launch_quantize(const QuantArgs& a, int dtype, hipStream_t s) {
  if (dtype == T_F32) quantize_launch<float>(a, s);
  else if (dtype == T_F16) quantize_launch<_Float16>(a, s);
  else quantize_launch<__bf16>(a, s);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const int8_t* x, int64_t ldx, int rows, int cols, int8_t* q, int kpad,
                           hipStream_t s) {
  k_pad_rows<<<dim3((unsigned)std::min(rows, 1 << 20)), dim3(TPB), 0, s>>>(x, ldx, rows, cols, q,
                                                                          kpad);
  return hipGetLastError();
}

hipError_t launch_product(const ProductArgs& a, ProductMode mode, hipStream_t s) {
  switch (mode) {
    case MODE_LINEAR: product_launch<MODE_LINEAR>(a, s); break;
    case MODE_ACT: product_launch<MODE_ACT>(a, s); break;
    case MODE_ACT_GATED: product_launch<MODE_ACT_GATED>(a, s); break;
    case MODE_DOWN: product_launch<MODE_DOWN>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace sffn
