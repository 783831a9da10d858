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

// s_waitcnt operand (gfx9 encoding): LDS accesses only (lgkmcnt 0, vmcnt and expcnt at most)
constexpr int I8_WAIT_LGKM0 = 0xC07F;

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

// Four values of a row, packed. Almost always every remainder is clearly inside half a step and
// q stands; the neighbours are looked at only where one is not.
__device__ __forceinline__ int quantize4(const float4_t& v, float s, float r) {
#pragma clang fp contract(off)
  const float lim = 0.4999f * s;
  int q[4];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = rintf(v[e] * r);
    near |= fabsf(__builtin_fmaf(-f, s, v[e])) > lim;
    q[e] = (int)f;
  }
  if (near) {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = quantize(v[e], s, r);
  }
  const unsigned lo = (q[0] & 0xff) | ((q[1] & 0xff) << 8);
  const unsigned hi = (q[2] & 0xff) | ((q[3] & 0xff) << 8);
  return (int)(lo | (hi << 16));
}

// A workgroup of W waves takes a row. NV groups of four values per thread stay in registers
// between the maximum and the rounding, so the row is read once (NV = 0: longer rows, twice).
template <typename T, bool VEC, int W, int NV>
__global__ __launch_bounds__(W * 64) void k_quantize(QuantArgs a) {
  constexpr int TH = W * 64;
  __shared__ unsigned s_max[W];
  const int rows = a.rows_dev ? min(*a.rows_dev, a.rows) : a.rows;
  const int nq = a.kpad / 4;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (size_t)row * a.ldx;
    int* q = reinterpret_cast<int*>(a.q + (size_t)row * a.ldq);
    unsigned m = 0;
    float r;
    float4_t v[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
      for (int u = 0; u < NV; ++u) v[u] = load4<T, VEC>(x, threadIdx.x + u * TH, a.cols);
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, mag(v[u][e]));
    } else {
      for (int i = threadIdx.x; i < nq; i += TH) {
        const float4_t t = load4<T, VEC>(x, i, a.cols);
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, mag(t[e]));
      }
    }
    m = wg_max<W>(m, s_max);
    const float s = row_scale(m, r);
    if (threadIdx.x == 0) a.scale[row] = s;
    if constexpr (NV > 0) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int i = threadIdx.x + u * TH;
        if (i < nq) q[i] = s > 0.f ? quantize4(v[u], s, r) : 0;
      }
    } else {
      for (int i = threadIdx.x; i < nq; i += TH)
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

// LDS accesses before it are done, in every wave of the workgroup, before any after it; loads
// from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The stream of weights reads whole 128-byte lines: one load takes 8 rows x 128 bytes, lane
// (r16 = lane % 16, g = lane / 16) the 16-byte chunk g + 4 (r16 / 8) of row r16 % 8, and a second
// one the 8 rows after them. The matrix cores want chunk g (then 4 + g) of row r16 in that
// lane: the two loads' values change places between the halves of each 16 lanes. Loads of 16
// rows x 64 bytes need no change but halve the lines: 6.1 against 6.9 TB/s for a plain stream.
constexpr int DPP_ROW_ROR8 = 0x128;
__device__ __forceinline__ void to_steps(const int4_t& a, const int4_t& b, int4_t& s0, int4_t& s1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s0[i] = __builtin_amdgcn_update_dpp(a[i], b[i], DPP_ROW_ROR8, 0xF, 0xC, false);
    s1[i] = __builtin_amdgcn_update_dpp(b[i], a[i], DPP_ROW_ROR8, 0xF, 0x3, false);
  }
}

// Few rows: the weights are streamed from memory once, straight into the matrix cores'
// registers. A workgroup of 8 waves takes tiles of 16 NC channels (gated: 8 NC neurons, gate and
// up rows in 16-row tiles 2 i and 2 i + 1) and up to 16 NR rows; its waves take blocks of 256
// bytes (128 where x comes from the caches: registers) of the length in turn and add their sums through LDS at
// the end of a tile, whole numbers, so the split changes nothing. The next block's loads, also
// those of the next tile, are issued before the current block's products, so that the stream
// does not stop at a tile's end.
// X = void: x is in 8 bits and comes from the caches. Otherwise x is X's rows, which each
// workgroup first holds in 8 bits in its own LDS: that costs less than a launch before this one
// while the rows are few.
constexpr int SK_W = 8;          // waves

// row `row` of x (X's, cols values) into 8 bits at s_q [kpad], by all W waves; its scale
template <typename X, int W>
__device__ __forceinline__ float quantize_to_lds(const X* x, int cols, int kpad, int8_t* s_q,
                                                 unsigned* s_max) {
  unsigned m = 0;
  for (int i = threadIdx.x; i < kpad / 4; i += W * 64) {
    const float4_t v = load4<X, true>(x, i, cols);
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, mag(v[e]));
  }
  m = wg_max<W>(m, s_max);
  float r;
  const float s = row_scale(m, r);
  for (int i = threadIdx.x; i < kpad / 4; i += W * 64)
    reinterpret_cast<int*>(s_q)[i] = s > 0.f ? quantize4(load4<X, true>(x, i, cols), s, r) : 0;
  return s;
}

template <int MODE, int NC, int NR, typename X>
__global__ __launch_bounds__(SK_W * 64, 4) void k_product_few(ProductArgs a) {
  // steps of 64 bytes in a block: as many as keep two workgroups' registers on a compute unit
  constexpr int S = std::is_void<X>::value ? 2 : 4;
  constexpr int BLK = S * 4;  // 16-byte chunks of a block
  constexpr bool G = MODE == MODE_ACT_GATED;
  constexpr bool FUSED = !std::is_void<X>::value;
  constexpr int NT = G ? 8 * NC : 16 * NC;
  __shared__ int s_sum[2][NC * NR][4][64];  // [tile parity][16 x 16 tile][channel][lane]
  __shared__ unsigned s_max[SK_W];
  extern __shared__ __attribute__((aligned(16))) int8_t s_x[];  // FUSED: rows of kpad bytes
  const int nnt = (a.n + NT - 1) / NT;
  const int nmt = FUSED ? (MODE == MODE_LINEAR ? 1 : a.k)
                        : MODE == MODE_LINEAR ? (a.rows + 16 * NR - 1) / (16 * NR) : *a.n_tiles;
  const int total = nmt * nnt;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int nw = G ? 2 * a.n : a.n;
  const int nb = (a.kch + BLK - 1) / BLK;
  const int kpad = nb * BLK * 16;  // FUSED: bytes of a row in LDS

  struct Tile {
    int id, e, r0, r1, n0;
  };
  // the first tile from id on (in steps of the grid) that has rows; its id is >= total if none
  auto tile_from = [&](int id) {
    Tile t{id, 0, 0, 0, 0};
    for (; t.id < total; t.id += gridDim.x) {
      const int mt = t.id / nnt;
      t.n0 = (t.id % nnt) * NT;
      if (FUSED && MODE != MODE_LINEAR) {  // one token: tile row mt is its slot
        t.e = a.src[mt];
        t.r0 = mt;
        t.r1 = mt + 1;
        if ((unsigned)t.e < (unsigned)a.experts) break;
      } else {
        tile_rows<MODE>(a, mt, t.e, t.r0, t.r1);
        t.r1 = min(t.r1, t.r0 + 16 * NR);
        break;
      }
    }
    return t;
  };
  const int lc = g + 4 * (r16 >> 3);  // chunk of 128 bytes that this lane loads
  const int8_t* wbase = nullptr;  // first row of the tile, one for all lanes
  unsigned wrow[NC][2];           // this lane's two rows of each 16 from there, in bytes
  const int8_t* px[NR];
  auto aim = [&](const Tile& t) {
    const int first = G ? 2 * t.n0 : t.n0;
    wbase = a.w + (size_t)t.e * a.w_group + (size_t)first * a.ldw;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int r = (r16 & 7) + 8 * q;
        const int row = G ? (i >> 1) * 32 + 2 * r + (i & 1) : i * 16 + r;
        wrow[i][q] = (unsigned)min(row, nw - 1 - first) * (unsigned)a.ldw;
      }
    }
    if constexpr (!FUSED) {
#pragma unroll
      for (int j = 0; j < NR; ++j)
        px[j] = a.x + (size_t)row_of_x<MODE>(a, min(t.r0 + j * 16 + r16, t.r1 - 1)) * a.ldx + g * 16;
    }
  };
  struct Block {
    int4_t w[S][NC], x[FUSED ? 1 : S][NR];
  };
  auto load = [&](Block& B, int b) {
    const unsigned o = (unsigned)b * (BLK * 16);
#pragma unroll
    for (int s = 0; s < S; s += 2) {
      // past w's row x is zero (its rows are padded to whole blocks), so any chunk will do
      const unsigned c = (unsigned)min(b * BLK + s * 4 + lc, a.kch - 1) * 16;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          B.w[s + q][i] = __builtin_nontemporal_load(
              reinterpret_cast<const int4_t*>(wbase + (size_t)(wrow[i][q] + c)));
    }
    if constexpr (!FUSED) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < NR; ++j)
          B.x[s][j] = *reinterpret_cast<const int4_t*>(px[j] + (size_t)o + s * 64);
    }
  };
  Tile t = tile_from(blockIdx.x);
  if (t.id >= total) return;
  Block B0, B1;
  if (wave < nb) {
    aim(t);
    load(B0, wave);
  }
  for (int i = tid; i < 2 * NC * NR * 256; i += SK_W * 64) (&s_sum[0][0][0][0])[i] = 0;
  const int rows_x = MODE == MODE_LINEAR ? a.rows : 1;
  float xs_own = 0.f;
  if constexpr (FUSED) {
    for (int m = 0; m < rows_x; ++m) {
      const float s = quantize_to_lds<X, SK_W>(reinterpret_cast<const X*>(a.x) + (size_t)m * a.ldx,
                                               a.cols, kpad, s_x + m * kpad,
                                               s_max);
      if (m == r16 || MODE != MODE_LINEAR) xs_own = s;
    }
  }
  lds_barrier();
  const int8_t* fx = s_x + (MODE == MODE_LINEAR ? min(r16, rows_x - 1) : 0) * kpad + g * 16;
  for (int par = 0; t.id < total; par ^= 1) {
    const Tile next = tile_from(t.id + gridDim.x);
    int4_t acc[NC][NR];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[i][j] = int4_t{0, 0, 0, 0};
    for (int b = wave; b < nb; b += SK_W) {
      if (b + SK_W < nb) {
        load(B1, b + SK_W);
      } else if (next.id < total) {
        aim(next);
        load(B1, wave);
      }
#pragma unroll
      for (int s = 0; s < S; s += 2) {
        int4_t w[2][NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) to_steps(B0.w[s][i], B0.w[s + 1][i], w[0][i], w[1][i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int4_t x[NR];
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            if constexpr (FUSED)
              x[j] = *reinterpret_cast<const int4_t*>(fx + b * (BLK * 16) + (s + h) * 64);
            else
              x[j] = B0.x[s + h][j];
          }
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h][i], x[j], acc[i][j], 0, 0, 0);
        }
      }
      B0 = B1;
    }
    if (wave < nb) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) atomicAdd(&s_sum[par][i * NR + j][c][lane], acc[i][j][c]);
    }
    // The sums of the tile two before this one were read and cleared before this wave's
    // arrival here, and the other parity's are free to be added to after it.
    lds_barrier();
    auto take = [&](int q) {
      int4_t v;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] = s_sum[par][q][c][lane];
        s_sum[par][q][c][lane] = 0;
      }
      return v;
    };
    // wave w: tiles w, w + 8, ... (gated: pairs of tiles); lane: row r16, channels 4 g .. +3
    for (int q = wave; q < (G ? NC / 2 : NC) * NR; q += SK_W) {
      const int i = q / NR, j = q % NR;
      const int r = t.r0 + j * 16 + r16;
      int4_t v, u = {0, 0, 0, 0};
      if (G) {
        v = take(2 * i * NR + j);
        u = take((2 * i + 1) * NR + j);
      } else {
        v = take(q);
      }
      if (r >= t.r1) continue;
      const float xs = FUSED ? xs_own : a.xs[row_of_x<MODE>(a, r)];
      emit<MODE>(a, t.e, r, xs, t.n0 + i * 16 + 4 * g, v, u);
    }
    t = next;
  }
}

// The down product of one token, with everything around it: each workgroup holds the rows h of
// the token's slots in 8 bits in its LDS, 16 waves take blocks of 256 bytes of all slots'
// lengths in turn for 16 channels of every slot's expert, and the weighted sum over the slots,
// in slot order, is the token's output. Sums of one slot meet in LDS by whole-number adds.
constexpr int TD_W = 16;
constexpr int SK_BLK = 16;       // 16-byte chunks of a block

__global__ __launch_bounds__(TD_W * 64) void k_token_down(ProductArgs a, const float* __restrict__ weights) {
  __shared__ int s_sum[2][64][16];  // [tile parity][slot][channel]
  __shared__ float s_hs[64];
  __shared__ int s_e[64];           // expert of the v-th slot that has one, and its slot
  __shared__ int s_slot[64];
  __shared__ unsigned s_max[64];
  extern __shared__ __attribute__((aligned(16))) int8_t s_h[];  // [slots][kpad]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int nb = (a.kch + SK_BLK - 1) / SK_BLK, kpad = nb * SK_BLK * 16;
  // every wave lists the slots that have an expert
  const int my = lane < a.k ? a.src[lane] : -1;
  const uint64_t on = __ballot((unsigned)my < (unsigned)a.experts);
  const int nv = __popcll(on);
  if (wave == 0 && ((on >> lane) & 1)) {
    const int v = __popcll(on & ((1ull << lane) - 1));
    s_e[v] = my;
    s_slot[v] = lane;
  }
  if (tid < 64) s_max[tid] = 0;
  for (int i = tid; i < 2 * 64 * 16; i += TD_W * 64) (&s_sum[0][0][0])[i] = 0;
  lds_barrier();
  const int units = nv * nb;
  const int nnt = (a.n + 15) / 16;
  int4_t w0[4], w1[4];
  auto load = [&](int4_t* w, int nt, int u) {
    const int8_t* p = a.w + (size_t)__builtin_amdgcn_readfirstlane(s_e[u / nb]) * a.w_group +
                      (size_t)(nt * 16) * a.ldw;
    const int rows = a.n - 1 - nt * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // 8 rows x 128 bytes each (see to_steps)
      const int row = min((r16 & 7) + 8 * (s & 1), rows);
      const int c = min((u % nb) * SK_BLK + (s >> 1) * 8 + g + 4 * (r16 >> 3), a.kch - 1);
      w[s] = __builtin_nontemporal_load(reinterpret_cast<const int4_t*>(
          p + (size_t)((unsigned)row * (unsigned)a.ldw + (unsigned)c * 16)));
    }
  };
  int nt = blockIdx.x;
  if (wave < units && nt < nnt) load(w0, nt, wave);
  // h into 8 bits: the slots' maxima, then the whole numbers
  const float* h = reinterpret_cast<const float*>(a.x);
  for (int v = 0; v < nv; ++v) {
    unsigned m = 0;
    for (int i = tid; i < kpad / 4; i += TD_W * 64) {
      const float4_t t = load4<float, true>(h + (size_t)s_slot[v] * a.ldx, i, a.cols);
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, mag(t[e]));
    }
    for (int o = 32; o; o >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, o));
    if (lane == 0) atomicMax(&s_max[v], m);
  }
  lds_barrier();
  for (int v = 0; v < nv; ++v) {
    float r;
    const float s = row_scale(s_max[v], r);
    if (tid == 0) s_hs[v] = s;
    for (int i = tid; i < kpad / 4; i += TD_W * 64)
      reinterpret_cast<int*>(s_h + v * kpad)[i] =
          s > 0.f ? quantize4(load4<float, true>(h + (size_t)s_slot[v] * a.ldx, i, a.cols), s, r) : 0;
  }
  lds_barrier();
  for (int par = 0; nt < nnt; nt += gridDim.x, par ^= 1) {
    const int nn = nt + gridDim.x;
    int4_t acc = {0, 0, 0, 0};
    for (int u = wave; u < units; u += TD_W) {
      if (u + TD_W < units) load(w1, nt, u + TD_W);
      else if (nn < nnt) load(w1, nn, wave);
      const int8_t* f = s_h + u * (SK_BLK * 16) + g * 16;  // slot u / nb, block u % nb
#pragma unroll
      for (int s = 0; s < 4; s += 2) {
        int4_t m[2];
        to_steps(w0[s], w0[s + 1], m[0], m[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              m[h], *reinterpret_cast<const int4_t*>(f + (s + h) * 64), acc, 0, 0, 0);
      }
      if (u + TD_W >= units || (u + TD_W) / nb != u / nb) {
        if (r16 == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) atomicAdd(&s_sum[par][u / nb][4 * g + j], acc[j]);
        }
        acc = int4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) w0[s] = w1[s];
    }
    lds_barrier();
    if (tid < 16) {
      const int c = nt * 16 + tid;
      float y = 0.f;
      for (int v = 0; v < nv; ++v) {
        const int sum = s_sum[par][v][tid];
        s_sum[par][v][tid] = 0;
        if (c < a.n) {
          const float p = (float)sum * (s_hs[v] * a.ws[(size_t)s_e[v] * a.n + c]);
          y += weights[s_slot[v]] * p;
        }
      }
      if (c < a.n) {
        if (a.out_type == T_F32) static_cast<float*>(a.out)[c] = y;
        else if (a.out_type == T_F16) static_cast<_Float16*>(a.out)[c] = (_Float16)y;
        else static_cast<__bf16*>(a.out)[c] = (__bf16)y;
      }
    }
  }
}

// Many rows: a workgroup of 8 waves takes 256 rows of w (channels; gated: 128 neurons, 16 gate
// rows and their 16 up rows in turn) and TK rows of x over the whole length, in stages of 64
// bytes. Both operands go from memory straight into LDS (global_load_lds_dwordx4: each lane's
// 16 bytes land at the next 16 bytes of a 1 KB block), NS stages deep. Within a block, 16 rows
// of 64 bytes, row r's 16-byte chunk c sits at position (c + r / 4) mod 4 of the row, so that a
// fragment read (16 rows, one chunk each) touches every LDS bank once. A step waits for the
// next stage, refills the buffer that was read with the stage NS ahead, and reads the next
// stage's fragments into registers while the matrix cores take the current ones.
constexpr int T_CH = 256;   // rows of w per tile
constexpr int T_K = 64;     // bytes per stage
constexpr int T_W = 8;      // waves

// this lane's 16 bytes at src to place 16 * lane of the 1 KB block at dst (LDS)
__device__ __forceinline__ void load_block(const int8_t* src, int8_t* dst) {
  __builtin_amdgcn_global_load_lds(reinterpret_cast<const u32x4*>(src),
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// until at most MOST (FEWER: for waves that load one block less a stage) of this wave's loads
// are in flight
template <int MOST, int FEWER>
__device__ __forceinline__ void wait_loads(bool most) {
  if (most)
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(MOST) : "memory");
  else
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(FEWER) : "memory");
}

template <int MODE, int TK>
__global__ __launch_bounds__(T_W * 64) void k_product(ProductArgs a) {
  constexpr bool G = MODE == MODE_ACT_GATED;
  constexpr int NT = G ? T_CH / 2 : T_CH;          // channels (neurons) per tile
  constexpr int WT = TK >= 256 ? 4 : TK >= 128 ? 2 : 1;  // waves along the rows of x
  constexpr int WC = T_W / WT;                     // waves along the channels
  constexpr int NI = T_CH / 16 / WC, NJ = TK / 16 / WT;  // 16 x 16 tiles of a wave
  constexpr int BW = T_CH * T_K, BX = TK * T_K, STAGE = BW + BX;
  constexpr int NS = 4;
  constexpr int NG = STAGE / 1024;                 // 1 KB loads a stage
  constexpr int DPS = (NG + T_W - 1) / T_W;        // most of one wave
  static_assert((NS - 1) * DPS <= 63, "vmcnt range");
  __shared__ __attribute__((aligned(16))) int8_t sbuf[NS * STAGE];
  const int nnt = (a.n + NT - 1) / NT;
  const int nmt = MODE == MODE_LINEAR ? (a.rows + TK - 1) / TK : *a.n_tiles;
  // Tiles in runs of 8 row tiles, channels outer: 32 neighbours share 8 row tiles and 4 channel
  // tiles. Workgroups 8 apart run on one XCD; each XCD takes a run of neighbours.
  const int total = nmt * nnt, per = (total + 7) / 8;
  const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int run = id / (8 * nnt), in = id % (8 * nnt);
  const int rm = min(8, nmt - run * 8);
  const int mt = run * 8 + in % rm, nt = in / rm;
  int e, r0, r1;
  if (!tile_rows<MODE>(a, mt, e, r0, r1)) return;
  r1 = min(r1, r0 + TK);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wt = wave / WC;
  const int r16 = lane & 15, g = lane >> 4;
  const int n0 = nt * NT;
  const int nw = G ? 2 * a.n : a.n;
  const int8_t* w = a.w + (size_t)e * a.w_group;

  // the lane's row in a 16-row block and the chunk its place holds
  const int lr = lane >> 2;
  const int lc = ((lane & 3) - (lr >> 2)) & 3;
  const int8_t* src[DPS];
#pragma unroll
  for (int v = 0; v < DPS; ++v) {
    const int u = wave + T_W * v;  // block of the stage, wave-uniform
    if (u < T_CH / 16) {
      const int row = G ? 2 * (n0 + (u >> 1) * 16 + lr) + (u & 1) : n0 + u * 16 + lr;
      src[v] = w + (size_t)min(row, nw - 1) * a.ldw;
    } else {
      src[v] = a.x + (size_t)row_of_x<MODE>(a, min(r0 + (u - T_CH / 16) * 16 + lr, r1 - 1)) * a.ldx;
    }
  }
  const int nk = (a.kch + 7) / 8 * 2;  // stages: x's rows end in zeros up to 128 bytes
  auto issue = [&](int st, int buf) {
    const int kc = st * (T_K / 16) + lc;
    const int kw = min(kc, a.kch - 1);  // past w's row x is zero: any chunk will do
#pragma unroll
    for (int v = 0; v < DPS; ++v) {
      const int u = wave + T_W * v;
      if (NG % T_W && u >= NG) break;
      load_block(src[v] + (size_t)(u < T_CH / 16 ? kw : kc) * 16, sbuf + buf * STAGE + u * 1024);
    }
  };
  auto frag = [&](const int8_t* base, int block) {
    return *reinterpret_cast<const int4_t*>(base + block * 1024 +
                                            (r16 * 4 + ((g + (r16 >> 2)) & 3)) * 16);
  };
  int4_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = int4_t{0, 0, 0, 0};
  struct Frags {
    int4_t w[NI], x[NJ];
  };
  auto read_frags = [&](Frags& F, int st) {
    const int8_t* base = sbuf + (st % NS) * STAGE;
#pragma unroll
    for (int j = 0; j < NJ; ++j) F.x[j] = frag(base, T_CH / 16 + wt * NJ + j);
#pragma unroll
    for (int i = 0; i < NI; ++i) F.w[i] = frag(base, wc * NI + i);
  };
  auto products = [&](const Frags& F) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(F.w[i], F.x[j], acc[i][j], 0, 0, 0);
  };
  // Past the last stage the refill loads the last stage again (in bounds, never read), so
  // every step has the same loads in flight and no branch.
  const bool most = NG % T_W == 0 || wave < NG % T_W;  // else it loads one block less a stage
  auto step = [&](int st, Frags& Fc, Frags& Fn) {
    wait_loads<(NS - 2) * DPS, (NS - 2) * (DPS - 1)>(most);
    __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);  // this wave's reads of stage st are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    issue(min(st + NS, nk - 1), st % NS);
    read_frags(Fn, st + 1);
    products(Fc);
  };
#pragma unroll
  for (int st = 0; st < NS; ++st) issue(min(st, nk - 1), st);
  wait_loads<(NS - 1) * DPS, (NS - 1) * (DPS - 1)>(most);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  Frags F0, F1;
  read_frags(F0, 0);
  for (int st = 0; st < nk; st += 2) {  // nk is even
    step(st, F0, F1);
    step(st + 1, F1, F0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may land in LDS after the loop
  // lane holds rows 16 j + r16 and channels 16 i + 4 g .. +3 of the wave's part
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int r = r0 + (wt * NJ + j) * 16 + r16;
    if (r >= r1) continue;
    const float xs = a.xs[row_of_x<MODE>(a, r)];
#pragma unroll
    for (int i = 0; i < NI; i += G ? 2 : 1)
      emit<MODE>(a, e, r, xs, n0 + (G ? (wc * NI + i) / 2 : wc * NI + i) * 16 + 4 * g, acc[i][j],
                 acc[G ? i + 1 : i][j]);
  }
}

// workgroups of a kernel that the current device holds at once (asked once per kernel)
template <typename K>
int resident(K kernel, int threads, size_t lds) {
  int dev = 0, cus = 0, per = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, lds) != hipSuccess)
    return 512;
  return std::max(1, cus * per);
}

template <int MODE, int NC, int NR, typename X>
void few_launch(const ProductArgs& a, int64_t row_tiles, size_t lds, hipStream_t s) {
  constexpr int NT = MODE == MODE_ACT_GATED ? 8 * NC : 16 * NC;
  const int64_t tiles = row_tiles * ((a.n + NT - 1) / NT);
  const int at_once = resident(k_product_few<MODE, NC, NR, X>, SK_W * 64, lds);
  k_product_few<MODE, NC, NR, X>
      <<<dim3((unsigned)std::min<int64_t>(tiles, at_once)), dim3(SK_W * 64), lds, s>>>(a);
}

template <int MODE>
void product_launch(ProductArgs a, hipStream_t s) {
  a.vec_out = a.ldo % 4 == 0 &&
              reinterpret_cast<uintptr_t>(a.out) % (a.out_type == T_F32 ? 16 : 8) == 0;
  const int64_t tiles = MODE == MODE_LINEAR ? ((int64_t)a.rows + a.tile - 1) / a.tile : a.max_tiles;
  if (a.tile == 16) {
    few_launch<MODE, MODE == MODE_ACT_GATED ? 2 : 1, 1, void>(a, tiles, 0, s);
  } else if (a.tile == 32) {
    few_launch<MODE, MODE == MODE_ACT_GATED ? 2 : 1, 2, void>(a, tiles, 0, s);
  } else {
    constexpr int NT = MODE == MODE_ACT_GATED ? T_CH / 2 : T_CH;
    const dim3 grid((unsigned)((tiles * ((a.n + NT - 1) / NT) + 7) / 8 * 8)), block(T_W * 64);
    if (a.tile == 64) k_product<MODE, 64><<<grid, block, 0, s>>>(a);
    else if (a.tile == 128) k_product<MODE, 128><<<grid, block, 0, s>>>(a);
    else k_product<MODE, 256><<<grid, block, 0, s>>>(a);
  }
}

template <typename T, bool VEC>
void quantize_rows(const QuantArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)std::min(a.rows, 1 << 20));
  const int nq = a.kpad / 4;
  if (nq <= 4 * 64) k_quantize<T, VEC, 1, 4><<<grid, dim3(64), 0, s>>>(a);
  else if (nq <= 4 * 256) k_quantize<T, VEC, 4, 4><<<grid, dim3(256), 0, s>>>(a);
  else if (nq <= 4 * 1024) k_quantize<T, VEC, 16, 4><<<grid, dim3(1024), 0, s>>>(a);
  else k_quantize<T, VEC, 16, 0><<<grid, dim3(1024), 0, s>>>(a);
}

template <typename T>
void quantize_launch(const QuantArgs& a, hipStream_t s) {
  const bool vec = reinterpret_cast<uintptr_t>(a.x) % (4 * sizeof(T)) == 0 && a.ldx % 4 == 0;
  if (vec) quantize_rows<T, true>(a, s);
  else quantize_rows<T, false>(a, s);
}

template <int MODE, typename X>
void fused_launch(ProductArgs a, hipStream_t s) {
  a.vec_out = a.ldo % 4 == 0 &&
              reinterpret_cast<uintptr_t>(a.out) % (a.out_type == T_F32 ? 16 : 8) == 0;
  const size_t rows = MODE == MODE_LINEAR ? a.rows : 1;
  few_launch<MODE, MODE == MODE_ACT_GATED ? 2 : 1, 1, X>(a, MODE == MODE_LINEAR ? 1 : a.k,
                                                         rows * host::i8_kpad(a.cols), s);
}

template <typename X>
void fused_launch(const ProductArgs& a, ProductMode mode, hipStream_t s) {
  if (mode == MODE_LINEAR) fused_launch<MODE_LINEAR, X>(a, s);
  else if (mode == MODE_ACT) fused_launch<MODE_ACT, X>(a, s);
  else fused_launch<MODE_ACT_GATED, X>(a, s);
}

}  // namespace

hipError_t launch_product_fused(const ProductArgs& a, int x_type, ProductMode mode, hipStream_t s) {
  if (x_type == T_F32) fused_launch<float>(a, mode, s);
  else if (x_type == T_F16) fused_launch<_Float16>(a, mode, s);
  else fused_launch<__bf16>(a, mode, s);
  return hipGetLastError();
}

hipError_t launch_token_down(const ProductArgs& a, const float* weights, hipStream_t s) {
  const size_t lds = (size_t)a.k * host::i8_kpad(a.cols);
  const int at_once = resident(k_token_down, TD_W * 64, lds);
  k_token_down<<<dim3((unsigned)std::min((a.n + 15) / 16, at_once)), dim3(TD_W * 64), lds, s>>>(a, weights);
  return hipGetLastError();
}

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
