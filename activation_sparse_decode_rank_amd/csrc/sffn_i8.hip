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
// s_waitcnt operand (gfx9 encoding): LDS reads only (lgkmcnt 0, vmcnt and expcnt at most)
constexpr int I8_WAIT_LGKM0 = 0xC07F;

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
    constexpr int NT = MODE == MODE_ACT_GATED ? T_CH / 2 : T_CH;
    const dim3 grid((unsigned)((tiles * ((a.n + NT - 1) / NT) + 7) / 8 * 8)), block(T_W * 64);
    if (a.tile == 64) k_product<MODE, 64><<<grid, block, 0, s>>>(a);
    else if (a.tile == 128) k_product<MODE, 128><<<grid, block, 0, s>>>(a);
    else k_product<MODE, 256><<<grid, block, 0, s>>>(a);
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
