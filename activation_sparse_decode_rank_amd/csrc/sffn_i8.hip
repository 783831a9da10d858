// Rows held in 8 bits, and products of such rows on the matrix cores (gfx950).
//
// A row r is held as s = max|r| * (1 / 127) and q_j = the whole number nearest to r_j / s. A product
// of two such rows is the exact whole-number sum of q_j w_j (at most 131071 products of two
// 8-bit values fit 32 bits), times the two rows' scales.
#include <algorithm>
#include <atomic>

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
// Bound by that read: 8192 rows of 11008 fp32 in 104 us, 4.3 TB/s with the bytes written; a few
// rows take the 4 us of a launch, two round trips and the barrier.
template <typename T, int W, int NV>
__global__ __launch_bounds__(W * 64) void k_quantize(QuantArgs a) {
  constexpr int TH = W * 64;
  __shared__ unsigned s_max[W];
  const int rows = a.rows_dev ? min(*a.rows_dev, a.rows) : a.rows;
  const int nq = a.kpad / 4;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (size_t)row * a.ldx;
    int* q = reinterpret_cast<int*>(a.q + (size_t)row * a.ldq);
    unsigned m = 0;
    float r;
    float4_t v[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
      for (int u = 0; u < NV; ++u) v[u] = load4<T>(x, threadIdx.x + u * TH, a.cols);
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, mag(v[u][e]));
    } else {
      for (int i = threadIdx.x; i < nq; i += TH) {
        const float4_t t = load4<T>(x, i, a.cols);
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
        q[i] = s > 0.f ? quantize4(load4<T>(x, i, a.cols), s, r) : 0;
    }
  }
}

constexpr int DTPB = 1024;

// sorted rows: offs[e] = first row of expert e (offs[E] = rows in all), src[row] = slot, and
// the tile table (expert, first row), n_tiles. One workgroup of DTPB; a slot's place in its expert is what
// the count of the expert gave it, kept in a register for the first KEEP slots of a thread.
__device__ void sort_slots(const SortArgs& a) {
  const int32_t* __restrict__ idx = a.idx;
  const int R = a.R, E = a.E, tile = a.tile;
  int32_t *offs = a.offs, *src = a.src, *tiles = a.tiles, *n_tiles = a.n_tiles;
  constexpr int KEEP = 8;
  __shared__ int s_cnt[1024], s_at[1024];
  __shared__ int s_sum[2][DTPB / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  s_cnt[tid] = 0;
  __syncthreads();
  int e[KEEP], rank[KEEP];
#pragma unroll
  for (int u = 0; u < KEEP; ++u) {
    const int i = tid + u * DTPB;
    e[u] = i < R ? idx[i] : -1;
  }
#pragma unroll
  for (int u = 0; u < KEEP; ++u)
    if ((unsigned)e[u] < (unsigned)E) rank[u] = atomicAdd(&s_cnt[e[u]], 1);
  __syncthreads();
  const int kept = s_cnt[tid];  // of the slots whose places are known
  __syncthreads();
  for (int i = tid + KEEP * DTPB; i < R; i += DTPB) {
    const int q = idx[i];
    if ((unsigned)q < (unsigned)E) atomicAdd(&s_cnt[q], 1);
  }
  __syncthreads();
  // running sums of rows and tiles over the experts
  const int n = s_cnt[tid], nt = (n + tile - 1) / tile;
  const int rows = wave_incl_scan(n), tls = wave_incl_scan(nt);
  if (lane == 63) {
    s_sum[0][wave] = rows;
    s_sum[1][wave] = tls;
  }
  __syncthreads();
  int o = rows - n, t = tls - nt;
  for (int w = 0; w < wave; ++w) {
    o += s_sum[0][w];
    t += s_sum[1][w];
  }
  if (tid < E) {
    offs[tid] = o;
    for (int i = 0; i < nt; ++i) {
      tiles[2 * (t + i)] = tid;
      tiles[2 * (t + i) + 1] = o + i * tile;
    }
  }
  if (tid == E - 1) {
    offs[E] = o + n;
    *n_tiles = t + nt;
  }
  s_at[tid] = o;
  s_cnt[tid] = o + kept;  // where the slots that are counted again go on
  __syncthreads();
#pragma unroll
  for (int u = 0; u < KEEP; ++u)
    if ((unsigned)e[u] < (unsigned)E) src[s_at[e[u]] + rank[u]] = tid + u * DTPB;
  for (int i = tid + KEEP * DTPB; i < R; i += DTPB) {
    const int q = idx[i];
    if ((unsigned)q < (unsigned)E) src[atomicAdd(&s_cnt[q], 1)] = i;
  }
}

__global__ __launch_bounds__(DTPB) void k_sort(SortArgs a) { sort_slots(a); }

// The sort (first workgroup) beside the tokens' rows into 8 bits, RW waves a row: neither needs
// the other, and each alone leaves most of the device idle for a few microseconds.
template <typename T, int RW>
__global__ __launch_bounds__(DTPB) void k_prepare(SortArgs sort, QuantArgs a) {
  constexpr int NV = 4, WAVES = DTPB / 64;
  __shared__ unsigned s_max[WAVES];
  if (blockIdx.x == 0) {
    sort_slots(sort);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = wave / RW;
  const int64_t at = (int64_t)(blockIdx.x - 1) * (WAVES / RW) + group;
  const int row = (int)min<int64_t>(at, a.rows - 1);
  const int i0 = (wave % RW) * 64 + lane, nq = a.kpad / 4;
  const T* x = static_cast<const T*>(a.x) + (size_t)row * a.ldx;
  float4_t v[NV];
  unsigned m = 0;
#pragma unroll
  for (int u = 0; u < NV; ++u) v[u] = load4<T>(x, i0 + u * RW * 64, a.cols);
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, mag(v[u][e]));
  for (int o = 32; o; o >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, o));
  if (lane == 0) s_max[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < RW; ++w) m = max(m, s_max[group * RW + w]);
  if (at >= a.rows) return;
  float r;
  const float s = row_scale(m, r);
  if (wave % RW == 0 && lane == 0) a.scale[row] = s;
  int* q = reinterpret_cast<int*>(a.q + (size_t)row * a.ldq);
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = i0 + u * RW * 64;
    if (i < nq) q[i] = s > 0.f ? quantize4(v[u], s, r) : 0;
  }
}

template <typename T>
void prepare_launch(const SortArgs& sort, const QuantArgs& a, hipStream_t s) {
  const int nq = a.kpad / 4;
  auto grid = [&](int rows) { return dim3((unsigned)(1 + ((int64_t)a.rows + rows - 1) / rows)); };
  if (nq <= 4 * 64) k_prepare<T, 1><<<grid(16), dim3(DTPB), 0, s>>>(sort, a);
  else if (nq <= 4 * 256) k_prepare<T, 4><<<grid(4), dim3(DTPB), 0, s>>>(sort, a);
  else k_prepare<T, 16><<<grid(1), dim3(DTPB), 0, s>>>(sort, a);
}

__global__ __launch_bounds__(TPB) void k_pad_rows(const int8_t* __restrict__ x, int64_t ldx,
                                                  int rows, int cols, int8_t* __restrict__ q,
                                                  int kpad) {
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int j = threadIdx.x; j < kpad; j += TPB)
      q[(size_t)row * kpad + j] = j < cols ? x[(size_t)row * ldx + j] : 0;
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

// The scales of channels (neurons) c .. c + 3 of expert e, and their biases; in the gated form of
// the gate and the up rows. Read before the stores of a tile, which they could not pass.
template <int MODE>
struct Scales {
  static constexpr bool G = MODE == MODE_ACT_GATED;
  float4_t s, u, b;
  bool together;  // gated: relu of a sum times its scale is relu of the sum, times its scale
  __device__ __forceinline__ void load(const ProductArgs& a, int e, int c) {
    typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
    const size_t at = (size_t)e * a.n + c;
    const float* ws = a.ws + (G ? 2 : 1) * at;
    s = u = b = float4_t{0.f, 0.f, 0.f, 0.f};
    if (c + 4 <= a.n) {
      if (G) {
        const vec lo = *reinterpret_cast<const vec*>(ws), hi = *reinterpret_cast<const vec*>(ws + 4);
        s = float4_t{lo[0], lo[2], hi[0], hi[2]};
        u = float4_t{lo[1], lo[3], hi[1], hi[3]};
      } else {
        s = *reinterpret_cast<const vec*>(ws);
      }
      if (MODE != MODE_DOWN && a.bias) b = *reinterpret_cast<const vec*>(a.bias + at);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + j >= a.n) break;
        s[j] = ws[G ? 2 * j : j];
        if (G) u[j] = ws[2 * j + 1];
        if (MODE != MODE_DOWN && a.bias) b[j] = a.bias[at + j];
      }
    }
    if (G) {
      together = !a.bias;
#pragma unroll
      for (int j = 0; j < 4; ++j) together = together && s[j] >= 0.f && s[j] < __builtin_inff();
    }
  }
};

// What becomes of the sums at channels (neurons) c .. c + 3: v, and in the gated form u of the up
// rows. xs: the scale of the row of x; ro: the row of out. Returns the largest |h|'s bits (ACT
// forms).
template <int MODE>
__device__ __forceinline__ unsigned emit(const ProductArgs& a, int ro, float xs, int c,
                                         const Scales<MODE>& S, const int4_t& v, const int4_t& u) {
  if (c >= a.n) return 0;
  unsigned big = 0;
  const int left = a.n - c;
  const size_t o = (size_t)ro * a.ldo + c;
  float4_t y;
  if constexpr (MODE == MODE_ACT || MODE == MODE_ACT_GATED) {
    // h in 64 bits up to its one rounding: it decides between whole numbers afterwards
    if (MODE == MODE_ACT_GATED && S.together) {
      // the scales together: two products of 64 bits less for each value (not where a gate's
      // scale is negative, an infinity or NaN)
      const double x2 = (double)xs * (double)xs;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = (float)((double)max(v[j], 0) * (double)u[j] * (x2 * ((double)S.s[j] * (double)S.u[j])));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        double h = (double)v[j] * ((double)xs * (double)S.s[j]) + (double)S.b[j];
        h = h < 0.0 ? 0.0 : h;  // NaN stays
        if (MODE == MODE_ACT_GATED) h *= (double)u[j] * ((double)xs * (double)S.u[j]);
        y[j] = (float)h;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) big = max(big, mag(y[j]));
    store4<float>(a.out, o, y, left);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = (float)v[j] * (xs * S.s[j]);
      if (MODE == MODE_LINEAR) y[j] += S.b[j];
    }
    if (MODE == MODE_DOWN || a.out_type == T_F32) store4<float>(a.out, o, y, left);
    else if (a.out_type == T_F16) store4<_Float16>(a.out, o, y, left);
    else store4<__bf16>(a.out, o, y, left);
  }
  return big;
}

// The same for channels c .. c + 7 of a plain product
__device__ __forceinline__ void emit8(const ProductArgs& a, int ro, float xs, int c,
                                      const Scales<MODE_LINEAR>& S0, const Scales<MODE_LINEAR>& S1,
                                      const int4_t& v0, const int4_t& v1) {
  if (c >= a.n) return;
  const size_t o = (size_t)ro * a.ldo + c;
  float4_t y0, y1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y0[j] = (float)v0[j] * (xs * S0.s[j]) + S0.b[j];
    y1[j] = (float)v1[j] * (xs * S1.s[j]) + S1.b[j];
  }
  if (a.out_type == T_F32) store8<float>(a.out, o, y0, y1, a.n - c);
  else if (a.out_type == T_F16) store8<_Float16>(a.out, o, y0, y1, a.n - c);
  else store8<__bf16>(a.out, o, y0, y1, a.n - c);
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

// row of out that (sorted) row r gives
template <int MODE>
__device__ __forceinline__ int row_of_out(const ProductArgs& a, int r) {
  return MODE == MODE_DOWN ? a.src[r] : r;
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
// registers. SK waves take a tile of 16 rows of w (16 channels; gated: the gate rows, then the up
// rows of 8 neurons) and up to 16 NR rows of x, one block of 256 bytes of the length after the
// other in turn. Three buffers of a block, its weights and its x, take turns: one is refilled,
// with the block three ahead, also across the end of a tile, as soon as its products are issued
// (and never copied: a copy would wait for the loads). With enough tiles one wave does a tile alone (SK = 1) and meets nobody; otherwise the
// sums of the workgroup's W = SK waves are added through LDS, whole numbers, so the split
// changes nothing.
// X = void: x is in 8 bits and comes from the caches. Otherwise x is X's rows (at most
// host::kFusedRows), which each workgroup first holds in 8 bits in its own LDS while its first
// weights are on their way: that costs less than a launch before this one.
constexpr int F_BLK = 16;  // 16-byte chunks of a block

// M rows of x (X's, cols values) into 8 bits in LDS, by all W waves: W / M waves take a row.
// load() only issues the reads (before the weights', whose wait would include theirs).
template <typename X, int W>
struct RowsToLds {
  static constexpr int KEEP = 6;  // groups of four values per thread that stay in registers
  const X* xr;
  int row, i0, step, nq, cols, M;
  bool kept;
  float4_t v[KEEP];
  __device__ __forceinline__ void load(const X* x, int64_t ldx, int rows, int n, int kpad) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = W / rows;
    M = rows;
    cols = n;
    row = wave / per;
    i0 = (wave % per) * 64 + lane;
    step = per * 64;
    nq = kpad / 4;
    xr = x + (size_t)min(row, M - 1) * ldx;
    kept = nq <= KEEP * step;
    if (kept && row < M) {
#pragma unroll
      for (int u = 0; u < KEEP; ++u) v[u] = load4<X>(xr, i0 + u * step, cols);
    }
  }
  // s_q [M][kpad]; s_max: M cleared words; returns the scale of row lane % 16 (row 0 past the last)
  __device__ __forceinline__ float finish(int kpad, int8_t* s_q, unsigned* s_max) {
    const int lane = threadIdx.x & 63;
    float r;
    if (row < M) {
      unsigned m = 0;
      if (kept) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max(m, mag(v[u][e]));
      } else {
        for (int i = i0; i < nq; i += step) {
          const float4_t t = load4<X>(xr, i, cols);
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max(m, mag(t[e]));
        }
      }
      for (int o = 32; o; o >>= 1) m = max(m, (unsigned)__shfl_xor((int)m, o));
      if (lane == 0) atomicMax(&s_max[row], m);
    }
    lds_barrier();
    if (row < M) {
      const float s = row_scale(s_max[row], r);
      int* q = reinterpret_cast<int*>(s_q + (size_t)row * kpad);
      if (kept) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u)
          if (i0 + u * step < nq) q[i0 + u * step] = s > 0.f ? quantize4(v[u], s, r) : 0;
      } else {
        for (int i = i0; i < nq; i += step)
          q[i] = s > 0.f ? quantize4(load4<X>(xr, i, cols), s, r) : 0;
      }
    }
    return row_scale(s_max[(lane & 15) < M ? lane & 15 : 0], r);
  }
};

// waves per SIMD that the registers of the three buffers leave
template <int NR, typename X>
constexpr int FEW_WAVES = std::is_void<X>::value ? (NR == 1 ? 3 : 2) : 4;

template <int MODE, int NR, typename X, int W, int SK>
__global__ __launch_bounds__(W * 64, (FEW_WAVES<NR, X>)) void k_product_few(ProductArgs a) {
  static_assert(SK == 1 || SK == W, "a wave alone or the whole workgroup");
  constexpr bool G = MODE == MODE_ACT_GATED;
  constexpr bool FUSED = !std::is_void<X>::value;
  constexpr int NT = G ? 8 : 16;  // channels (neurons) of a tile
  __shared__ int s_sum[SK > 1 ? 2 : 1][SK > 1 ? NR : 1][4][64];  // [tile parity][16 rows of x][channel][lane]
  __shared__ unsigned s_max[host::kFusedRows];
  extern __shared__ __attribute__((aligned(16))) int8_t s_x[];  // FUSED: rows of kpad bytes
  const int nnt = (a.n + NT - 1) / NT;
  const int nmt = FUSED ? (MODE == MODE_LINEAR ? 1 : a.k)
                        : MODE == MODE_LINEAR ? (a.rows + 16 * NR - 1) / (16 * NR) : *a.n_tiles;
  const int total = nmt * nnt;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int nw = G ? 2 * a.n : a.n;
  const int nb = (a.kch + F_BLK - 1) / F_BLK;
  const int kpad = nb * F_BLK * 16;  // FUSED: bytes of a row in LDS
  const int wk = SK > 1 ? wave : 0;
  const int first = SK > 1 ? blockIdx.x : blockIdx.x * W + wave;
  const int step = SK > 1 ? gridDim.x : gridDim.x * W;

  struct Tile {
    int id, e, r0, r1, n0;
  };
  // the first tile from id on (in steps of the grid) that has rows; its id is >= total if none
  auto tile_from = [&](int id) {
    Tile t{id, 0, 0, 0, 0};
    for (; t.id < total; t.id += step) {
      const int mt = t.id / nnt;
      t.n0 = (t.id % nnt) * NT;
      if (FUSED && MODE != MODE_LINEAR) {  // one token: row mt is its slot
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
  // this lane's rows of x in a tile
  auto rows_of = [&](const Tile& q, int (&row)[NR]) {
#pragma unroll
    for (int j = 0; j < NR; ++j)
      row[j] = FUSED || q.id >= total ? 0 : row_of_x<MODE>(a, min(q.r0 + j * 16 + r16, q.r1 - 1));
  };
  // the stream: next block (tile, block of it) to load
  const int lc = g + 4 * (r16 >> 3);  // chunk of 128 bytes that this lane loads
  Tile ft = tile_from(first);
  int fb = wk;
  const int8_t* wbase = nullptr;  // first row of w of that tile, one for all lanes
  unsigned wrow[2];               // this lane's two rows from there, in bytes
  int frow[NR], fnext[NR];        // its rows of x, and those of the tile after it
  Tile fn = tile_from(ft.id + step);
  auto aim = [&]() {
    const int row0 = G ? 2 * ft.n0 : ft.n0;
    wbase = a.w + (size_t)ft.e * a.w_group + (size_t)row0 * a.ldw;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int row = G ? 2 * (r16 & 7) + q : (r16 & 7) + 8 * q;
      wrow[q] = (unsigned)min(row, nw - 1 - row0) * (unsigned)a.ldw;
    }
  };
  struct Block {
    int4_t w[4], x[FUSED ? 1 : 4][NR];
  };
  auto fetch = [&](Block& B) {
    if (ft.id >= total) return;
#pragma unroll
    for (int s = 0; s < 4; s += 2) {
      // past w's row x is zero (its rows are padded to whole blocks), so any chunk will do
      const unsigned c = (unsigned)min(fb * F_BLK + s * 4 + lc, a.kch - 1) * 16;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        B.w[s + q] = __builtin_nontemporal_load(
            reinterpret_cast<const int4_t*>(wbase + (size_t)(wrow[q] + c)));
    }
    if constexpr (!FUSED) {
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int8_t* px = a.x + (size_t)frow[j] * a.ldx + g * 16;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          // x's rows are read up to a multiple of 128 bytes: steps past that repeat the last
          const int c = min(fb * F_BLK + s * 4, (a.kch - 1) / 4 * 4);
          B.x[s][j] = *reinterpret_cast<const int4_t*>(px + (size_t)c * 16);
        }
      }
    }
    fb += SK;
    if (fb >= nb) {
      fb = wk;
      ft = fn;
      if (ft.id < total) {
        aim();
        fn = tile_from(ft.id + step);
#pragma unroll
        for (int j = 0; j < NR; ++j) frow[j] = fnext[j];
        rows_of(fn, fnext);
      }
    }
  };
  Tile t = ft;
  if (SK > 1 && t.id >= total) return;
  const bool works = wk < nb;  // a wave past the blocks of a row only meets the others
  const int rows_x = MODE == MODE_LINEAR ? a.rows : 1;
  typedef typename std::conditional<FUSED, X, float>::type XT;
  RowsToLds<XT, W> own;
  if constexpr (FUSED) own.load(reinterpret_cast<const XT*>(a.x), a.ldx, rows_x, a.cols, kpad);
  const int8_t* fx = s_x + (MODE == MODE_LINEAR ? min(r16, rows_x - 1) : 0) * kpad + g * 16;
  Block ring[3];
  // what the end of a tile needs, read at its start
  float xs[NR];
  int ro[NR];
  Scales<MODE> sc;
  auto begin_tile = [&]() {
    if (t.id >= total) return;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const int r = min(t.r0 + j * 16 + r16, t.r1 - 1);
      ro[j] = row_of_out<MODE>(a, r);
      if (!FUSED) xs[j] = a.xs[row_of_x<MODE>(a, r)];
    }
    sc.load(a, t.e, t.n0 + 4 * (G ? g & 1 : g));
  };
  rows_of(ft, frow);
  rows_of(fn, fnext);
  begin_tile();
  if (works && t.id < total) {
    aim();
#pragma unroll
    for (int i = 0; i < 3; ++i) fetch(ring[i]);
  }
  if constexpr (SK > 1)
    for (int i = tid; i < 2 * NR * 256; i += W * 64) (&s_sum[0][0][0][0])[i] = 0;
  if constexpr (FUSED) {
    if (tid < host::kFusedRows) s_max[tid] = 0;
    lds_barrier();
    const float s = own.finish(kpad, s_x, s_max);
#pragma unroll
    for (int j = 0; j < NR; ++j) xs[j] = s;
  }
  if (SK > 1 || FUSED) lds_barrier();

  int4_t acc[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) acc[j] = int4_t{0, 0, 0, 0};
  int b = wk, par = 0;
  // rows 16 j .. +15 of the tile; lane: row r16, channels 4 g .. +3 (gated: lanes of g 2 and 3
  // hold the up sums of those of g 0 and 1)
  auto finish = [&](int j, const int4_t& v, const int4_t& u) {
    const int r = t.r0 + j * 16 + r16;
    unsigned big = 0;
    if (r < t.r1 && (!G || lane < 32)) big = emit<MODE>(a, ro[j], xs[j], t.n0 + 4 * g, sc, v, u);
    if (FUSED && MODE != MODE_LINEAR) {  // the largest |h| of the tile, for the down product
      for (int o = 16; o <= 32; o <<= 1) big = max(big, (unsigned)__shfl_xor((int)big, o));
      if (lane == 0) a.tile_max[t.r0 * nnt + t.n0 / NT] = big;
    }
  };
  auto end_tile = [&]() {
    if constexpr (SK == 1) {
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        int4_t u = {0, 0, 0, 0};
        if (G) {
#pragma unroll
          for (int c = 0; c < 4; ++c) u[c] = __shfl_xor(acc[j][c], 32);
        }
        finish(j, acc[j], u);
      }
    } else {
      if (works) {
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) atomicAdd(&s_sum[par][j][c][lane], acc[j][c]);
      }
      // The sums of the tile two before this one were read and cleared before their reader's
      // arrival here, and the other parity's are free to be added to after it.
      lds_barrier();
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        if (wave != j) continue;
        int4_t v, u = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v[c] = s_sum[par][j][c][lane];
          if (G) u[c] = s_sum[par][j][c][lane ^ 32];
        }
        wave_lds_sync();  // another lane reads what this one clears
#pragma unroll
        for (int c = 0; c < 4; ++c) s_sum[par][j][c][lane] = 0;
        finish(j, v, u);
      }
    }
#pragma unroll
    for (int j = 0; j < NR; ++j) acc[j] = int4_t{0, 0, 0, 0};
    par ^= 1;
    b = wk;
    t = tile_from(t.id + step);
    begin_tile();
  };
  if (!works) {
    while (t.id < total) end_tile();
    return;
  }
  auto block = [&](Block& B) {
#pragma unroll
    for (int s = 0; s < 4; s += 2) {
      int4_t w[2];
      to_steps(B.w[s], B.w[s + 1], w[0], w[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // steps past the row's end repeat earlier ones: their weights do not count
        if (!FUSED && b * F_BLK + (s + h) * 4 >= a.kch) w[h] = int4_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          int4_t x;
          if constexpr (FUSED) x = *reinterpret_cast<const int4_t*>(fx + b * (F_BLK * 16) + (s + h) * 64);
          else x = B.x[s + h][j];
          acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h], x, acc[j], 0, 0, 0);
        }
      }
    }
    fetch(B);
    b += SK;
    if (b >= nb) end_tile();
  };
  while (t.id < total) {
    block(ring[0]);
    if (t.id >= total) break;
    block(ring[1]);
    if (t.id >= total) break;
    block(ring[2]);
  }
}

// The down product of one token, with everything around it: each workgroup holds the rows h of
// the token's slots in 8 bits in its LDS (the scales from the tiles' maxima that the launch
// before left), 16 waves take blocks of 256 bytes of all slots' lengths in turn for 16 channels
// of every slot's expert, and the weighted sum over the slots, in slot order, is the token's
// output. Sums of one slot meet in LDS by whole-number adds. The reads of h go before the
// weights', whose wait would include theirs. 90 MB of weights in 22 us, of which about 9 are the
// launch, h and the end of the tile; that is less than a launch for h, one for the products and
// one for the sum (8 + 22 + 10 us).
constexpr int TD_W = 16;

__global__ __launch_bounds__(TD_W * 64) void k_token_down(ProductArgs a, const float* __restrict__ weights) {
  constexpr int TH = TD_W * 64;
  constexpr int KEEP = 8;           // groups of four values of h per thread that stay in registers
  __shared__ int s_sum[2][64][16];  // [tile parity][slot][channel]
  __shared__ int s_e[64];           // expert of the v-th slot that has one, and its slot
  __shared__ int s_slot[64];
  __shared__ float s_w[64];         // its weight
  __shared__ unsigned s_max[64];    // by slot
  extern __shared__ __attribute__((aligned(16))) int8_t s_h[];  // [slots][kpad]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int nb = (a.kch + F_BLK - 1) / F_BLK, kpad = nb * F_BLK * 16, nq = kpad / 4;
  const float* h = reinterpret_cast<const float*>(a.x);
  const int my = lane < a.k ? a.src[lane] : -1;
  const float my_w = lane < a.k ? weights[lane] : 0.f;
  const int groups = a.k * nq;
  // quotients by whole multiplication: a.div_nq, a.div_nb are 2^32 / nq, / nb rounded up, and
  // the numerators stay below 2^15
  auto by_nq = [&](int i) { return (int)__umulhi((unsigned)i, a.div_nq); };
  auto by_nb = [&](int i) { return nb > 1 ? (int)__umulhi((unsigned)i, a.div_nb) : i; };
  const bool kept = groups <= KEEP * TH;
  float4_t v[KEEP];
  if (kept) {
#pragma unroll
    for (int u = 0; u < KEEP; ++u) {
      const int i = tid + u * TH;
      const int s = by_nq(i);
      if (i < groups) v[u] = load4<float>(h + (size_t)s * a.ldx, i - s * nq, a.cols);
    }
  }
  unsigned most = 0;  // this wave's share of slot wave % k's maxima
  const int ms = wave % a.k, mw = wave / a.k, mstep = ((TD_W - 1 - ms) / a.k + 1) * 64;
  const bool shared = a.k <= TD_W;
  if (shared) {
    for (int i = mw * 64 + lane; i < a.max_tiles; i += mstep)
      most = max(most, a.tile_max[ms * a.max_tiles + i]);
  }
  // every wave lists the slots that have an expert
  const uint64_t on = __ballot((unsigned)my < (unsigned)a.experts);
  const int nv = __popcll(on);
  if (wave == 0) {
    if ((on >> lane) & 1) {
      const int n = __popcll(on & ((1ull << lane) - 1));
      s_e[n] = my;
      s_slot[n] = lane;
      s_w[n] = my_w;
    }
    s_max[lane] = 0;
  }
  for (int i = tid; i < 2 * 64 * 16; i += TH) (&s_sum[0][0][0])[i] = 0;
  lds_barrier();
  const int units = nv * nb;
  const int nnt = (a.n + 15) / 16;
  // the stream: units (blocks of all slots' lengths)
  constexpr int RING = 3;
  int4_t ring[RING][4];
  int nt = blockIdx.x, fnt = nt, fu = wave;
  auto fetch = [&](int4_t* w) {
    if (fnt >= nnt || fu >= units) return;
    const int slot = by_nb(fu), block = fu - slot * nb;
    const int8_t* p = a.w + (size_t)__builtin_amdgcn_readfirstlane(s_e[slot]) * a.w_group +
                      (size_t)(fnt * 16) * a.ldw;
    const int rows = a.n - 1 - fnt * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // 8 rows x 128 bytes each (see to_steps)
      const int row = min((r16 & 7) + 8 * (s & 1), rows);
      const int c = min(block * F_BLK + (s >> 1) * 8 + g + 4 * (r16 >> 3), a.kch - 1);
      w[s] = __builtin_nontemporal_load(reinterpret_cast<const int4_t*>(
          p + (size_t)((unsigned)row * (unsigned)a.ldw + (unsigned)c * 16)));
    }
    fu += TD_W;
    if (fu >= units) {
      fu = wave;
      fnt += gridDim.x;
    }
  };
#pragma unroll
  for (int i = 0; i < RING; ++i) fetch(ring[i]);
  if (shared) {
    for (int o = 32; o; o >>= 1) most = max(most, (unsigned)__shfl_xor((int)most, o));
    if (lane == 0) atomicMax(&s_max[ms], most);
  } else {
    for (int s = wave; s < a.k; s += TD_W) {
      for (int i = lane; i < a.max_tiles; i += 64) most = max(most, a.tile_max[s * a.max_tiles + i]);
      for (int o = 32; o; o >>= 1) most = max(most, (unsigned)__shfl_xor((int)most, o));
      if (lane == 0) s_max[s] = most;
      most = 0;
    }
  }
  lds_barrier();
  // slots without an expert have no maximum, and no unit reads their rows
  auto put = [&](int i, const float4_t& x) {
    float r;
    const float s = row_scale(s_max[by_nq(i)], r);
    reinterpret_cast<int*>(s_h)[i] = s > 0.f ? quantize4(x, s, r) : 0;
  };
  if (kept) {
#pragma unroll
    for (int u = 0; u < KEEP; ++u)
      if (tid + u * TH < groups) put(tid + u * TH, v[u]);
  } else {
    for (int i = tid; i < groups; i += TH)
      put(i, load4<float>(h + (size_t)by_nq(i) * a.ldx, i - by_nq(i) * nq, a.cols));
  }
  lds_barrier();
  int4_t acc = {0, 0, 0, 0};
  int u = wave, par = 0;
  auto end_tile = [&]() {
    lds_barrier();
    if (tid < 16) {
      const int c = nt * 16 + tid;
      float y = 0.f;
      for (int n = 0; n < nv; ++n) {
        const int sum = s_sum[par][n][tid];
        s_sum[par][n][tid] = 0;
        if (c < a.n) {
          float r;
          const float hs = row_scale(s_max[s_slot[n]], r);
          y += s_w[n] * ((float)sum * (hs * a.ws[(size_t)s_e[n] * a.n + c]));
        }
      }
      if (c < a.n) {
        if (a.out_type == T_F32) static_cast<float*>(a.out)[c] = y;
        else if (a.out_type == T_F16) static_cast<_Float16*>(a.out)[c] = (_Float16)y;
        else static_cast<__bf16*>(a.out)[c] = (__bf16)y;
      }
    }
    par ^= 1;
    u = wave;
    nt += gridDim.x;
  };
  if (wave >= units) {  // nothing of the stream is this wave's
    while (nt < nnt) end_tile();
    return;
  }
  // one unit, from a buffer that is refilled with the unit RING ahead and never copied (a copy
  // would wait for the loads)
  auto unit = [&](int4_t* w) {
    const int n = by_nb(u);
    const int8_t* f = s_h + (size_t)s_slot[n] * kpad + (u - n * nb) * (F_BLK * 16) + g * 16;
#pragma unroll
    for (int s = 0; s < 4; s += 2) {
      int4_t m[2];
      to_steps(w[s], w[s + 1], m[0], m[1]);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            m[q], *reinterpret_cast<const int4_t*>(f + (s + q) * 64), acc, 0, 0, 0);
    }
    fetch(w);
    u += TD_W;
    if (u >= units || by_nb(u) != n) {
      if (r16 == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) atomicAdd(&s_sum[par][n][4 * g + j], acc[j]);
      }
      acc = int4_t{0, 0, 0, 0};
    }
    if (u >= units) end_tile();
  };
  while (nt < nnt) {
    unit(ring[0]);
    if (nt >= nnt) break;
    unit(ring[1]);
    if (nt >= nnt) break;
    unit(ring[2]);
  }
}

// Many rows: a workgroup of WC x WT waves takes CH rows of w (channels; gated: CH / 2 neurons, 16
// gate rows and their 16 up rows in turn) and TK rows of x over the whole length, in stages of
// 128 bytes, a whole line of every row. Both operands go from memory straight into LDS
// (global_load_lds_dwordx4: each lane's 16 bytes land at the next 16 bytes of 8 rows x 128
// bytes), NS stages deep. Row r of 16 holds its 16-byte chunk c at place c ^ (r / 2): the sixteen
// lanes that LDS serves together in a 16-byte read (0-3, 12-15 and 20-27 of each 32, and the
// rest) then touch different banks. A stage is two steps of 64 bytes with one barrier between
// them: the first step's products run while the second step's operands are read; at the barrier
// every wave is done with the stage's LDS and the next stage has landed; the second step's
// products run while the freed stage is refilled and the next stage's first operands are read.
// Reads and loads are issued between the products, not before them.
// Bound by the loop, in which the matrix cores are busy 47% of the time, and by what surrounds a
// tile's products: 4096 x 4096 x 11008 in 177 us (2.09 POP/s; under the profiler 182 at least, 194
// in the mean); of a 256 x 256 tile's 57 us about 10 are its first loads and its stores. 256 rows
// of w and of x need 64 KB a stage, a 128 x 64 part for each of 8 waves 24 KB of LDS reads against
// 32 products' 1024 cycles; 256 x 128 tiles take 7% longer, 128 x 128 20%, 32 x 32 products 5%,
// four waves 45%.
// this lane's 16 bytes at src to place 16 * lane of the 1 KB block at dst (LDS)
__device__ __forceinline__ void load_block(const int8_t* src, int8_t* dst) {
  __builtin_amdgcn_global_load_lds(reinterpret_cast<const u32x4*>(src),
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// until at most N of this wave's loads are in flight
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// instruction kinds of __builtin_amdgcn_sched_group_barrier
constexpr int SG_MFMA = 0x8, SG_LOAD = 0x20, SG_LDS_READ = 0x100;

template <int MODE, int CH, int TK, int WC, int WT, int NS>
__global__ __launch_bounds__(WC * WT * 64) void k_product(ProductArgs a) {
  constexpr bool G = MODE == MODE_ACT_GATED;
  // rows of w in an order that gives a lane 8 neighbouring channels in two tiles: 16-bit outputs
  // leave in 64-byte pieces of a row, not 32 (5% less time at 4096 x 4096 x 11008)
  constexpr bool PAIRS = MODE == MODE_LINEAR;
  constexpr int W = WC * WT;
  constexpr int NT = G ? CH / 2 : CH;                    // channels (neurons) per tile
  constexpr int NI = CH / 16 / WC, NJ = TK / 16 / WT;    // 16 x 16 tiles of a wave
  constexpr int STAGE = (CH + TK) * 128;
  constexpr int UW = CH / 8, NG = (CH + TK) / 8;         // 1 KB loads of w, of both, a stage
  constexpr int DPS = NG / W;                            // of one wave
  static_assert(NG % W == 0 && W % 2 == 0 && NI % 2 == 0, "whole loads per wave, pairs of tiles");
  static_assert((NS - 1) * DPS <= 63, "vmcnt range");
  __shared__ __attribute__((aligned(16))) int8_t sbuf[NS * STAGE];
  const int nnt = (a.n + NT - 1) / NT;
  const int nmt = MODE == MODE_LINEAR ? (a.rows + TK - 1) / TK : *a.n_tiles;
  // Tiles in runs of 4 row tiles, channels outer: 32 neighbours share 4 row tiles and 8 channel
  // tiles (4096 x 4096 x 11008: 4% less than with 8 and 4, 10% less than 16 and 2). Workgroups 8 apart run on one XCD; each XCD takes a run of neighbours.
  const int total = nmt * nnt, per = (total + 7) / 8;
  const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int run = id / (4 * nnt), in = id % (4 * nnt);
  const int rm = min(4, nmt - run * 4);
  const int mt = run * 4 + in % rm, nt = in / rm;
  int e, r0, r1;
  if (!tile_rows<MODE>(a, mt, e, r0, r1)) return;
  r1 = min(r1, r0 + TK);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wt = wave / WC;
  const int r16 = lane & 15, g = lane >> 4;
  const int n0 = nt * NT;
  const int nw = G ? 2 * a.n : a.n;
  const int8_t* w = a.w + (size_t)e * a.w_group;

  const int lc = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));  // chunk that this lane loads
  const int8_t* src[DPS];
#pragma unroll
  for (int v = 0; v < DPS; ++v) {
    const int u = wave + W * v;  // 8 rows of the stage, wave-uniform
    if (u < UW) {
      const int R = 8 * u + (lane >> 3);
      const int row = G ? 2 * (n0 + (R >> 5) * 16 + (R & 15)) + ((R >> 4) & 1)
                    : PAIRS ? n0 + (R & ~31) + 8 * ((R >> 2) & 3) + 4 * ((R >> 4) & 1) + (R & 3) : n0 + R;
      src[v] = w + (size_t)min(row, nw - 1) * a.ldw;
    } else {
      src[v] = a.x + (size_t)row_of_x<MODE>(a, min(r0 + 8 * (u - UW) + (lane >> 3), r1 - 1)) * a.ldx;
    }
  }
  const int nk = (a.kch + 7) / 8;  // stages: x's rows end in zeros up to 128 bytes
  auto issue = [&](int st, int buf) {
    const int kc = st * 8 + lc;
    const int kw = min(kc, a.kch - 1);  // past w's row x is zero: any chunk will do
#pragma unroll
    for (int v = 0; v < DPS; ++v) {
      const int u = wave + W * v;
      load_block(src[v] + (size_t)(u < UW ? kw : kc) * 16, sbuf + buf * STAGE + u * 1024);
    }
  };
  int4_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = int4_t{0, 0, 0, 0};
  struct Frags {
    int4_t w[NI], x[NJ];
  };
  // this lane's place in 16 rows, of step 0 and 1
  const int place0 = r16 * 128 + (g ^ (r16 >> 1)) * 16, place1 = place0 ^ 64;
  auto read_frags = [&](Frags& F, int buf, int place) {
    const int8_t* base = sbuf + buf * STAGE + place;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      F.x[j] = *reinterpret_cast<const int4_t*>(base + (CH / 16 + wt * NJ + j) * 2048);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      F.w[i] = *reinterpret_cast<const int4_t*>(base + (wc * NI + i) * 2048);
  };
  auto products = [&](const Frags& F) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(F.w[i], F.x[j], acc[i][j], 0, 0, 0);
  };
  constexpr int READS = NI + NJ, PER = NI * NJ / READS > 0 ? NI * NJ / READS : 1;
  auto barrier = [&]() {
    __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);  // this wave's reads are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  Frags F0, F1;
#pragma unroll
  for (int st = 0; st < NS; ++st) issue(min(st, nk - 1), st);
  wait_loads<(NS - 1) * DPS>();
  barrier();
  read_frags(F0, 0, place0);
  int buf = 0;
  for (int st = 0; st < nk; ++st) {
    read_frags(F1, buf, place1);
    products(F0);
#pragma unroll
    for (int q = 0; q < READS; ++q) {
      __builtin_amdgcn_sched_group_barrier(SG_LDS_READ, 1, 0);
      __builtin_amdgcn_sched_group_barrier(SG_MFMA, PER, 0);
    }
    // Past the last stage the refill loads the last stage again (in bounds, never read), so
    // every stage has the same loads in flight and no branch.
    wait_loads<(NS - 2) * DPS>();
    barrier();
    const int next = buf + 1 == NS ? 0 : buf + 1;
    issue(min(st + NS, nk - 1), buf);
    read_frags(F0, next, place0);
    products(F1);
#pragma unroll
    for (int q = 0; q < READS; ++q) {
      __builtin_amdgcn_sched_group_barrier(SG_LDS_READ, 1, 1);
      if (q < DPS) __builtin_amdgcn_sched_group_barrier(SG_LOAD, 1, 1);
      __builtin_amdgcn_sched_group_barrier(SG_MFMA, PER, 1);
    }
    buf = next;
  }
  wait_loads<0>();  // no load may land in LDS after the loop
  // lane holds rows 16 j + r16 and channels 16 i + 4 g .. +3 (PAIRS: 16 i + 8 g .. +3 in even
  // tiles i, the four after them in the next one) of the wave's part
  constexpr int NE = G ? NI / 2 : NI;
  auto channel = [&](int i) {
    const int t = wc * NE + i;
    return PAIRS ? n0 + (t & ~1) * 16 + 8 * g + 4 * (t & 1) : n0 + t * 16 + 4 * g;
  };
  Scales<MODE> sc[NE];
  float xs[NJ];
  int ro[NJ];
#pragma unroll
  for (int i = 0; i < NE; ++i) sc[i].load(a, e, channel(i));
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int r = min(r0 + (wt * NJ + j) * 16 + r16, r1 - 1);
    xs[j] = a.xs[row_of_x<MODE>(a, r)];
    ro[j] = row_of_out<MODE>(a, r);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    if (r0 + (wt * NJ + j) * 16 + r16 >= r1) continue;
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < NE; i += 2)
        emit8(a, ro[j], xs[j], channel(i), sc[i], sc[i + 1], acc[i][j], acc[i + 1][j]);
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        emit<MODE>(a, ro[j], xs[j], channel(i), sc[i], acc[G ? 2 * i : i][j], acc[G ? 2 * i + 1 : i][j]);
    }
  }
}

template <int MODE, int CH, int TK, int WC, int WT, int NS>
void tile_launch(const ProductArgs& a, int64_t row_tiles, hipStream_t s) {
  constexpr int NT = MODE == MODE_ACT_GATED ? CH / 2 : CH;
  const int64_t tiles = row_tiles * ((a.n + NT - 1) / NT);
  k_product<MODE, CH, TK, WC, WT, NS>
      <<<dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(WC * WT * 64), 0, s>>>(a);
}

// Workgroups of a kernel that the current device holds at once. The last answer is kept: device,
// dynamic LDS (below 2^24) and number in one word.
template <auto Kernel>
int resident(int threads, size_t lds) {
  static std::atomic<uint64_t> kept{0};
  int dev = 0, cus = 0, per = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 512;
  const uint64_t key = ((uint64_t)(dev + 1) << 48) | ((uint64_t)lds << 24);
  const uint64_t last = kept.load(std::memory_order_relaxed);
  if ((last & ~(uint64_t)0xFFFFFF) == key) return (int)(last & 0xFFFFFF);
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      hipOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, threads, lds) != hipSuccess)
    return 512;
  const int n = std::min(std::max(1, cus * per), 0xFFFFFF);
  kept.store(key | (uint64_t)n, std::memory_order_relaxed);
  return n;
}

template <int MODE, int NR, typename X, int W, int SK>
void few_launch(const ProductArgs& a, int64_t tiles, size_t lds, hipStream_t s) {
  const int64_t groups = SK == 1 ? (tiles + W - 1) / W : tiles;
  const int at_once = resident<k_product_few<MODE, NR, X, W, SK>>(W * 64, lds);
  k_product_few<MODE, NR, X, W, SK>
      <<<dim3((unsigned)std::min<int64_t>(groups, at_once)), dim3(W * 64), lds, s>>>(a);
}
// Waves of a tile. One where rows are short (up to 32 blocks) and the tiles give every compute unit
// ten: a wave alone waits for nobody (16 tokens' up products through 8 experts, d 4096, d_ffn
// 11008: 131 us; four waves take 25% more, eight 36%). Else four (16 tokens through the whole layer
// 195 to 205 us, 5% more with eight for the down products), or eight where the workgroups hold x in
// 8 bits themselves and fewer of them do it (1 token x 4096 x 11008: 11.5 us, 12.0 with four).
template <int MODE, int NR, typename X>
void few_launch(const ProductArgs& a, int64_t row_tiles, size_t lds, hipStream_t s) {
  constexpr int NT = MODE == MODE_ACT_GATED ? 8 : 16;
  constexpr int SK = std::is_void<X>::value ? 4 : 8;
  const int64_t tiles = row_tiles * ((a.n + NT - 1) / NT);
  if (tiles >= 2560 && a.kch <= 32 * F_BLK) few_launch<MODE, NR, X, 4, 1>(a, tiles, lds, s);
  else few_launch<MODE, NR, X, SK, SK>(a, tiles, lds, s);
}

template <int MODE>
void product_launch(const ProductArgs& a, hipStream_t s) {
  const int64_t tiles = MODE == MODE_LINEAR ? ((int64_t)a.rows + a.tile - 1) / a.tile : a.max_tiles;
  if (a.tile == 16) {
    few_launch<MODE, 1, void>(a, tiles, 0, s);
  } else if (a.tile == 32) {
    few_launch<MODE, 2, void>(a, tiles, 0, s);
  } else {
    // Channels of a tile of 64 rows: 128, or 64 where those would leave compute units without work
    // (333 x 1013 x 1101: 6.6 us, 9.0 with 128, 14.8 with 256 x 128; 64 experts of 65 rows, d 2048,
    // d_ffn 1408: 104 + 61 us with 128, 121 + 68 with 64, 111 + 67 with 256 x 128).
    const int rows_w = a.n * (MODE == MODE_ACT_GATED ? 2 : 1);
    if (a.tile == 64 && tiles * ((rows_w + 127) / 128) < 512) tile_launch<MODE, 64, 64, 2, 2, 4>(a, tiles, s);
    else if (a.tile == 64) tile_launch<MODE, 128, 64, 2, 2, 3>(a, tiles, s);
    else if (a.tile == 128) tile_launch<MODE, 256, 128, 4, 2, 3>(a, tiles, s);
    else tile_launch<MODE, 256, 256, 2, 4, 2>(a, tiles, s);
  }
}

template <typename T>
void quantize_launch(const QuantArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)std::min(a.rows, 1 << 20));
  const int nq = a.kpad / 4;
  if (nq <= 4 * 64) k_quantize<T, 1, 4><<<grid, dim3(64), 0, s>>>(a);
  else if (nq <= 4 * 256) k_quantize<T, 4, 4><<<grid, dim3(256), 0, s>>>(a);
  else if (nq <= 4 * 1024) k_quantize<T, 16, 4><<<grid, dim3(1024), 0, s>>>(a);
  else k_quantize<T, 16, 0><<<grid, dim3(1024), 0, s>>>(a);
}

template <int MODE, typename X>
void fused_launch(const ProductArgs& a, hipStream_t s) {
  const size_t rows = MODE == MODE_LINEAR ? a.rows : 1;
  few_launch<MODE, 1, X>(a, MODE == MODE_LINEAR ? 1 : a.k,
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

int act_tiles(int f, bool gated) { return gated ? (f + 7) / 8 : (f + 15) / 16; }

hipError_t launch_token_down(ProductArgs a, const float* weights, hipStream_t s) {
  const int nb = (a.kch + F_BLK - 1) / F_BLK, nq = nb * F_BLK * 4;
  auto inverse = [](int n) { return n > 1 ? (unsigned)((((uint64_t)1 << 32) + n - 1) / n) : 0u; };
  a.div_nq = inverse(nq);
  a.div_nb = inverse(nb);
  const size_t lds = (size_t)a.k * host::i8_kpad(a.cols);
  const int at_once = resident<k_token_down>(TD_W * 64, lds);
  k_token_down<<<dim3((unsigned)std::min((a.n + 15) / 16, at_once)), dim3(TD_W * 64), lds, s>>>(a, weights);
  return hipGetLastError();
}

hipError_t launch_quantize(const QuantArgs& a, int dtype, hipStream_t s) {
  if (dtype == T_F32) quantize_launch<float>(a, s);
  else if (dtype == T_F16) quantize_launch<_Float16>(a, s);
  else quantize_launch<__bf16>(a, s);
  return hipGetLastError();
}

hipError_t launch_sort_and_quantize(const SortArgs& sort, const QuantArgs& a, int dtype,
                                    hipStream_t s) {
  if (a.kpad > 4 * 4 * DTPB) {  // longer than a workgroup's registers hold
    k_sort<<<dim3(1), dim3(DTPB), 0, s>>>(sort);
    return launch_quantize(a, dtype, s);
  }
  if (dtype == T_F32) prepare_launch<float>(sort, a, s);
  else if (dtype == T_F16) prepare_launch<_Float16>(sort, a, s);
  else prepare_launch<__bf16>(sort, a, s);
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
