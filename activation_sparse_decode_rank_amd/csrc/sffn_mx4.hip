// Products of rows in 4-bit blocks on the matrix cores (gfx950).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes a block of 32 codes (16 bytes) and its scale byte from
// each lane: lane (r16 = lane % 16, g = lane / 16) holds block g of row r16 of either operand.
#include <algorithm>

#include "sffn_mx4.h"
#include "sffn_mx4_rows.h"
#include "sffn_pipeline.h"

namespace sffn {
namespace {

typedef int int2_t __attribute__((ext_vector_type(2)));
typedef int int8_vec __attribute__((ext_vector_type(8)));

constexpr int FMT_FP4 = 4;  // the instruction's operand format

// acc += the products of 16 rows of w and 16 rows of x, four blocks long
template <int SW, int SX>
__device__ __forceinline__ float4_t mfma16(const int4_t& w, const int4_t& x, const float4_t& acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      int8_vec{w[0], w[1], w[2], w[3], 0, 0, 0, 0}, int8_vec{x[0], x[1], x[2], x[3], 0, 0, 0, 0}, acc,
      FMT_FP4, FMT_FP4, SW, sw, SX, sx);
}

typedef float float16_t __attribute__((ext_vector_type(16)));

// acc += the products of 32 rows of w and 32 rows of x, two blocks long. Lane (r32 = lane % 32,
// h = lane / 32) holds block h of row r32 of either operand; S: the byte of sw and sx.
template <int S>
__device__ __forceinline__ float16_t mfma32(const int4_t& w, const int4_t& x, const float16_t& acc, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
      int8_vec{w[0], w[1], w[2], w[3], 0, 0, 0, 0}, int8_vec{x[0], x[1], x[2], x[3], 0, 0, 0, 0}, acc,
      FMT_FP4, FMT_FP4, S, sw, S, sx);
}

// The bias of four neighbouring channels
__device__ __forceinline__ float4_t bias4(const Mx4ProductArgs& a, int c) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  float4_t b = {0.f, 0.f, 0.f, 0.f};
  if (!a.bias) return b;
  if (c + 4 <= a.n) return *reinterpret_cast<const vec*>(a.bias + c);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < a.n) b[j] = a.bias[c + j];
  return b;
}

// The bias of a tile's 16 channels from n0 on (one tile for all lanes), of which lane group g takes
// four. Scalar loads: a vector load's answer is waited for behind the weights that are on their way
// (1 x 12288 x 49152: 51.6 us, 56.5 with vector loads; 50 to 52 without a bias).
__device__ __forceinline__ float4_t bias16(const Mx4ProductArgs& a, int n0, int g) {
  typedef const float __attribute__((address_space(4))) * scalars;
  float4_t b = {0.f, 0.f, 0.f, 0.f};
  if (!a.bias) return b;
  const scalars p = (scalars)(uintptr_t)a.bias;
  float s[16];
  if (n0 + 16 <= a.n) {
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = p[n0 + j];
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = p[min(n0 + j, a.n - 1)];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = g < 2 ? (g == 0 ? s[e] : s[4 + e]) : g == 2 ? s[8 + e] : s[12 + e];
  return b;
}

// Four neighbouring sums of a row, and their bias, as outputs
__device__ __forceinline__ void emit4(const Mx4ProductArgs& a, int64_t r, int c, float4_t v, const float4_t& b) {
  if (c >= a.n) return;
  v += b;
  const size_t o = (size_t)r * a.ldo + c;
  if (a.out_type == T_F32) store4<float>(a.out, o, v, a.n - c);
  else if (a.out_type == T_F16) store4<_Float16>(a.out, o, v, a.n - c);
  else store4<__bf16>(a.out, o, v, a.n - c);
}

// v, taken where all lanes run: matrix instructions have no effect that would keep the compiler from moving
// them behind a branch that some lanes do not take, where those lanes' operands are missing. It leaves
// exchanges between lanes where they stand, and what they read: this one gives each lane its own value (and
// the wait for the matrix instruction's result is the compiler's, as before any instruction).
constexpr int DPP_SAME_LANE = 0xE4;  // quad_perm 0 1 2 3
__device__ __forceinline__ float4_t in_all_lanes(float4_t v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float own = v[e];  // a bit cast of v[e] itself would take v[0] for every e
    v[e] = __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, own), DPP_SAME_LANE, 0xF, 0xF, true));
  }
  return v;
}

// Few rows, or short ones: the weights are streamed from memory, straight into the matrix cores'
// registers, and x is read from LDS. A tile is 16 rows of w and up to 16 rows of x; a wave takes one
// block of 256 bytes of its length (16 blocks of numbers, whose scales are 16 bytes) after the other.
// Each workgroup first holds its rows of x in 4-bit blocks in its own LDS while its first weights are
// on their way (X = uint8_t: copies those of x that are so held): that costs less than a launch before
// this one, and x is then read from there for every tile.
// S = 8, few rows: eight waves share a tile and take every eighth block of it. Three buffers of a block
// take turns: one is refilled, with the wave's block three ahead, also across the end of a tile, as
// soon as its products are issued. The waves' sums of a tile meet in LDS and are added in the waves'
// order. S = 1, rows of one block: a wave has a tile to itself, and its next one is on its way
// meanwhile; `per` workgroups share the tiles of 16 rows of x. Chunk c (16 bytes) of row r lies at place
// c ^ (r % 16) of the block's 16, so that lanes that LDS serves together touch different banks.
constexpr int G_BLK = host::kMx4Group;  // blocks of numbers (16 bytes of codes) a block of the stream

template <typename X, int S>
__global__ __launch_bounds__(512, 4) void k_mx4_few(Mx4ProductArgs a, int per) {
  constexpr bool HELD = std::is_same<X, uint8_t>::value;
  constexpr int W = 8, G = W / S;  // waves; tiles at once
  static_assert(S == 1 || S == W, "a tile is one wave's, or all waves'");
  __shared__ __attribute__((aligned(16))) float4_t s_sum[S > 1 ? 2 * W * 64 : 1];  // [tile parity][wave][lane]
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];                    // codes, then scales
  const int nnt = (a.n + 15) / 16;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int nbk = S > 1 ? (a.nb + G_BLK - 1) / G_BLK : 1;
  const int down = S > 1 ? 0 : (int)(blockIdx.x / per), r0 = down * 16, rows = min(16, a.rows - r0);
  const int first = wave % S, step = per * G;  // first block of a tile; tiles from one to the next
  // Lane g of four (16 lanes apart) loads word g of a row's 16 scales; the instruction wants bytes
  // g, 4 + g, 8 + g and 12 + g in it: the bytes change places like a 4 x 4 matrix's, between lanes
  // 32 apart, then 16 apart.
  const unsigned far = g < 2 ? 0x05040100u : 0x07060302u, near = g & 1 ? 0x07030501u : 0x06020400u;
  auto to_scales = [&](unsigned v) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const unsigned q = __builtin_amdgcn_perm(p[1], p[0], far);
    const auto r = __builtin_amdgcn_permlane16_swap(q, q, false, false);
    return __builtin_amdgcn_perm(r[1], r[0], near);
  };
  // the stream: next block (tile, block of it) to load
  const int lc = g + 4 * (r16 >> 3);  // chunk of 128 bytes that this lane loads
  int t = ((int)blockIdx.x - down * per) * G + wave / S;
  int ft = t, fb = first;
  const uint8_t *wbase = nullptr, *sbase = nullptr;  // first rows of that tile, one for all lanes
  unsigned wrow[2], srow;  // this lane's two rows of codes, and its row of scales, from there
  auto aim = [&]() {
    const int n0 = ft * 16;
    wbase = a.w + (size_t)n0 * a.ldw;
    sbase = a.ws + (size_t)n0 * a.ldws;
#pragma unroll
    for (int q = 0; q < 2; ++q) wrow[q] = (unsigned)min((r16 & 7) + 8 * q, a.n - 1 - n0) * (unsigned)a.ldw;
    srow = (unsigned)min(r16, a.n - 1 - n0) * (unsigned)a.ldws + 4 * g;
  };
  struct Block {
    int4_t w[4];
    unsigned s;
  };
  auto fetch = [&](Block& B) {
    if (ft >= nnt) return;
#pragma unroll
    for (int s = 0; s < 4; s += 2) {
      // past w's row x is zero, so any chunk will do
      const unsigned c = (unsigned)min(fb * G_BLK + s * 4 + lc, a.nb - 1) * 16;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int4_t* from = reinterpret_cast<const int4_t*>(wbase + (size_t)(wrow[q] + c));
        B.w[s + q] = S > 1 ? __builtin_nontemporal_load(from) : *from;
      }
    }
    B.s = *reinterpret_cast<const unsigned*>(sbase + (size_t)(srow + (unsigned)fb * 16));
    fb += S;
    if (fb >= nbk) {
      fb = first;
      ft += step;
      if (ft < nnt) aim();
    }
  };
  const bool works = first < nbk;  // a wave past the blocks of a row only meets the others
  constexpr int RING = S > 1 ? 3 : 1;
  Block ring[RING];
  if (works && t < nnt) {
    aim();
#pragma unroll
    for (int i = 0; i < RING; ++i) fetch(ring[i]);
  }
  // x's rows: codes [rows][nbk * 256], scales [rows][nbk] of four words, word g the bytes of blocks
  // g, 4 + g, 8 + g and 12 + g
  uint8_t* sc = s_x + (size_t)rows * nbk * 256;
  auto place = [](int r, int c) { return S > 1 ? c : (c ^ r) & 15; };
  if constexpr (HELD) {
    auto copy = [&](int r, int i) {
      int4_t v = {0, 0, 0, 0};
      uint8_t e = 127;
      if (i < a.nb) {
        v = *reinterpret_cast<const int4_t*>(a.x + (size_t)(r0 + r) * a.ldx + 16 * i);
        e = a.xs[(size_t)(r0 + r) * a.ldxs + i];
      }
      const int b = i >> 4, c = i & 15;
      *reinterpret_cast<int4_t*>(s_x + (size_t)(r * nbk + b) * 256 + place(r, c) * 16) = v;
      sc[(size_t)(r * nbk + b) * 16 + (c & 3) * 4 + (c >> 2)] = e;
    };
    if constexpr (S == 1) {
      if (tid < rows * G_BLK) copy(tid / G_BLK, tid % G_BLK);
    } else {
      for (int r = 0; r < rows; ++r)
        for (int i = tid; i < nbk * G_BLK; i += W * 64) copy(r, i);
    }
  } else {
    constexpr int U = 4;  // of them on their way at once: 4 x 4096 x 4096 4.6 us, 5.0 with two
    // a wave takes a block of the length of a row after the other, a lane eight values of it
    const X* x = reinterpret_cast<const X*>(a.x) + (size_t)r0 * a.ldx;
    const int dr = W / nbk, db = W % nbk, c = lane >> 2;
    int r = wave / nbk, b = wave % nbk;
    while (r < rows) {
      vec8<X> f[U];
      int rr[U], bb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        rr[u] = r;
        bb[u] = b;
        if (r < rows) f[u] = raw8(x + (size_t)r * a.ldx + b * 512, lane, a.cols - b * 512);
        r += dr;
        b += db;
        if (b >= nbk) {
          b -= nbk;
          ++r;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (rr[u] < rows) {
          unsigned E;
          const unsigned q = mx4_encode(floats8(f[u]), E);
          *reinterpret_cast<unsigned*>(s_x + (size_t)(rr[u] * nbk + bb[u]) * 256 + place(rr[u], c) * 16 + (lane & 3) * 4) = q;
          if ((lane & 3) == 0) sc[(size_t)(rr[u] * nbk + bb[u]) * 16 + (c & 3) * 4 + (c >> 2)] = (uint8_t)E;
        }
    }
  }
  lds_barrier();
  const int xr = min(r16, rows - 1);  // lanes past the rows read some of x, and write nothing
  const uint8_t *fx = s_x + (size_t)xr * nbk * 256, *fs = sc + (size_t)xr * nbk * 16 + g * 4;
  int at[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) at[s] = place(r16, 4 * s + g) * 16;
  float4_t acc = {0.f, 0.f, 0.f, 0.f};
  int b = first, par = 0;
  auto end_tile = [&]() {
    if constexpr (S > 1) {
      float4_t* sum = s_sum + par * W * 64 + lane;
      sum[wave * 64] = acc;
      float4_t bias;
      if (wave == 0) bias = bias16(a, t * 16, g);
      // The sums of the tile two before this one were read before their reader's arrival here, and
      // the other parity's are free to be written after it.
      lds_barrier();
      if (wave == 0) {
        float4_t v = sum[0];
#pragma unroll
        for (int q = 1; q < W; ++q) {
          const float4_t u = sum[q * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += u[e];
        }
        if (r16 < rows) emit4(a, r0 + r16, t * 16 + 4 * g, v, bias);
      }
      par ^= 1;
    } else {
      const float4_t bias = bias16(a, t * 16, g);
      acc = in_all_lanes(acc);
      if (r16 < rows) emit4(a, r0 + r16, t * 16 + 4 * g, acc, bias);
    }
    acc = float4_t{0.f, 0.f, 0.f, 0.f};
    b = first;
    t += step;
  };
  if (!works) {
    while (t < nnt) end_tile();
    return;
  }
  auto block = [&](Block& B) {
    unsigned sw = to_scales(B.s);
    const int sx = *reinterpret_cast<const int*>(fs + b * 16);
    if ((b + 1) * G_BLK > a.nb) {  // past the row's end the scales may be anything: 1 stands there
      const int left = (a.nb - b * G_BLK - g + 3) >> 2;  // steps of this lane
      const unsigned keep = left >= 4 ? ~0u : (1u << (8 * max(left, 0))) - 1;
      sw = (sw & keep) | (0x7f7f7f7fu & ~keep);
    }
    auto pair = [&](auto s0) {
      constexpr int s = decltype(s0)::value;
      int4_t w[2];
      to_steps(B.w[s], B.w[s + 1], w[0], w[1]);
      const uint8_t* x = fx + b * 256;
      acc = mfma16<s, s>(w[0], *reinterpret_cast<const int4_t*>(x + at[s]), acc, (int)sw, sx);
      acc = mfma16<s + 1, s + 1>(w[1], *reinterpret_cast<const int4_t*>(x + at[s + 1]), acc, (int)sw, sx);
    };
    pair(std::integral_constant<int, 0>{});
    pair(std::integral_constant<int, 2>{});
    if constexpr (S > 1) fetch(B);
    b += S;
    if (b >= nbk) end_tile();
  };
  if constexpr (S > 1) {
    while (t < nnt) {
      block(ring[0]);
      if (t >= nnt) break;
      block(ring[1]);
      if (t >= nnt) break;
      block(ring[2]);
    }
  } else {
    // one copy of the code: what a short product takes is latency, and its instructions' first
    while (t < nnt) {
      Block next;
      fetch(next);
      block(ring[0]);
      ring[0] = next;
    }
  }
}

// Many rows: a workgroup of WC x WT waves takes CH rows of w (channels) and TK rows of x over the
// whole length, in stages of 128 bytes (256 values), a whole line of every row. Both operands go
// from memory straight into LDS, two stages deep; row r of 32 holds its 16-byte chunk c at place
// c ^ (r / 2 % 8), so that the lanes that LDS serves together touch different banks. A stage is
// four steps of two blocks; a step's operands are read while the products of the step before it
// run. Before the last step's products every wave is done with the stage's LDS and the next stage
// has landed: they run while the freed stage is refilled and the next stage's first operands are
// read. The scales, 16 bytes of a row for two stages, lie beside the stages; a lane's eight of them
// (blocks h, 2 + h, .., 14 + h) become two words by two permutations, and the matrix instruction
// takes the byte of its step.
// A wave's rows of w are dealt so that a lane's 16 sums are neighbouring channels.
// Rows held in 4-bit blocks already, out in bf16: 4096 x 4096 x 11008 119 us (3.1 PFLOP/s, the last of 2.7
// rounds of tiles 69% full), 4096 x 16384 x 8192 261 us (4.2). The matrix cores are busy 33 to 37% of the
// time. The products alone, without loads and LDS reads, keep them busy 64% (6.3 PFLOP/s), and the loads
// and LDS reads alone take 0.7 of the whole time: neither hides the other, and every stage waits for all
// its loads and for all waves. Power is a part of it: on zeros the same kernel takes 6 to 19% less. Rings
// of three and four stages (of half lines or smaller tiles), four waves of 128 x 128, waves' priorities
// and other orders of the reads, loads and products take as long or longer.
template <int CH, int TK, int WC, int WT>
__global__ __launch_bounds__(WC * WT * 64) void k_mx4_tiles(Mx4ProductArgs a) {
  constexpr int W = WC * WT, NS = 2;
  constexpr int NI = CH / 32 / WC, NJ = TK / 32 / WT;  // 32 x 32 tiles of a wave
  constexpr int ROWS = CH + TK, STAGE = ROWS * 128;
  constexpr int UW = CH / 8, DPS = ROWS / 8 / W;       // 1 KB loads of w a stage; of one wave
  constexpr int SG = ROWS / 64, SPW = (SG + W - 1) / W;  // 1 KB loads of scales for two stages
  static_assert(ROWS / 8 % W == 0 && W % 2 == 0 && CH % 64 == 0 && TK % 64 == 0, "whole loads");
  __shared__ __attribute__((aligned(16))) int8_t sbuf[NS * STAGE];
  __shared__ __attribute__((aligned(16))) int8_t s_scale[2 * ROWS * 16];
  const int nnt = (a.n + CH - 1) / CH, nmt = (a.rows + TK - 1) / TK;
  // Tiles in runs of 4 row tiles, channels outer; workgroups 8 apart run on one XCD, and each XCD
  // takes a run of neighbours.
  const int total = nmt * nnt, per = (total + 7) / 8;
  const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int run = id / (4 * nnt), in = id % (4 * nnt);
  const int rm = min(4, nmt - run * 4);
  const int r0 = (run * 4 + in % rm) * TK, n0 = in / rm * CH;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wc = wave % WC, wt = wave / WC;
  const int r32 = lane & 31, h = lane >> 5;
  // the channel behind row R of the tile
  auto channel = [](int R) { return (R & ~31) + 16 * ((R >> 2) & 1) + 4 * ((R >> 3) & 3) + (R & 3); };
  const uint8_t* wbase = a.w + (size_t)n0 * a.ldw;
  const uint8_t* xbase = a.x + (size_t)r0 * a.ldx;
  // this lane's rows, in bytes from there (below 2^32: 256 rows, 2^24 apart at most)
  unsigned row[DPS];
#pragma unroll
  for (int v = 0; v < DPS; ++v) {
    const int u = wave + W * v, R = 8 * u + (lane >> 3);
    row[v] = u < UW ? (unsigned)min(channel(R), a.n - 1 - n0) * (unsigned)a.ldw
                    : (unsigned)min(R - CH, a.rows - 1 - r0) * (unsigned)a.ldx;
  }
  // the chunk of a line that this lane loads (its row of 32 is 8 (u % 4) + lane / 8)
  const int lc = (lane & 7) ^ ((wave & 1) * 4 + (lane >> 4));
  const uint8_t* sc[SPW];
#pragma unroll
  for (int v = 0; v < SPW; ++v) {
    const int R = ((wave + W * v) % SG) * 64 + lane;
    sc[v] = R < CH ? a.ws + (size_t)min(n0 + channel(R), a.n - 1) * a.ldws
                   : a.xs + (size_t)min(r0 + R - CH, a.rows - 1) * a.ldxs;
  }
  const int nst = (a.nb + 7) / 8;
  auto issue = [&](int st, int buf) {
    const int kc = st * 8 + lc;
    const unsigned k = (unsigned)min(kc, a.nb - 1) * 16;  // past the row's end any chunk will do
#pragma unroll
    for (int v = 0; v < DPS; ++v) {
      const int u = wave + W * v;
      load_block(reinterpret_cast<const int8_t*>((u < UW ? wbase : xbase) + (size_t)(row[v] + k)),
                 sbuf + buf * STAGE + u * 1024);
    }
  };
  auto issue_scales = [&](int grp) {
#pragma unroll
    for (int v = 0; v < SPW; ++v)
      load_block(reinterpret_cast<const int8_t*>(sc[v] + (size_t)grp * 16),
                 s_scale + (grp & 1) * ROWS * 16 + ((wave + W * v) % SG) * 1024);
  };
  float16_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  struct Frags {
    int4_t w[NI], x[NJ];
  };
  struct Scales {
    int w[2][NI], x[2][NJ];
  } S;
  auto read_frags = [&](Frags& F, int buf, int step) {
    const int8_t* base = sbuf + buf * STAGE + r32 * 128 + (((2 * step + h) ^ (r32 >> 1)) & 7) * 16;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      F.x[j] = *reinterpret_cast<const int4_t*>(base + (CH / 32 + wt * NJ + j) * 4096);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      F.w[i] = *reinterpret_cast<const int4_t*>(base + (wc * NI + i) * 4096);
  };
  const unsigned pick = h ? 0x07050301u : 0x06040200u;  // odd or even bytes of eight
  // Scales of group grp (16 blocks). Past the row's end, in the last group, the bytes may be
  // anything: 1 stands there.
  auto read_scales = [&](int grp) {
    const int8_t* base = s_scale + (grp & 1) * ROWS * 16 + r32 * 16;
    unsigned keep[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int left = (a.nb - grp * 16 - 8 * q - h + 1) >> 1;  // blocks of this lane
      keep[q] = left >= 4 ? ~0u : (1u << (8 * max(left, 0))) - 1;
    }
    auto get = [&](int R, int& s0, int& s1) {
      const int4_t v = *reinterpret_cast<const int4_t*>(base + R * 16);
      s0 = (int)((__builtin_amdgcn_perm((unsigned)v[1], (unsigned)v[0], pick) & keep[0]) | (0x7f7f7f7fu & ~keep[0]));
      s1 = (int)((__builtin_amdgcn_perm((unsigned)v[3], (unsigned)v[2], pick) & keep[1]) | (0x7f7f7f7fu & ~keep[1]));
    };
#pragma unroll
    for (int j = 0; j < NJ; ++j) get(CH + (wt * NJ + j) * 32, S.x[0][j], S.x[1][j]);
#pragma unroll
    for (int i = 0; i < NI; ++i) get((wc * NI + i) * 32, S.w[0][i], S.w[1][i]);
  };
  auto products = [&](const Frags& F, auto step) {  // step of the group, 0 .. 7
    constexpr int Q = decltype(step)::value / 4, B = decltype(step)::value % 4;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mfma32<B>(F.w[i], F.x[j], acc[i][j], S.w[Q][i], S.x[Q][j]);
  };
  constexpr int READS = NI + NJ, PER = NI * NJ / READS > 0 ? NI * NJ / READS : 1;
  constexpr int LOADS = (DPS + READS - 1) / READS;
  auto barrier = [&]() {
    __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);  // this wave's reads are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // reads between the products, not before them
  auto mix = [&]() {
#pragma unroll
    for (int q = 0; q < READS; ++q) {
      __builtin_amdgcn_sched_group_barrier(SG_LDS_READ, 1, 0);
      __builtin_amdgcn_sched_group_barrier(SG_MFMA, PER, 0);
    }
  };
  Frags F0, F1;
  issue_scales(0);
#pragma unroll
  for (int st = 0; st < NS; ++st) issue(min(st, nst - 1), st);
  wait_loads<0>();
  barrier();
  read_scales(0);
  read_frags(F0, 0, 0);
  int buf = 0;
  // Stage st, the PH-th of its group. Past the last stage the refill loads the last stage again (in
  // bounds, never read), so every stage has the same loads in flight and no branch.
  auto stage = [&](int st, auto phase) {
    constexpr int PH = decltype(phase)::value;
    read_frags(F1, buf, 1);
    products(F0, std::integral_constant<int, 4 * PH>{});
    mix();
    read_frags(F0, buf, 2);
    products(F1, std::integral_constant<int, 4 * PH + 1>{});
    mix();
    read_frags(F1, buf, 3);
    products(F0, std::integral_constant<int, 4 * PH + 2>{});
    mix();
    wait_loads<0>();
    barrier();
    if (PH == 0) issue_scales(min(st + NS, nst - 1) / 2);
    issue(min(st + NS, nst - 1), buf);
    buf ^= 1;
    read_frags(F0, buf, 0);
    products(F1, std::integral_constant<int, 4 * PH + 3>{});
#pragma unroll
    for (int q = 0; q < READS; ++q) {
      __builtin_amdgcn_sched_group_barrier(SG_LDS_READ, 1, 0);
      __builtin_amdgcn_sched_group_barrier(SG_LOAD, LOADS, 0);
      __builtin_amdgcn_sched_group_barrier(SG_MFMA, PER, 0);
    }
    if (PH == 1) read_scales((st + 1) / 2);
  };
  const int full = a.nb / 8;
  int st = 0;
  for (; st + 2 <= full; st += 2) {
    stage(st, std::integral_constant<int, 0>{});
    stage(st + 1, std::integral_constant<int, 1>{});
  }
  if (st < full) stage(st, std::integral_constant<int, 0>{});
  if (full < nst) {
    // the row ends inside the last stage: the codes of x past its end become zeros
    if (full & 1) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) S.x[0][j] = S.x[1][j];
#pragma unroll
      for (int i = 0; i < NI; ++i) S.w[0][i] = S.w[1][i];
    }
    auto step = [&](auto s) {
      constexpr int Q = decltype(s)::value;
      if (Q > 0) read_frags(F0, buf, Q);
      if (full * 8 + 2 * Q + h >= a.nb) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) F0.x[j] = int4_t{0, 0, 0, 0};
      }
      products(F0, s);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
  wait_loads<0>();  // no load may land in LDS after the loop
  if constexpr (NI == 2 && W * NJ * 4096 <= NS * STAGE) {
    // 16-bit outputs of a whole tile leave 128 bytes of a row at a time, a wave's 64 channels, put
    // together in LDS (4096 x 4096 x 11008: 121 us, 126 with the 32 bytes that a lane holds)
    if (a.out_type != T_F32 && n0 + CH <= a.n) {
      lds_barrier();
      typedef unsigned short h8 __attribute__((ext_vector_type(8)));
      typedef unsigned short h8u __attribute__((ext_vector_type(8), aligned(2)));
      int8_t* own = sbuf + wave * NJ * 4096;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int c = n0 + (wc * NI + i) * 32 + 16 * h;
        float b[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = a.bias ? a.bias[c + e] : 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            h8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float y = acc[i][j][8 * q + e] + b[8 * q + e];
              v[e] = a.out_type == T_F16 ? __builtin_bit_cast(unsigned short, (_Float16)y)
                                         : __builtin_bit_cast(unsigned short, (__bf16)y);
            }
            *reinterpret_cast<h8*>(own + (j * 32 + r32) * 128 + (((4 * i + 2 * h + q) ^ (r32 >> 1)) & 7) * 16) = v;
          }
      }
      wave_lds_sync();
      unsigned short* out = static_cast<unsigned short*>(a.out) + n0 + wc * 64 + (lane & 7) * 8;
#pragma unroll
      for (int q = 0; q < NJ * 4; ++q) {
        const int t = q * 8 + (lane >> 3);
        const h8 v = *reinterpret_cast<const h8*>(own + t * 128 + (((lane & 7) ^ (t >> 1)) & 7) * 16);
        const int r = r0 + wt * NJ * 32 + t;
        if (r < a.rows) *reinterpret_cast<h8u*>(out + (size_t)r * a.ldo) = v;
      }
      return;
    }
  }
  // lane holds row r32 of tile j and channels 16 h .. +15 of tile i
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = n0 + (wc * NI + i) * 32 + 16 * h;
    if (c >= a.n) continue;
    const int left = a.n - c;
    float4_t b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) b[q][e] = a.bias && 4 * q + e < left ? a.bias[c + 4 * q + e] : 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r = r0 + (wt * NJ + j) * 32 + r32;
      if (r >= a.rows) continue;
      const size_t o = (size_t)r * a.ldo + c;
      float4_t v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[q][e] = acc[i][j][4 * q + e] + b[q][e];
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        if (a.out_type == T_F32) store8<float>(a.out, o + 4 * q, v[q], v[q + 1], left - 4 * q);
        else if (a.out_type == T_F16) store8<_Float16>(a.out, o + 4 * q, v[q], v[q + 1], left - 4 * q);
        else store8<__bf16>(a.out, o + 4 * q, v[q], v[q + 1], left - 4 * q);
      }
    }
  }
}

// Some rows, and few tiles: eight waves share a tile of CH rows of w and TK rows of x and split the
// length, in stages of 256 bytes (16 blocks, two lines of every row, NS stages deep): wave q takes
// blocks 2 q and 2 q + 1 of each stage. A tile's chain of dependent products is an eighth as long,
// which is what bounds a tile that a compute unit has to itself. A 16-byte chunk c of row r of 32
// lies at place c ^ (r % 16) of the row's 16. At the end the waves' sums meet in LDS, and each wave
// adds a share of them in the waves' order. 333 x 1013 x 1101 takes 5.3 us, of which a launch is 2 to 3:
// latency; 64 x 4096 x 11008 9 us, 11.5 in tiles whose waves do not split the length.
template <int CH, int TK, int NS>
__global__ __launch_bounds__(512) void k_mx4_split(Mx4ProductArgs a) {
  constexpr int W = 8;
  constexpr int NI = CH / 32, NJ = TK / 32;
  constexpr int ROWS = CH + TK, STAGE = ROWS * 256;
  constexpr int UW = CH / 4, UN = ROWS / 4, DPS = UN / W;  // 1 KB loads (4 rows) of w, of both; of one wave
  constexpr int PIECES = NI * NJ * 4;
  static_assert(UN % W == 0 && ROWS <= 256, "whole loads");
  constexpr int BUF = NS * STAGE > W * PIECES * 1024 ? NS * STAGE : W * PIECES * 1024;
  __shared__ __attribute__((aligned(16))) int8_t sbuf[BUF];
  __shared__ __attribute__((aligned(16))) int8_t s_scale[NS * 256 * 16];
  const int nnt = (a.n + CH - 1) / CH;
  const int n0 = (int)(blockIdx.x % nnt) * CH, r0 = (int)(blockIdx.x / nnt) * TK;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, h = lane >> 5;
  auto channel = [](int R) { return (R & ~31) + 16 * ((R >> 2) & 1) + 4 * ((R >> 3) & 3) + (R & 3); };
  const uint8_t* wbase = a.w + (size_t)n0 * a.ldw;
  const uint8_t* xbase = a.x + (size_t)r0 * a.ldx;
  unsigned row[DPS];
  int lc[DPS];  // the chunk that this lane loads
#pragma unroll
  for (int v = 0; v < DPS; ++v) {
    const int u = wave + W * v, R = 4 * u + (lane >> 4);
    row[v] = u < UW ? (unsigned)min(channel(R), a.n - 1 - n0) * (unsigned)a.ldw
                    : (unsigned)min(R - CH, a.rows - 1 - r0) * (unsigned)a.ldx;
    lc[v] = (lane & 15) ^ (R & 15);
  }
  // waves 0 to 3 load the scales of 64 rows each
  const int sr = min(wave * 64 + lane, ROWS - 1);
  const uint8_t* sc = sr < CH ? a.ws + (size_t)min(n0 + channel(sr), a.n - 1) * a.ldws
                              : a.xs + (size_t)min(r0 + sr - CH, a.rows - 1) * a.ldxs;
  const int nst = (a.nb + 15) / 16;
  auto issue = [&](int st, int buf) {
    if (wave < 4)
      load_block(reinterpret_cast<const int8_t*>(sc + (size_t)st * 16), s_scale + buf * 4096 + wave * 1024);
#pragma unroll
    for (int v = 0; v < DPS; ++v) {
      const int u = wave + W * v;
      // past the row's end any chunk will do
      const unsigned k = (unsigned)min(st * 16 + lc[v], a.nb - 1) * 16;
      load_block(reinterpret_cast<const int8_t*>((u < UW ? wbase : xbase) + (size_t)(row[v] + k)),
                 sbuf + buf * STAGE + u * 1024);
    }
  };
  float16_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) issue(min(st, nst - 1), st);
  const int c = 2 * wave + h;
  const int8_t* at = sbuf + r32 * 256 + ((c ^ r32) & 15) * 16;
  const int8_t* sat = s_scale + r32 * 16 + c;
  int buf = 0;
  for (int st = 0; st < nst; ++st) {
    // the NS - 2 stages after this one stay in flight
    if (wave < 4) wait_loads<(NS - 2) * (DPS + 1)>();
    else wait_loads<(NS - 2) * DPS>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    int4_t fw[NI], fx[NJ];
    int sw[NI], sx[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      fx[j] = *reinterpret_cast<const int4_t*>(at + buf * STAGE + (NI + j) * 8192);
      sx[j] = *reinterpret_cast<const uint8_t*>(sat + buf * 4096 + (NI + j) * 512);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      fw[i] = *reinterpret_cast<const int4_t*>(at + buf * STAGE + i * 8192);
      sw[i] = *reinterpret_cast<const uint8_t*>(sat + buf * 4096 + i * 512);
    }
    // the buffer of the stage before this one is free: every wave read it before the barrier
    issue(min(st + NS - 1, nst - 1), buf == 0 ? NS - 1 : buf - 1);
    if (st * 16 + c >= a.nb) {  // past the row's end: codes of zero and scales of 1
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        fx[j] = int4_t{0, 0, 0, 0};
        sx[j] = 127;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) sw[i] = 127;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mfma32<0>(fw[i], fx[j], acc[i][j], sw[i], sx[j]);
    buf = buf + 1 == NS ? 0 : buf + 1;
    __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);  // this wave's reads are done before the next barrier
  }
  wait_loads<0>();  // no load may land in LDS after the loop
  lds_barrier();
  float4_t* sums = reinterpret_cast<float4_t*>(sbuf) + lane;  // [wave][piece][lane]
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sums[(wave * PIECES + (i * NJ + j) * 4 + q) * 64] =
            float4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  lds_barrier();
  for (int p = wave; p < PIECES; p += W) {
    float4_t v = sums[p * 64];
#pragma unroll
    for (int k = 1; k < W; ++k) {
      const float4_t u = sums[(k * PIECES + p) * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
    }
    const int i = p / (4 * NJ), j = p / 4 % NJ, q = p & 3;
    const int r = r0 + j * 32 + r32;
    const int cq = n0 + i * 32 + 16 * h + 4 * q;
    if (r < a.rows) emit4(a, r, cq, v, bias4(a, cq));
  }
}

// The same with tiles of 16 rows of w and 16 NJ rows of x, for products whose larger tiles would leave
// compute units idle: what one of them can have in flight bounds it. Stages of 512 bytes (32 blocks)
// of a row: wave q takes blocks 4 q to 4 q + 3 of each. Chunk c of row r lies at place c ^ (r % 16) of
// the row's 32. 24 x 11008 x 4096 (512 workgroups) takes 8.0 us, 3.0 TB/s of weights.
template <int NJ>
__global__ __launch_bounds__(512) void k_mx4_split16(Mx4ProductArgs a) {
  constexpr int W = 8, NS = 3, TK = 16 * NJ;
  constexpr int ROWS = 16 + TK, STAGE = ROWS * 512;
  constexpr int UW = 8, DPS = ROWS / 2 / W;  // 1 KB loads (2 rows) of w; of one wave
  constexpr int SROWS = (ROWS + 63) / 64 * 64, SLOADS = SROWS / 64 * 2;  // rows of scales; loads of them
  static_assert(ROWS % 16 == 0 && SLOADS <= W, "whole loads");
  __shared__ __attribute__((aligned(16))) int8_t sbuf[NS * STAGE];
  __shared__ __attribute__((aligned(16))) int8_t s_scale[NS * SROWS * 32];  // [half of a stage][row][16]
  const int nnt = (a.n + 15) / 16;
  const int n0 = (int)(blockIdx.x % nnt) * 16, r0 = (int)(blockIdx.x / nnt) * TK;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const uint8_t* wbase = a.w + (size_t)n0 * a.ldw;
  const uint8_t* xbase = a.x + (size_t)r0 * a.ldx;
  unsigned row[DPS];
  int lc[DPS];  // the chunk that this lane loads
#pragma unroll
  for (int v = 0; v < DPS; ++v) {
    const int u = wave + W * v, R = 2 * u + (lane >> 5);
    row[v] = u < UW ? (unsigned)min(R, a.n - 1 - n0) * (unsigned)a.ldw
                    : (unsigned)min(R - 16, a.rows - 1 - r0) * (unsigned)a.ldx;
    lc[v] = (lane & 31) ^ (R & 15);
  }
  // waves below SLOADS load the scales of 64 rows of one half of a stage
  const int sr = min((wave >> 1) * 64 + lane, ROWS - 1);
  const uint8_t* sc = sr < 16 ? a.ws + (size_t)min(n0 + sr, a.n - 1) * a.ldws
                              : a.xs + (size_t)min(r0 + sr - 16, a.rows - 1) * a.ldxs;
  const int nst = (a.nb + 31) / 32, groups = (a.nb + 15) / 16;
  auto issue = [&](int st, int buf) {
    if (wave < SLOADS)
      load_block(reinterpret_cast<const int8_t*>(sc + (size_t)min(2 * st + (wave & 1), groups - 1) * 16),
                 s_scale + (buf * 2 + (wave & 1)) * SROWS * 16 + (wave >> 1) * 1024);
#pragma unroll
    for (int v = 0; v < DPS; ++v) {
      const int u = wave + W * v;
      // past the row's end any chunk will do
      const unsigned k = (unsigned)min(st * 32 + lc[v], a.nb - 1) * 16;
      load_block(reinterpret_cast<const int8_t*>((u < UW ? wbase : xbase) + (size_t)(row[v] + k)),
                 sbuf + buf * STAGE + u * 1024);
    }
  };
  float4_t acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) issue(min(st, nst - 1), st);
  const int c = 4 * wave + g;
  const int8_t* at = sbuf + r16 * 512 + (c ^ r16) * 16;
  const int8_t* sat = s_scale + (wave >> 2) * SROWS * 16 + r16 * 16 + (c & 15);
  int buf = 0;
  for (int st = 0; st < nst; ++st) {
    // the stage after this one stays in flight
    if (wave < SLOADS) wait_loads<(NS - 2) * (DPS + 1)>();
    else wait_loads<(NS - 2) * DPS>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    int4_t fw = *reinterpret_cast<const int4_t*>(at + buf * STAGE), fx[NJ];
    int sw = *reinterpret_cast<const uint8_t*>(sat + buf * SROWS * 32), sx[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      fx[j] = *reinterpret_cast<const int4_t*>(at + buf * STAGE + (1 + j) * 8192);
      sx[j] = *reinterpret_cast<const uint8_t*>(sat + buf * SROWS * 32 + (1 + j) * 256);
    }
    // the buffer of the stage before this one is free: every wave read it before the barrier
    issue(min(st + NS - 1, nst - 1), buf == 0 ? NS - 1 : buf - 1);
    if (st * 32 + c >= a.nb) {  // past the row's end: codes of zero and scales of 1
      sw = 127;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        fx[j] = int4_t{0, 0, 0, 0};
        sx[j] = 127;
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = mfma16<0, 0>(fw, fx[j], acc[j], sw, sx[j]);
    buf = buf + 1 == NS ? 0 : buf + 1;
    __builtin_amdgcn_s_waitcnt(I8_WAIT_LGKM0);  // this wave's reads are done before the next barrier
  }
  wait_loads<0>();  // no load may land in LDS after the loop
  lds_barrier();
  float4_t* sums = reinterpret_cast<float4_t*>(sbuf) + lane;  // [wave][16 rows of x][lane]
#pragma unroll
  for (int j = 0; j < NJ; ++j) sums[(wave * NJ + j) * 64] = acc[j];
  const float4_t bias = bias4(a, n0 + 4 * g);
  lds_barrier();
  if (wave < NJ) {
    float4_t v = sums[wave * 64];
#pragma unroll
    for (int k = 1; k < W; ++k) {
      const float4_t u = sums[(k * NJ + wave) * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
    }
    const int r = r0 + wave * 16 + r16;
    if (r < a.rows) emit4(a, r, n0 + 4 * g, v, bias);
  }
}

template <int NJ>
void split16_launch(const Mx4ProductArgs& a, hipStream_t s) {
  const int64_t tiles = (((int64_t)a.rows + 16 * NJ - 1) / (16 * NJ)) * (((int64_t)a.n + 15) / 16);
  k_mx4_split16<NJ><<<dim3((unsigned)tiles), dim3(512), 0, s>>>(a);
}

template <int CH, int TK, int NS>
void split_launch(const Mx4ProductArgs& a, hipStream_t s) {
  const int64_t tiles = (((int64_t)a.rows + TK - 1) / TK) * (((int64_t)a.n + CH - 1) / CH);
  k_mx4_split<CH, TK, NS><<<dim3((unsigned)tiles), dim3(512), 0, s>>>(a);
}

template <int CH, int TK, int WC, int WT>
void tile_launch(const Mx4ProductArgs& a, hipStream_t s) {
  const int64_t tiles = (((int64_t)a.rows + TK - 1) / TK) * (((int64_t)a.n + CH - 1) / CH);
  k_mx4_tiles<CH, TK, WC, WT>
      <<<dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(WC * WT * 64), 0, s>>>(a);
}

// Eight waves a tile: 1 row x 12288 x 49152 in 50 us (6.4 TB/s of weights and scales; four waves 52,
// sixteen 81), 1 x 4096 x 11008 in 6.6 (four waves 7.1, sixteen 9.7).
template <typename X>
void few_launch(const Mx4ProductArgs& a, hipStream_t s) {
  const size_t lds = host::mx4_few_lds((size_t)a.rows, a.cols);
  const int at_once = resident<k_mx4_few<X, 8>>(512, lds);
  const int per = std::min((a.n + 15) / 16, at_once);
  k_mx4_few<X, 8><<<dim3((unsigned)per), dim3(512), lds, s>>>(a, per);
}
// As many workgroups as there are eight tiles for, or a device holds
template <typename X>
void short_launch(const Mx4ProductArgs& a, hipStream_t s) {
  const size_t lds = host::mx4_few_lds((size_t)std::min(a.rows, 16), a.cols);
  const int at_once = resident<k_mx4_few<X, 1>>(512, lds), down = (a.rows + 15) / 16;
  const int per = std::max(1, std::min((a.n + 127) / 128, at_once / down));
  k_mx4_few<X, 1><<<dim3((unsigned)(per * down)), dim3(512), lds, s>>>(a, per);
}

}  // namespace

hipError_t launch_mx4_product(Mx4ProductArgs a, hipStream_t s) {
  auto go = [&](int form) {
    switch (form) {
      case host::kMx4Few: few_launch<uint8_t>(a, s); break;
      case host::kMx4Short: short_launch<uint8_t>(a, s); break;
      case host::kMx4Split16: split16_launch<1>(a, s); break;
      case host::kMx4Split16x32: split16_launch<2>(a, s); break;
      case host::kMx4Split32: split_launch<32, 32, 3>(a, s); break;
      case host::kMx4Split64: split_launch<64, 64, 3>(a, s); break;
      case host::kMx4Tile64: tile_launch<64, 64, 2, 2>(a, s); break;
      case host::kMx4Tile64x128: tile_launch<64, 128, 2, 2>(a, s); break;
      case host::kMx4Tile128: tile_launch<128, 128, 2, 2>(a, s); break;
      default: tile_launch<256, 256, 4, 2>(a, s); break;
    }
    return hipGetLastError();
  };
  const host::Mx4Plan p = host::mx4_plan((size_t)a.rows, (size_t)a.n, a.nb);
  const int n = a.n;
  a.n = (int)p.n1;
  const hipError_t e = go(p.form);
  if (e != hipSuccess || a.n == n) return e;
  a.w += (size_t)a.n * a.ldw;
  a.ws += (size_t)a.n * a.ldws;
  if (a.bias) a.bias += a.n;
  a.out = static_cast<char*>(a.out) + (size_t)a.n * (a.out_type == T_F32 ? 4 : 2);
  a.n = n - a.n;
  return go(p.rest);
}

namespace {
template <typename X>
hipError_t own_launch(const Mx4ProductArgs& a, hipStream_t s) {
  if (host::mx4_few((size_t)a.rows, a.cols)) few_launch<X>(a, s);
  else short_launch<X>(a, s);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_mx4_own(const Mx4ProductArgs& a, int x_type, hipStream_t s) {
  if (x_type == T_F32) return own_launch<float>(a, s);
  if (x_type == T_F16) return own_launch<_Float16>(a, s);
  return own_launch<__bf16>(a, s);
}

}  // namespace sffn
