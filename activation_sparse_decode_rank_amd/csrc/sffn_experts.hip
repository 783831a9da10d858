// The routed experts' FFNs on 8-bit weights (gfx950).
//
// The slots (token t, s-th choice) that name an expert are sorted by expert; each expert's
// rows then meet its weights in tiles on the matrix cores (sffn_i8.hip): h = relu(...) as fp32,
// h into 8 bits, the down product of each slot, and the weighted sum over a token's slots in
// slot order. Every sum of the products is a whole number, so nothing depends on the order in
// which the sort leaves an expert's rows.
#include <algorithm>

#include "sffn_device.h"
#include "sffn_i8.h"

namespace sffn {
namespace {

// y_t = sum over slots s in order of weights[t][s] * part[t k + s], slots without an expert
// left out; a thread takes four channels
template <typename T>
__global__ __launch_bounds__(TPB) void k_combine(const float* __restrict__ part, int64_t ldp,
                                                 const int32_t* __restrict__ idx,
                                                 const float* __restrict__ weights, int k, int E,
                                                 int d, int blocks, T* __restrict__ y, int64_t ldy) {
  const int t = blockIdx.x / blocks;
  const int c = 4 * ((blockIdx.x % blocks) * TPB + threadIdx.x);
  if (c >= d) return;
  float4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < k; ++s) {
    const size_t r = (size_t)t * k + s;
    if ((unsigned)idx[r] < (unsigned)E)  // part's rows have room up to a multiple of 64 channels
      v += weights[r] * *reinterpret_cast<const float4_t*>(part + r * ldp + c);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < d) y[(size_t)t * ldy + c + j] = (T)v[j];
}

size_t esize(int type) { return type == T_F32 ? 4 : 2; }

// the weights' side of the two products
ProductArgs act_product(const ExpertsArgs& a) {
  ProductArgs p{};
  p.w = a.w_act;
  p.ldw = a.ld_act;
  p.ws = a.act_scale;
  p.bias = a.b_act;
  p.n = a.f;
  p.kch = (a.d + 15) / 16;
  p.cols = a.d;
  p.out_type = T_F32;
  p.experts = a.E;
  p.w_group = (int64_t)a.f * (a.gated ? 2 : 1) * a.ld_act;
  return p;
}
ProductArgs down_product(const ExpertsArgs& a) {
  ProductArgs p{};
  p.w = a.w_down;
  p.ldw = a.ld_down;
  p.ws = a.down_scale;
  p.n = a.d;
  p.kch = (a.f + 15) / 16;
  p.cols = a.f;
  p.out_type = T_F32;
  p.experts = a.E;
  p.w_group = (int64_t)a.d * a.ld_down;
  return p;
}

// One token: h of its slots, then their down products and weighted sum, in two launches.
hipError_t run_token(const ExpertsArgs& a, const void* x, int x_type, const int32_t* idx,
                     const float* weights, int k, void* y, int y_type, char* work,
                     const host::ExpertsCarve& c, hipStream_t s) {
  ProductArgs up = act_product(a);
  up.x = static_cast<const int8_t*>(x);
  up.rows = k;
  up.out = work + c.h;
  up.ldo = (int64_t)c.ldh;
  up.src = idx;
  up.k = k;
  // act_tiles(f) words a slot: less than the slot's row in 8 bits, which this path does not use
  up.tile_max = reinterpret_cast<unsigned*>(work + c.hq);
  const hipError_t e =
      launch_product_fused(up, x_type, a.gated ? MODE_ACT_GATED : MODE_ACT, s);
  if (e != hipSuccess) return e;
  ProductArgs dn = down_product(a);
  dn.x = reinterpret_cast<const int8_t*>(up.out);
  dn.ldx = up.ldo;
  dn.out = y;
  dn.out_type = y_type;
  dn.src = idx;
  dn.k = k;
  dn.tile_max = up.tile_max;
  dn.max_tiles = act_tiles(a.f, a.gated);
  return launch_token_down(dn, weights, s);
}

}  // namespace

hipError_t run_experts(const ExpertsArgs& a, const void* x, int x_type, int64_t ldx, int T,
                       const int32_t* idx, const float* weights, int k, void* y, int y_type,
                       int64_t ldy, void* work, int chunk, bool backward, hipStream_t s) {
  const host::Chunks chunks(T, chunk);
  for (int64_t n = 0; n < chunks.count; ++n) {
    const int64_t i = backward ? chunks.count - 1 - n : n;
    const int64_t t0 = chunks.first(i);
    const int Tc = chunks.tokens(i);
    const int R = Tc * k;
    const host::ExpertsCarve c = host::experts_carve(a.E, a.d, a.f, (size_t)Tc, (size_t)k);
    char* p = static_cast<char*>(work);
    int32_t* offs = reinterpret_cast<int32_t*>(p + c.offs);
    int32_t* src = reinterpret_cast<int32_t*>(p + c.src);
    int32_t* tiles = reinterpret_cast<int32_t*>(p + c.tiles);
    int32_t* count = reinterpret_cast<int32_t*>(p + c.count);
    const int32_t* ic = idx + (size_t)t0 * k;
    const float* wc = weights + (size_t)t0 * k;
    const char* xc = static_cast<const char*>(x) + (size_t)t0 * ldx * esize(x_type);
    char* yc = static_cast<char*>(y) + (size_t)t0 * ldy * esize(y_type);

    if (Tc == 1 && host::token_fused(a.d, a.f, k)) {
      const hipError_t e = run_token(a, xc, x_type, ic, wc, k, yc, y_type, p, c, s);
      if (e != hipSuccess) return e;
      continue;
    }
    const SortArgs sort{ic, R, a.E, c.tile, offs, src, tiles, count};
    QuantArgs qx{};
    qx.x = xc;
    qx.ldx = ldx;
    qx.rows = Tc;
    qx.cols = a.d;
    qx.kpad = host::i8_kpad(a.d);
    qx.q = reinterpret_cast<int8_t*>(p + c.xq);
    qx.ldq = qx.kpad;
    qx.scale = reinterpret_cast<float*>(p + c.xs);
    hipError_t e = launch_sort_and_quantize(sort, qx, x_type, s);
    if (e != hipSuccess) return e;

    ProductArgs up = act_product(a);
    up.x = qx.q;
    up.ldx = qx.ldq;
    up.xs = qx.scale;
    up.rows = R;
    up.out = p + c.h;
    up.ldo = (int64_t)c.ldh;
    up.offs = offs;
    up.tiles = tiles;
    up.n_tiles = count;
    up.src = src;
    up.max_tiles = c.max_tiles;
    up.tile = c.tile;
    up.k = k;
    e = launch_product(up, a.gated ? MODE_ACT_GATED : MODE_ACT, s);
    if (e != hipSuccess) return e;

    QuantArgs qh{};
    qh.x = up.out;
    qh.ldx = up.ldo;
    qh.rows = R;
    qh.cols = a.f;
    qh.kpad = host::i8_kpad(a.f);
    qh.q = reinterpret_cast<int8_t*>(p + c.hq);
    qh.ldq = qh.kpad;
    qh.scale = reinterpret_cast<float*>(p + c.hs);
    qh.rows_dev = offs + a.E;
    e = launch_quantize(qh, T_F32, s);
    if (e != hipSuccess) return e;

    ProductArgs dn = down_product(a);
    dn.x = qh.q;
    dn.ldx = qh.ldq;
    dn.xs = qh.scale;
    dn.rows = R;
    dn.out = p + c.part;
    dn.ldo = (int64_t)c.ldp;
    dn.offs = offs;
    dn.tiles = tiles;
    dn.n_tiles = count;
    dn.src = src;
    dn.max_tiles = c.max_tiles;
    dn.tile = c.tile;
    dn.k = k;
    e = launch_product(dn, MODE_DOWN, s);
    if (e != hipSuccess) return e;

    const float* part = reinterpret_cast<const float*>(p + c.part);
    const int blocks = (a.d + 4 * TPB - 1) / (4 * TPB);
    const dim3 grid((unsigned)(Tc * blocks)), block(TPB);
    if (y_type == T_F32)
      k_combine<float><<<grid, block, 0, s>>>(part, dn.ldo, ic, wc, k, a.E, a.d, blocks,
                                              reinterpret_cast<float*>(yc), ldy);
    else if (y_type == T_F16)
      k_combine<_Float16><<<grid, block, 0, s>>>(part, dn.ldo, ic, wc, k, a.E, a.d, blocks,
                                                 reinterpret_cast<_Float16*>(yc), ldy);
    else
      k_combine<__bf16><<<grid, block, 0, s>>>(part, dn.ldo, ic, wc, k, a.E, a.d, blocks,
                                               reinterpret_cast<__bf16*>(yc), ldy);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sffn
