// Internal interface of the 8-bit products and the expert layer (sffn_i8.hip,
// sffn_experts.hip, sffn_route.hip) towards the C-ABI host code (sffn_experts_api.hip). The
// public interface is include/sparse_ffn_experts.h.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sffn_i8_host.h"

namespace sffn {

// element types of activations and outputs: the values of the public dtype arguments
enum : int { T_F32 = 0, T_F16 = 1, T_BF16 = 2, T_I8 = 3 };

// rows [0, rows) (or [0, *rows_dev) when that is given) of x into 8 bits; the bytes from cols
// to kpad (a multiple of 16, at most ldq) are written as zeros
struct QuantArgs {
  const void* x;
  int64_t ldx;
  int rows, cols, kpad;
  int8_t* q;
  int64_t ldq;
  float* scale;
  const int32_t* rows_dev;
};
hipError_t launch_quantize(const QuantArgs& a, int dtype, hipStream_t s);

// The slots [0, R) of a chunk that name an expert (idx in [0, E)), sorted by expert: the tables
// of ProductArgs. With the tokens' rows into 8 bits in one launch.
struct SortArgs {
  const int32_t* idx;
  int R, E, tile;
  int32_t *offs, *src, *tiles, *n_tiles;
};
hipError_t launch_sort_and_quantize(const SortArgs& sort, const QuantArgs& a, int dtype,
                                    hipStream_t s);

// What a product does with its sums. LINEAR: y = sum * (sx * sw) + bias in out_type.
// ACT / ACT_GATED: h = relu(...) of an expert, fp32. DOWN: fp32 part rows of an expert.
enum ProductMode : int { MODE_LINEAR = 0, MODE_ACT = 1, MODE_ACT_GATED = 2, MODE_DOWN = 3 };

// One product of 8-bit rows x (tokens) with 8-bit rows w (channels), or of groups of them
// (group e multiplies its rows with
// w + e * w_group).
struct ProductArgs {
  const int8_t* x;     // rows of kch * 16 bytes that end in zeros up to a multiple of 128
  int64_t ldx;         // bytes
  const float* xs;     // scale of each row of x
  int rows;            // rows of x (groups: sorted rows, an upper bound)
  const int8_t* w;
  int64_t ldw;         // bytes
  const float* ws;
  const float* bias;   // may be null
  int n;               // channels (ACT_GATED: neurons, each of two rows of w)
  int kch;             // 16-byte chunks of a row
  int cols;            // values of a row of x (fused forms only)
  unsigned div_nq, div_nb;  // set by launch_token_down
  void* out;
  int64_t ldo;         // elements
  int out_type;
  int tile;            // rows of a tile (host::i8_tile)
  // groups only
  const int32_t* offs;    // [experts + 1] first sorted row of each expert
  const int32_t* tiles;   // [tile] (expert, first sorted row)
  const int32_t* n_tiles;
  const int32_t* src;     // [sorted row] slot t * k + s it stands for
  int max_tiles;
  unsigned* tile_max;     // fused ACT forms: bits of the largest |h| of each (slot, tile)
  int k;                  // slots of a token: row src's token is src / k
  int experts;
  int64_t w_group;        // bytes from an expert's w to the next one's
};
hipError_t launch_product(const ProductArgs& a, ProductMode mode, hipStream_t s);
// The same where a.x holds rows of x_type values (a.cols of them, a.ldx elements apart), which the kernel holds in 8 bits itself (host::i8_fused). LINEAR: a.rows
// rows. ACT, ACT_GATED: one token, a.src is its idx [k] and slot s gives row s of out.
hipError_t launch_product_fused(const ProductArgs& a, int x_type, ProductMode mode, hipStream_t s);
// One token's down products and their weighted sum: a.x holds fp32 rows h (a.cols values, a.ldx
// apart), a.tile_max the a.max_tiles maxima of each that the launch before left, a.src the token's idx [k], a.out the token's output row (host::token_fused).
int act_tiles(int f, bool gated);  // tiles of one slot in the fused ACT forms
hipError_t launch_token_down(ProductArgs a, const float* weights, hipStream_t s);

// x already in 8 bits, rows copied to zero-padded rows of kpad bytes
hipError_t launch_pad_rows(const int8_t* x, int64_t ldx, int rows, int cols, int8_t* q, int kpad,
                           hipStream_t s);

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int T, E, k, score;
  const float* bias;
  int groups, top_groups, group_top, renorm;
  float scale;
  int32_t* idx;
  float* weights;
};
hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s);

struct ExpertsArgs {
  int E, d, f, gated;
  const int8_t* w_act;
  int64_t ld_act;
  const float* act_scale;
  const float* b_act;
  const int8_t* w_down;
  int64_t ld_down;
  const float* down_scale;
};
// backward: the last chunk first (host::chunk_order)
hipError_t run_experts(const ExpertsArgs& a, const void* x, int x_type, int64_t ldx, int T,
                       const int32_t* idx, const float* weights, int k, void* y, int y_type,
                       int64_t ldy, void* work, int chunk, bool backward, hipStream_t s);

}  // namespace sffn
