// Internal interface of the norm and the 4-bit blocks (sffn_norm.hip, sffn_mx4.hip) towards the
// C-ABI host code (sffn_mx4_api.hip). The public interface is include/sparse_ffn_mx4.h.
#pragma once
#include "sffn_i8.h"
#include "sffn_mx4_host.h"

namespace sffn {

enum : int { T_MX4 = 4 };  // beside T_F32 .. T_I8

struct NormArgs {
  const void* x;
  const void* res;  // null: none
  const void* w;    // null: 1
  void* sum;
  void* y;
  void* scale;      // I8: fp32 [rows]; MX4: bytes
  int64_t ldx, ldr, ldsum, ldy, lds;
  int rows, cols, w_type;
  double eps, per_col;  // per_col: 1 / cols
};
hipError_t launch_norm(const NormArgs& a, int x_type, int y_type, hipStream_t s);
hipError_t launch_norm_f32(const NormArgs& a, int y_type, hipStream_t s);
hipError_t launch_norm_f16(const NormArgs& a, int y_type, hipStream_t s);
hipError_t launch_norm_bf16(const NormArgs& a, int y_type, hipStream_t s);

// rows of x into blocks; blocks from the row's end up to `blocks` are written as zeros
struct Mx4QuantArgs {
  const void* x;
  int64_t ldx;
  int rows, cols, blocks;
  uint8_t* q;
  int64_t ldq;
  uint8_t* scale;
  int64_t lds;
};
hipError_t launch_quantize_mx4(const Mx4QuantArgs& a, int x_type, hipStream_t s);

struct Mx4DequantArgs {
  const uint8_t* q;
  int64_t ldq;
  const uint8_t* scale;
  int64_t lds;
  int rows, cols;
  void* y;
  int64_t ldy;
};
hipError_t launch_dequantize_mx4(const Mx4DequantArgs& a, int y_type, hipStream_t s);

struct Mx4ProductArgs {
  const uint8_t* x;   // codes, rows ldx bytes apart
  const uint8_t* xs;  // scales, rows ldxs bytes apart
  int64_t ldx, ldxs;
  int rows;
  const uint8_t* w;
  const uint8_t* ws;
  int64_t ldw, ldws;
  const float* bias;  // may be null
  int n;              // rows of w
  int nb;             // blocks of a row
  int cols;           // values of a row of x
  void* out;
  int64_t ldo;
  int out_type;
};
hipError_t launch_mx4_product(Mx4ProductArgs a, hipStream_t s);
// The same where a.x holds rows of x_type values (a.cols of them, a.ldx elements apart), which the
// kernel holds in 4-bit blocks itself (host::mx4_own).
hipError_t launch_mx4_own(const Mx4ProductArgs& a, int x_type, hipStream_t s);

}  // namespace sffn
