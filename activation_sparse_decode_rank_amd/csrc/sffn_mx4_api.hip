// C-ABI host code of the norm and the 4-bit blocks (include/sparse_ffn_mx4.h): argument checks and
// scratch sizes. Every check happens before anything is enqueued; no C++ exception escapes (nothing
// here allocates or throws).
#include <hip/hip_runtime.h>

#include "../../include/sparse_ffn_mx4.h"
#include "sffn_mx4.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool float_type(int t) { return t == SFFN_F32 || t == SFFN_F16 || t == SFFN_BF16; }
uintptr_t type_size(int t) { return t == SFFN_F32 ? 4 : 2; }
int status(hipError_t e) { return e == hipSuccess ? SFFN_OK : SFFN_ERR_HIP; }

// rows of codes and of scales: their distances hold a row of K values
bool blocks_ok(int64_t ldq, int64_t lds, int K) {
  const int64_t nb = sffn::host::mx4_blocks(K);
  return ldq % 16 == 0 && lds % 16 == 0 && ldq >= 16 * nb && lds >= nb;
}
bool too_far(int64_t ldq, int64_t lds) {
  return ldq > sffn::host::kI8MaxLd || lds > sffn::host::kI8MaxLd;
}

}  // namespace

extern "C" {

int sparse_ffn_rms_norm(const void* x, int32_t dtype, int64_t ldx, const void* residual,
                        int64_t ldr, int32_t rows, int32_t cols, const void* w, int32_t w_dtype,
                        double eps, void* sum, int64_t ldsum, void* y, int32_t y_dtype,
                        int64_t ldy, void* scale, int64_t lds, void* stream) {
  const bool i8 = y_dtype == SFFN_I8, mx4 = y_dtype == SFFN_MX4;
  if (!float_type(dtype) || (!float_type(y_dtype) && !i8 && !mx4) || rows < 0 || cols < 1 ||
      ldx < cols)
    return SFFN_ERR_INVALID;
  if ((w && !float_type(w_dtype)) || !(eps >= 0.0) || eps > 1.7976931348623157e308 ||
      (eps > 0.0 && eps < 2.2250738585072014e-308))
    return SFFN_ERR_INVALID;
  if ((residual != nullptr) != (sum != nullptr) || (sum && (ldr < cols || ldsum < cols)))
    return SFFN_ERR_INVALID;
  if (i8 ? ldy % 16 != 0 || ldy < ((int64_t)cols + 15) / 16 * 16
         : mx4 ? !blocks_ok(ldy, lds, cols) : ldy < cols)
    return SFFN_ERR_INVALID;
  if (cols > sffn::host::kI8MaxCount || (mx4 && too_far(ldy, lds))) return SFFN_ERR_UNSUPPORTED;
  if (rows == 0) return SFFN_OK;
  if (!x || !y || ((i8 || mx4) != (scale != nullptr))) return SFFN_ERR_INVALID;
  const uintptr_t e = type_size(dtype);
  if (!aligned(x, e) || !aligned(residual, e) || !aligned(sum, e) ||
      (w && !aligned(w, type_size(w_dtype))) || !aligned(y, i8 || mx4 ? 16 : type_size(y_dtype)) ||
      !aligned(scale, mx4 ? 16 : 4))
    return SFFN_ERR_INVALID;
  sffn::NormArgs a{};
  a.x = x;
  a.res = residual;
  a.w = w;
  a.sum = sum;
  a.y = y;
  a.scale = scale;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldsum = ldsum;
  a.ldy = ldy;
  a.lds = lds;
  a.rows = rows;
  a.cols = cols;
  a.w_type = w_dtype;
  a.eps = eps;
  a.per_col = 1.0 / cols;
  return status(sffn::launch_norm(a, dtype, y_dtype, static_cast<hipStream_t>(stream)));
}

int sparse_ffn_quantize_mx4(const void* x, int32_t dtype, int64_t ldx, int32_t rows, int32_t cols,
                            uint8_t* q, int64_t ldq, uint8_t* scale, int64_t lds, void* stream) {
  if (!float_type(dtype) || rows < 0 || cols < 1 || ldx < cols || !blocks_ok(ldq, lds, cols))
    return SFFN_ERR_INVALID;
  if (cols > sffn::host::kI8MaxCount || too_far(ldq, lds)) return SFFN_ERR_UNSUPPORTED;
  if (rows == 0) return SFFN_OK;
  if (!x || !q || !scale || !aligned(x, type_size(dtype)) || !aligned(q, 16) || !aligned(scale, 16))
    return SFFN_ERR_INVALID;
  sffn::Mx4QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.blocks = sffn::host::mx4_blocks(cols);
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  a.lds = lds;
  return status(sffn::launch_quantize_mx4(a, dtype, static_cast<hipStream_t>(stream)));
}

int sparse_ffn_dequantize_mx4(const uint8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds,
                              int32_t rows, int32_t cols, void* y, int32_t dtype, int64_t ldy,
                              void* stream) {
  if (!float_type(dtype) || rows < 0 || cols < 1 || ldy < cols || !blocks_ok(ldq, lds, cols))
    return SFFN_ERR_INVALID;
  if (cols > sffn::host::kI8MaxCount || too_far(ldq, lds)) return SFFN_ERR_UNSUPPORTED;
  if (rows == 0) return SFFN_OK;
  if (!q || !scale || !y || !aligned(y, type_size(dtype)) || !aligned(q, 16) || !aligned(scale, 16))
    return SFFN_ERR_INVALID;
  sffn::Mx4DequantArgs a{};
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  a.lds = lds;
  a.rows = rows;
  a.cols = cols;
  a.y = y;
  a.ldy = ldy;
  return status(sffn::launch_dequantize_mx4(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t sparse_ffn_mx4_matmul_work_bytes(int32_t x_dtype, int32_t M, int32_t N, int32_t K) {
  if ((!float_type(x_dtype) && x_dtype != SFFN_MX4) || M < 0 || N < 1 || K < 1 ||
      K > SFFN_MX4_MAX_K)
    return (size_t)-1;
  if (M == 0 || x_dtype == SFFN_MX4 || sffn::host::mx4_own((size_t)M, (size_t)N, K)) return 0;
  return sffn::host::mx4_carve((size_t)M, K).bytes;
}

int sparse_ffn_mx4_matmul(const void* x, int32_t x_dtype, const uint8_t* x_scale, int64_t ldx,
                          int64_t ldxs, int32_t M, int32_t K, const uint8_t* w, int64_t ldw,
                          const uint8_t* w_scale, int64_t ldws, const float* bias, int32_t N,
                          void* y, int32_t y_dtype, int64_t ldy, void* work, size_t work_bytes,
                          void* stream) {
  const bool mx4 = x_dtype == SFFN_MX4;
  if ((!float_type(x_dtype) && !mx4) || !float_type(y_dtype)) return SFFN_ERR_INVALID;
  if (M < 0 || N < 1 || K < 1 || ldy < N || !blocks_ok(ldw, ldws, K)) return SFFN_ERR_INVALID;
  if (mx4 ? K % 32 != 0 || !blocks_ok(ldx, ldxs, K) : ldx < K) return SFFN_ERR_INVALID;
  if (K > SFFN_MX4_MAX_K || too_far(ldw, ldws) || (mx4 && too_far(ldx, ldxs)))
    return SFFN_ERR_UNSUPPORTED;
  // tiles round rows and channels up in 32 bits; a launch holds less than 2^32 threads
  if (M > sffn::host::kI8MaxCount || N > sffn::host::kI8MaxCount ||
      !sffn::host::mx4_launches((size_t)(M > 0 ? M : 1), (size_t)N))
    return SFFN_ERR_UNSUPPORTED;
  if (M == 0) return SFFN_OK;
  if (!x || (mx4 != (x_scale != nullptr)) || !w || !w_scale || !y) return SFFN_ERR_INVALID;
  if (!aligned(x, mx4 ? 16 : type_size(x_dtype)) || !aligned(x_scale, 16) || !aligned(w, 16) ||
      !aligned(w_scale, 16) || !aligned(y, type_size(y_dtype)) || !aligned(bias, 4))
    return SFFN_ERR_INVALID;
  sffn::Mx4ProductArgs a{};
  a.rows = M;
  a.w = w;
  a.ws = w_scale;
  a.ldw = ldw;
  a.ldws = ldws;
  a.bias = bias;
  a.n = N;
  a.nb = sffn::host::mx4_blocks(K);
  a.out = y;
  a.ldo = ldy;
  a.out_type = y_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  a.cols = K;
  // few or short rows: held in 4-bit blocks by the product's own workgroups
  if (!mx4 && sffn::host::mx4_own((size_t)M, (size_t)N, K)) {
    a.x = static_cast<const uint8_t*>(x);
    a.ldx = ldx;
    return status(sffn::launch_mx4_own(a, x_dtype, s));
  }
  if (mx4) {
    a.x = static_cast<const uint8_t*>(x);
    a.xs = x_scale;
    a.ldx = ldx;
    a.ldxs = ldxs;
  } else {
    const sffn::host::Mx4Carve c = sffn::host::mx4_carve((size_t)M, K);
    if (!work || !aligned(work, 256) || work_bytes < c.bytes) return SFFN_ERR_INVALID;
    sffn::Mx4QuantArgs q{};
    q.x = x;
    q.ldx = ldx;
    q.rows = M;
    q.cols = K;
    q.blocks = sffn::host::mx4_padded(K);
    q.q = static_cast<uint8_t*>(work) + c.q;
    q.ldq = (int64_t)q.blocks * 16;
    q.scale = static_cast<uint8_t*>(work) + c.scale;
    q.lds = q.blocks;
    if (sffn::launch_quantize_mx4(q, x_dtype, s) != hipSuccess) return SFFN_ERR_HIP;
    a.x = q.q;
    a.xs = q.scale;
    a.ldx = q.ldq;
    a.ldxs = q.lds;
  }
  return status(sffn::launch_mx4_product(a, s));
}

}  // extern "C"
