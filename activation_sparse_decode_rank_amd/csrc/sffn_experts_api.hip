// C-ABI host code of the expert layer and the 8-bit products (include/sparse_ffn_experts.h):
// argument checks and scratch sizes. Every check happens before anything is enqueued; no C++
// exception escapes (nothing here allocates or throws).
#include <hip/hip_runtime.h>

#include "../../include/sparse_ffn_experts.h"
#include "sffn_i8.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool float_type(int t) { return t == SFFN_F32 || t == SFFN_F16 || t == SFFN_BF16; }
uintptr_t type_size(int t) { return t == SFFN_F32 ? 4 : t == SFFN_I8 ? 1 : 2; }
int64_t row16(int64_t k) { return (k + 15) / 16 * 16; }
int status(hipError_t e) { return e == hipSuccess ? SFFN_OK : SFFN_ERR_HIP; }

// an 8-bit matrix: 16-byte aligned rows of K bytes, ld apart
bool i8_matrix_ok(const void* w, int64_t ld, int64_t K) {
  return w && aligned(w, 16) && ld % 16 == 0 && ld >= row16(K);
}

int check_experts(const sffn_experts_desc* d) {
  if (!d || d->experts < 1 || d->d < 1 || d->d_ffn < 1) return SFFN_ERR_INVALID;
  if (d->gated != 0 && d->gated != 1) return SFFN_ERR_INVALID;
  if (d->experts > SFFN_MAX_EXPERTS || d->d > SFFN_I8_MAX_K || d->d_ffn > SFFN_I8_MAX_K ||
      d->ld_act > sffn::host::kI8MaxLd || d->ld_down > sffn::host::kI8MaxLd)
    return SFFN_ERR_UNSUPPORTED;
  return SFFN_OK;
}

}  // namespace

extern "C" {

int sparse_ffn_route(const void* logits, int32_t dtype, int64_t ld, int32_t T, int32_t E,
                     int32_t k, int32_t score, const float* bias, int32_t groups,
                     int32_t top_groups, int32_t group_top, int32_t renormalize, float scale,
                     int32_t* idx, float* weights, void* stream) {
  if (!float_type(dtype) || T < 0 || E < 1 || k < 1 || k > E || ld < E) return SFFN_ERR_INVALID;
  if (score != SFFN_SCORE_SOFTMAX && score != SFFN_SCORE_SIGMOID) return SFFN_ERR_INVALID;
  if (groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups)
    return SFFN_ERR_INVALID;
  if ((group_top != 1 && group_top != 2) || (renormalize != 0 && renormalize != 1))
    return SFFN_ERR_INVALID;
  if (E > SFFN_MAX_EXPERTS || k > SFFN_MAX_TOPK || groups > 64) return SFFN_ERR_UNSUPPORTED;
  if (T == 0) return SFFN_OK;
  if (!logits || !idx || !weights || !aligned(logits, type_size(dtype)) || !aligned(idx, 4) ||
      !aligned(weights, 4) || !aligned(bias, 4))
    return SFFN_ERR_INVALID;
  sffn::RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.T = T;
  a.E = E;
  a.k = k;
  a.score = score;
  a.bias = bias;
  a.groups = groups;
  a.top_groups = top_groups;
  a.group_top = group_top;
  a.renorm = renormalize;
  a.scale = scale;
  a.idx = idx;
  a.weights = weights;
  return status(sffn::launch_route(a, dtype, static_cast<hipStream_t>(stream)));
}

int sparse_ffn_quantize_rows(const void* x, int32_t dtype, int64_t ldx, int32_t rows,
                             int32_t cols, int8_t* q, int64_t ldq, float* scale, void* stream) {
  if (!float_type(dtype) || rows < 0 || cols < 1 || ldx < cols || ldq % 16 != 0 ||
      ldq < row16(cols))
    return SFFN_ERR_INVALID;
  if (cols > sffn::host::kI8MaxCount) return SFFN_ERR_UNSUPPORTED;  // rounded up in 32 bits
  if (rows == 0) return SFFN_OK;
  if (!x || !q || !scale || !aligned(x, type_size(dtype)) || !aligned(q, 16) || !aligned(scale, 4))
    return SFFN_ERR_INVALID;
  sffn::QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.kpad = (int)row16(cols);
  a.q = q;
  a.ldq = ldq;
  a.scale = scale;
  return status(sffn::launch_quantize(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t sparse_ffn_i8_matmul_work_bytes(int32_t x_dtype, int32_t M, int32_t N, int32_t K) {
  if ((!float_type(x_dtype) && x_dtype != SFFN_I8) || M < 0 || N < 1 || K < 1 ||
      K > SFFN_I8_MAX_K)
    return (size_t)-1;
  if (M == 0 || (x_dtype != SFFN_I8 && sffn::host::i8_fused((size_t)M, K))) return 0;
  return sffn::host::i8_matmul_carve((size_t)M, K).bytes;
}

int sparse_ffn_i8_matmul(const void* x, int32_t x_dtype, const float* x_scale, int64_t ldx,
                         int32_t M, int32_t K, const int8_t* w, int64_t ldw,
                         const float* w_scale, const float* bias, int32_t N, void* y,
                         int32_t y_dtype, int64_t ldy, void* work, size_t work_bytes,
                         void* stream) {
  const bool i8 = x_dtype == SFFN_I8;
  if ((!float_type(x_dtype) && !i8) || !float_type(y_dtype)) return SFFN_ERR_INVALID;
  if (M < 0 || N < 1 || K < 1 || ldx < K || ldy < N) return SFFN_ERR_INVALID;
  if (K > SFFN_I8_MAX_K || ldw > sffn::host::kI8MaxLd) return SFFN_ERR_UNSUPPORTED;
  if ((((int64_t)M + 63) / 64) * (((int64_t)N + 15) / 16) >= (int64_t)1 << 31)
    return SFFN_ERR_UNSUPPORTED;
  // tiles round rows and channels up in 32 bits; a launch holds less than 2^32 threads
  if (M > sffn::host::kI8MaxCount || N > sffn::host::kI8MaxCount ||
      !sffn::host::i8_launches((size_t)M, (size_t)N))
    return SFFN_ERR_UNSUPPORTED;
  if (M == 0) return SFFN_OK;
  if (!x || (i8 != (x_scale != nullptr)) || !w_scale || !y || !i8_matrix_ok(w, ldw, K))
    return SFFN_ERR_INVALID;
  if (!aligned(x, type_size(x_dtype)) || !aligned(y, type_size(y_dtype)) || !aligned(x_scale, 4) ||
      !aligned(w_scale, 4) || !aligned(bias, 4))
    return SFFN_ERR_INVALID;
  sffn::ProductArgs a{};
  a.cols = K;
  a.rows = M;
  a.tile = sffn::host::i8_tile((size_t)M, 1, (size_t)N);
  a.w = w;
  a.ldw = ldw;
  a.ws = w_scale;
  a.bias = bias;
  a.n = N;
  a.kch = (K + 15) / 16;
  a.out = y;
  a.ldo = ldy;
  a.out_type = y_dtype;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // few rows: held in 8 bits by the product's own workgroups
  if (!i8 && sffn::host::i8_fused((size_t)M, K)) {
    a.x = static_cast<const int8_t*>(x);
    a.ldx = ldx;
    return status(sffn::launch_product_fused(a, x_dtype, sffn::MODE_LINEAR, s));
  }
  const sffn::host::I8MatmulCarve c = sffn::host::i8_matmul_carve((size_t)M, K);
  if (!work || !aligned(work, 256) || work_bytes < c.bytes) return SFFN_ERR_INVALID;
  char* p = static_cast<char*>(work);
  const int kpad = sffn::host::i8_kpad(K);
  if (i8) {
    // rows on 16 bytes that need no zeros behind them: read in place, otherwise copied
    if (K % sffn::host::kI8Read == 0 && ldx % 16 == 0 && aligned(x, 16)) {
      a.x = static_cast<const int8_t*>(x);
      a.ldx = ldx;
    } else {
      int8_t* q = reinterpret_cast<int8_t*>(p + c.q);
      const hipError_t e =
          sffn::launch_pad_rows(static_cast<const int8_t*>(x), ldx, M, K, q, kpad, s);
      if (e != hipSuccess) return SFFN_ERR_HIP;
      a.x = q;
      a.ldx = kpad;
    }
    a.xs = x_scale;
  } else {
    sffn::QuantArgs q{};
    q.x = x;
    q.ldx = ldx;
    q.rows = M;
    q.cols = K;
    q.kpad = kpad;
    q.q = reinterpret_cast<int8_t*>(p + c.q);
    q.ldq = kpad;
    q.scale = reinterpret_cast<float*>(p + c.scale);
    if (sffn::launch_quantize(q, x_dtype, s) != hipSuccess) return SFFN_ERR_HIP;
    a.x = q.q;
    a.ldx = kpad;
    a.xs = q.scale;
  }
  return status(sffn::launch_product(a, sffn::MODE_LINEAR, s));
}

size_t sparse_ffn_experts_work_bytes(const sffn_experts_desc* desc, int32_t tokens, int32_t k) {
  if (check_experts(desc) != SFFN_OK || tokens < 1 || k < 1 || k > SFFN_MAX_TOPK) return 0;
  // a chunk never holds more tokens than this
  const size_t most = sffn::host::experts_max_tokens(desc->d, k);
  const size_t T = (size_t)tokens < most ? (size_t)tokens : most;
  return sffn::host::experts_carve(desc->experts, desc->d, desc->d_ffn, T, (size_t)k).bytes;
}

int sparse_ffn_experts(const sffn_experts_desc* desc, const void* x, int32_t x_dtype,
                       int64_t ldx, int32_t T, const int32_t* idx, const float* weights,
                       int32_t k, void* y, int32_t y_dtype, int64_t ldy, void* work,
                       size_t work_bytes, void* stream) {
  const int rc = check_experts(desc);
  if (rc != SFFN_OK) return rc;
  if (!float_type(x_dtype) || !float_type(y_dtype)) return SFFN_ERR_INVALID;
  if (T < 0 || k < 1 || ldx < desc->d || ldy < desc->d) return SFFN_ERR_INVALID;
  if (k > SFFN_MAX_TOPK) return SFFN_ERR_UNSUPPORTED;
  if (T == 0) return SFFN_OK;
  if (!x || !idx || !weights || !y || !desc->act_scale || !desc->down_scale ||
      !i8_matrix_ok(desc->w_act, desc->ld_act, desc->d) ||
      !i8_matrix_ok(desc->w_down, desc->ld_down, desc->d_ffn))
    return SFFN_ERR_INVALID;
  if (!aligned(x, type_size(x_dtype)) || !aligned(y, type_size(y_dtype)) || !aligned(idx, 4) ||
      !aligned(weights, 4) || !aligned(desc->act_scale, 4) || !aligned(desc->down_scale, 4) ||
      !aligned(desc->b_act, 4))
    return SFFN_ERR_INVALID;
  if (!work || !aligned(work, 256)) return SFFN_ERR_INVALID;
  const int chunk =
      sffn::host::experts_chunk(desc->experts, desc->d, desc->d_ffn, T, k, work_bytes);
  if (chunk < 1) return SFFN_ERR_INVALID;
  const int64_t xe = (int64_t)type_size(x_dtype), ye = (int64_t)type_size(y_dtype);
  const sffn::host::ChunkOrder order = sffn::host::chunk_order(
      sffn::host::Chunks(T, chunk), reinterpret_cast<uintptr_t>(x), ldx * xe, desc->d * xe,
      reinterpret_cast<uintptr_t>(y), ldy * ye, desc->d * ye);
  if (order == sffn::host::ChunkOrder::None) return SFFN_ERR_INVALID;
  sffn::ExpertsArgs a{};
  a.E = desc->experts;
  a.d = desc->d;
  a.f = desc->d_ffn;
  a.gated = desc->gated;
  a.w_act = desc->w_act;
  a.ld_act = desc->ld_act;
  a.act_scale = desc->act_scale;
  a.b_act = desc->b_act;
  a.w_down = desc->w_down;
  a.ld_down = desc->ld_down;
  a.down_scale = desc->down_scale;
  return status(sffn::run_experts(a, x, x_dtype, ldx, T, idx, weights, k, y, y_dtype, ldy, work,
                                  chunk, order == sffn::host::ChunkOrder::Backward,
                                  static_cast<hipStream_t>(stream)));
}

}  // extern "C"
