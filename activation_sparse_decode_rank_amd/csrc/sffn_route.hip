// Expert router (gfx950): scores of a token's experts, the best k of them, and their weights.
//
//   s_e = softmax or sigmoid of the logits, c_e = s_e + b_e (without a bias: the logit),
//   group worth = the best c_e or the sum of the two best, top groups, top k of c_e,
//   weights s_e (/ their sum) * scale
//
// One wave takes one token, expert e in lane e % 64 as its value e / 64. Scores are compared
// in 64 bits, so that the choice is that of the exact scores.
#include <algorithm>

#include "sffn_device.h"
#include "sffn_i8.h"

namespace sffn {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return (float)v;
}

constexpr int RWAVES = TPB / 64;

// J: experts per lane (E <= 64 J)
template <typename T, int J>
__global__ __launch_bounds__(TPB) void k_route(RouteArgs a) {
  __shared__ double s_c[RWAVES][64 * J];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * RWAVES + wave;
  if (t >= a.T) return;
  const double NINF = -__builtin_inf();
  const T* l = static_cast<const T*>(a.logits) + (size_t)t * a.ld;
  double v[J], c[J], sc[J];
  double m = NINF;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    double x = e < a.E ? (double)to_f32(l[e]) : NINF;
    v[j] = x == x ? x : NINF;  // NaN: off
    m = fmax(m, v[j]);
  }
  if (a.score == 0) {
    for (int o = 32; o; o >>= 1) m = fmax(m, __shfl_xor(m, o));
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      sc[j] = v[j] == NINF ? 0.0 : v[j] == m ? 1.0 : exp(v[j] - m);
      sum += sc[j];
    }
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    sum = fmax(sum, 1.0);
#pragma unroll
    for (int j = 0; j < J; ++j) sc[j] /= sum;
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) sc[j] = 1.0 / (1.0 + exp(-v[j]));
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    double x = v[j];
    if (a.bias && e < a.E) x = sc[j] + (double)a.bias[e];
    c[j] = v[j] > NINF && x == x ? x : NINF;
  }
  if (a.groups > 1) {
    const int per = a.E / a.groups;
#pragma unroll
    for (int j = 0; j < J; ++j)
      s_c[wave][lane + 64 * j] =
          a.group_top == 1 || a.bias ? c[j] : (v[j] > NINF ? sc[j] : NINF);
    wave_lds_sync();
    double worth = NINF;
    if (lane < a.groups) {
      double b1 = NINF, b2 = NINF;
      for (int i = 0; i < per; ++i) {
        const double x = s_c[wave][lane * per + i];
        if (x > b1) {
          b2 = b1;
          b1 = x;
        } else if (x > b2) {
          b2 = x;
        }
      }
      worth = b1;
      if (a.group_top == 2 && b2 > NINF) worth += b2;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(worth, g);
      rank += o > worth || (o == worth && g < lane) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 64 * j;
      if (e < a.E && !((kept >> (e / per)) & 1)) c[j] = NINF;
    }
  }
  // the score of a chosen expert is read back by its slot's lane
  wave_lds_sync();
#pragma unroll
  for (int j = 0; j < J; ++j) s_c[wave][lane + 64 * j] = sc[j];
  wave_lds_sync();
  int mine = -1;
  double w = 0.0;
  for (int s = 0; s < a.k; ++s) {
    double best = NINF;
    int at = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (c[j] > best) {
        best = c[j];
        at = lane + 64 * j;
      }
    for (int o = 32; o; o >>= 1) {
      const double ob = __shfl_xor(best, o);
      const int oa = __shfl_xor(at, o);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (best == NINF) break;
    if (lane == s) {
      mine = at;
      w = s_c[wave][at];
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (at == lane + 64 * j) c[j] = NINF;
  }
  if (a.renorm) {
    double sum = w;
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    a.idx[(size_t)t * a.k + lane] = mine;
    a.weights[(size_t)t * a.k + lane] = (float)(w * (double)a.scale);
  }
}

template <typename T>
void route_launch(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T + RWAVES - 1) / RWAVES)), block(TPB);
  if (a.E <= 64) k_route<T, 1><<<grid, block, 0, s>>>(a);
  else if (a.E <= 128) k_route<T, 2><<<grid, block, 0, s>>>(a);
  else if (a.E <= 256) k_route<T, 4><<<grid, block, 0, s>>>(a);
  else if (a.E <= 512) k_route<T, 8><<<grid, block, 0, s>>>(a);
  else k_route<T, 16><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
  if (dtype == T_F32) route_launch<float>(a, s);
  else if (dtype == T_F16) route_launch<_Float16>(a, s);
  else route_launch<__bf16>(a, s);
  return hipGetLastError();
}

}  // namespace sffn
