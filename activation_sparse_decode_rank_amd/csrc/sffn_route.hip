// Expert router (gfx950): scores of a token's experts, the best k of them, and their weights.
//
//   s_e = softmax or sigmoid of the logits, c_e = s_e + b_e (without a bias: the logit),
//   group worth = the best c_e or the sum of the two best, top groups, top k of c_e,
//   weights s_e (/ their sum) * scale
//
// One wave takes one token, expert e in lane e % 64 as its value e / 64; a choice is a maximum
// over the wave (DPP) and a ballot for its lowest index. Bound by those instructions: the logits
// are read once.
//
// Without a bias the logits themselves are compared, which is exact; only the chosen experts' (or,
// where the softmax is not renormalised, all) exponentials are taken. Scores that are compared are
// computed in 32 bits first, off by at most a known margin; where every comparison that decided
// was won by more than that, the choice is that of the exact scores, and otherwise the wave does
// the token again in 64 bits.
#include <algorithm>

#include "sffn_device.h"
#include "sffn_i8.h"

namespace sffn {
namespace {

constexpr int RWAVES = TPB / 64;

template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ float dpp_max(float v) {
  // lanes without a source keep their own value
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                                __builtin_bit_cast(int, v), __builtin_bit_cast(int, v),
                                                CTRL, ROW_MASK, 0xF, false)));
}
__device__ __forceinline__ float from_lane(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// largest over the wave, in every lane (one scalar)
__device__ __forceinline__ float wave_max(float v) {
  v = dpp_max<DPP_QP_XOR1>(v);
  v = dpp_max<DPP_QP_XOR2>(v);
  v = dpp_max<DPP_HALF_MIRROR>(v);
  v = dpp_max<DPP_MIRROR>(v);
  v = dpp_max<DPP_BCAST15, 0xA>(v);
  v = dpp_max<DPP_BCAST31, 0xC>(v);
  return from_lane(v, 63);
}
__device__ __forceinline__ float wave_total(float v) { return from_lane(wave_sum(v), WAVE_SUM_LANE); }

__device__ __forceinline__ double with_words(int lo, int hi) {
  return __builtin_bit_cast(double, ((uint64_t)(unsigned)hi << 32) | (unsigned)lo);
}
__device__ __forceinline__ int low(double v) { return (int)__builtin_bit_cast(uint64_t, v); }
__device__ __forceinline__ int high(double v) { return (int)(__builtin_bit_cast(uint64_t, v) >> 32); }
__device__ __forceinline__ double from_lane(double v, int lane) {
  return with_words(__builtin_amdgcn_readlane(low(v), lane), __builtin_amdgcn_readlane(high(v), lane));
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ double dpp_of(double v, double other) {
  return with_words(__builtin_amdgcn_update_dpp(low(other), low(v), CTRL, ROW_MASK, 0xF, false),
                    __builtin_amdgcn_update_dpp(high(other), high(v), CTRL, ROW_MASK, 0xF, false));
}
__device__ __forceinline__ double wave_max(double v) {
  v = fmax(v, dpp_of<DPP_QP_XOR1>(v, v));
  v = fmax(v, dpp_of<DPP_QP_XOR2>(v, v));
  v = fmax(v, dpp_of<DPP_HALF_MIRROR>(v, v));
  v = fmax(v, dpp_of<DPP_MIRROR>(v, v));
  v = fmax(v, dpp_of<DPP_BCAST15, 0xA>(v, v));
  v = fmax(v, dpp_of<DPP_BCAST31, 0xC>(v, v));
  return from_lane(v, 63);
}
__device__ __forceinline__ double wave_total(double v) {
  v += dpp_of<DPP_QP_XOR1>(v, 0.0);
  v += dpp_of<DPP_QP_XOR2>(v, 0.0);
  v += dpp_of<DPP_HALF_MIRROR>(v, 0.0);
  v += dpp_of<DPP_MIRROR>(v, 0.0);
  v += dpp_of<DPP_BCAST15, 0xA>(v, 0.0);
  v += dpp_of<DPP_BCAST31, 0xC>(v, 0.0);
  return from_lane(v, 63);
}

__device__ __forceinline__ float infinity(float) { return __builtin_inff(); }
__device__ __forceinline__ double infinity(double) { return __builtin_inf(); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float magnitude(float a) { return fabsf(a); }
__device__ __forceinline__ double magnitude(double a) { return fabs(a); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }

// The groups that stay, from the values x in s_v (minus infinity: none): a group's worth is its
// best one, or with `pairs` the sum of its two best. L lanes, a power of two of them, look through
// a group; bit g L of the result is group g. least, most: the least worth that stays, the most
// that does not (minus infinity: none). addends (if not null): the largest sum of the magnitudes
// that a group's worth is made of.
template <typename F>
__device__ __forceinline__ uint64_t groups_kept(const RouteArgs& a, const F* s_v, bool pairs, int L,
                                                F& least, F& most, F* addends) {
  const int lane = threadIdx.x & 63;
  const F NINF = -infinity(F());
  const int per = a.E / a.groups, g = lane / L;
  F b1 = NINF, b2 = NINF;
  if (g < a.groups)
    for (int i = lane % L; i < per; i += L) {
      const F x = s_v[g * per + i];
      b2 = larger(b2, smaller(b1, x));
      b1 = larger(b1, x);
    }
  for (int o = L / 2; o; o >>= 1) {
    const F o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
    b2 = larger(larger(b2, o2), smaller(b1, o1));
    b1 = larger(b1, o1);
  }
  const F more = pairs && b2 > NINF ? b2 : F(0);
  const F worth = b1 + more;
  if (addends) *addends = wave_max(b1 > NINF ? magnitude(b1) + magnitude(more) : F(0));
  int rank = 0;
  for (int q = 0; q < a.groups; ++q) {
    const F o = from_lane(worth, q * L);
    rank += o > worth || (o == worth && q < g) ? 1 : 0;
  }
  const bool in = g < a.groups && rank < a.top_groups;
  least = -wave_max(in ? -worth : NINF);
  most = wave_max(g < a.groups && !in ? worth : NINF);
  return __ballot(in);
}

// whether expert e's group stays
__device__ __forceinline__ bool stays(const RouteArgs& a, uint64_t kept, int L, int e) {
  // (e + 1/2) / per is at least 1 / (2 per) away from a whole number: rounding cannot cross it
  const int g = (int)(((float)e + 0.5f) * ((float)a.groups / (float)a.E));
  return e < a.E && ((kept >> (g * L)) & 1);
}

// Lane and value j of the lowest index that has `best`
template <int J, typename F>
__device__ __forceinline__ void lowest(const F (&c)[J], F best, int& lane, int& jat) {
  uint64_t has = 0;
  jat = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (has == 0) {
      has = __ballot(c[j] == best);
      jat = j;
    }
  }
  lane = __builtin_ctzll(has);
}

// The token's slots in lanes 0 .. k - 1: index (-1: none) and score
struct Chosen {
  int idx;
  double w;
};

// The token in 64 bits. v: its logits (minus infinity: off); m: the largest of them.
template <int J>
__device__ Chosen route_exact(const RouteArgs& a, const float (&v)[J], float m, double* s_c, int L) {
  const int lane = threadIdx.x & 63;
  const double NINF = -__builtin_inf();
  double c[J], sc[J];
  if (a.score == 0) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      sc[j] = v[j] == -__builtin_inff() ? 0.0 : v[j] == m ? 1.0 : exp((double)v[j] - (double)m);
      sum += sc[j];
    }
    sum = fmax(wave_total(sum), 1.0);
#pragma unroll
    for (int j = 0; j < J; ++j) sc[j] /= sum;
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) sc[j] = 1.0 / (1.0 + exp(-(double)v[j]));
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    double x = (double)v[j];
    if (a.bias && e < a.E) x = sc[j] + (double)a.bias[e];
    c[j] = v[j] > -__builtin_inff() && x == x ? x : NINF;
  }
  if (a.groups > 1) {
    const bool pairs = a.group_top == 2;
    wave_lds_sync();
#pragma unroll
    for (int j = 0; j < J; ++j)
      s_c[lane + 64 * j] = !pairs || a.bias ? c[j] : (c[j] > NINF ? sc[j] : NINF);
    wave_lds_sync();
    double least, most;
    const uint64_t kept = groups_kept(a, s_c, pairs, L, least, most, static_cast<double*>(nullptr));
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (!stays(a, kept, L, lane + 64 * j)) c[j] = NINF;
  }
  Chosen r{-1, 0.0};
  for (int s = 0; s < a.k; ++s) {
    double best = c[0];
#pragma unroll
    for (int j = 1; j < J; ++j) best = fmax(best, c[j]);
    best = wave_max(best);
    if (best == NINF) break;
    int at, jat;
    lowest<J>(c, best, at, jat);
    double x = sc[0];
#pragma unroll
    for (int j = 1; j < J; ++j) x = jat == j ? sc[j] : x;
    x = from_lane(x, at);
    if (lane == s) {
      r.idx = at + 64 * jat;
      r.w = x;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (jat == j && lane == at) c[j] = NINF;
  }
  return r;
}

// Margins of 32-bit scores, twice what one is off. A sigmoid: its exponential, the sum and the
// quotient lose 2^-24 of it each, at most two for the exponential; a bias' sum 2^-24 of 1 + its
// magnitude: 6 2^-24 in all (a worth of two: twice that, and 2^-24 of what is added). A softmax:
// the argument down to -104 (below, it is zero) makes its exponential off by up to 104 2^-24, but
// only where it is small: x e^-x is at most 0.37, so 2^-24 of the largest score and those above
// with the longer sum: 16 2^-24; relative to itself, where scores are compared without a bias,
// 128 2^-24. That holds for normal numbers only: below 2^-126 a score is off by up to 2^-149, and
// a sigmoid whose exponential overflows (logits below -88.7) by all of itself, less than 2^-126.
// Neither counts beside a worth of at least SMALLEST_WORTH, of which the margin is 2^-116; smaller
// ones are compared in 64 bits.
constexpr float MARGIN_SIGMOID = 0x1p-20f, MARGIN_SOFTMAX = 0x1p-19f;  // of 1 + the larger magnitude
constexpr float MARGIN_ITSELF = 0x1p-16f;                              // of the larger one
constexpr float SMALLEST_WORTH = 0x1p-100f;
// From here down e^-l passes the largest 64-bit number, and the score is zero in 64 bits.
constexpr float ZERO_SIGMOID = -709.7827f;

// J: experts per lane (E <= 64 J); BIAS: c = s + b
template <typename T, int J, bool BIAS>
__global__ __launch_bounds__(TPB) void k_route(RouteArgs a) {
  __shared__ double s_c[RWAVES][64 * J];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * RWAVES + wave;
  if (t >= a.T) return;
  const float NINF = -__builtin_inff();
  const T* l = static_cast<const T*>(a.logits) + (size_t)t * a.ld;
  float v[J], c[J], sc[J], b[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j;
    const float x = e < a.E ? (float)l[e] : NINF;
    b[j] = BIAS && e < a.E ? a.bias[e] : 0.f;
    v[j] = x == x ? x : NINF;  // NaN: off
  }
  float m = v[0];
#pragma unroll
  for (int j = 1; j < J; ++j) m = fmaxf(m, v[j]);
  m = wave_max(m);
  const bool soft = a.score == 0;
  const bool pairs = a.groups > 1 && a.group_top == 2;
  // all scores, where they are compared or their sum counts
  float total = 1.f;
  if (BIAS || pairs || (soft && !a.renorm)) {
    if (soft) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        sc[j] = v[j] == NINF ? 0.f : v[j] == m ? 1.f : expf(v[j] - m);
        sum += sc[j];
      }
      total = fmaxf(wave_total(sum), 1.f);
      if (BIAS || pairs) {
#pragma unroll
        for (int j = 0; j < J; ++j) sc[j] = sc[j] / total;
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) sc[j] = 1.f / (1.f + expf(-v[j]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) sc[j] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float x = BIAS ? sc[j] + b[j] : v[j];
    c[j] = v[j] > NINF && x == x ? x : NINF;
  }
  bool sure = true;
  const float margin = soft ? MARGIN_SOFTMAX : MARGIN_SIGMOID;
  const int L = a.groups > 1 ? 1 << (31 - __builtin_clz(64 / a.groups)) : 64;
  if (a.groups > 1) {
    float* s_v = reinterpret_cast<float*>(s_c[wave]);
#pragma unroll
    for (int j = 0; j < J; ++j)
      s_v[lane + 64 * j] = BIAS || !pairs ? c[j] : (v[j] > NINF ? sc[j] : NINF);
    wave_lds_sync();
    float least, most, addends;
    const uint64_t kept = groups_kept(a, s_v, pairs, L, least, most, BIAS ? &addends : nullptr);
    // two scores a side, which may cancel: the margin goes by what was added, not by the sums
    // (an infinity there: a bias, or a sum that 32 bits cannot hold)
    if (BIAS)
      sure = addends < __builtin_inff() && (most == NINF || least - most > 2.f * margin * (1.f + addends));
    else if (pairs) sure = most == NINF || (least > SMALLEST_WORTH && least - most > MARGIN_ITSELF * least);
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (!stays(a, kept, L, lane + 64 * j)) c[j] = NINF;
  }
  int mine = -1;
  float won = 0.f;  // its logit, or with a bias its score
  float before = __builtin_inff();
  // with a bias one more than k: the last choice must be clear of the best one left out
  const int rounds = BIAS ? a.k + 1 : a.k;
  for (int s = 0; s < rounds; ++s) {
    float best = c[0];
#pragma unroll
    for (int j = 1; j < J; ++j) best = fmaxf(best, c[j]);
    best = wave_max(best);
    if (best == NINF) break;
    if (BIAS) {
      if (s > 0 && !(before - best > margin * (1.f + fabsf(best)))) sure = false;
      before = best;
      if (!sure || s == a.k) break;
    }
    int at, jat;
    lowest<J>(c, best, at, jat);
    float val = best;
    if (BIAS) {
      float x = sc[0];
#pragma unroll
      for (int j = 1; j < J; ++j) x = jat == j ? sc[j] : x;
      val = from_lane(x, at);
    }
    if (lane == s) {
      mine = at + 64 * jat;
      won = val;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (jat == j && lane == at) c[j] = NINF;
  }
  float w = won, sum = 1.f;
  if (!BIAS) w = !soft ? 1.f / (1.f + expf(-won)) : won == m ? 1.f : expf(won - m);
  if (!BIAS && soft && !a.renorm) w = w / total;
  if (mine < 0) w = 0.f;
  if (a.renorm) {
    sum = wave_total(w);
    // scores that 32 bits do not hold beside each other: their quotients may still count
    if (sum < 1.f && -wave_max(mine >= 0 ? -w : NINF) < 0x1p-100f) sure = false;
  }
  if (sure) {
    if (a.renorm) w = sum > 0.f ? w / sum : 0.f;
    w *= a.scale;
  } else {
    const Chosen r = route_exact<J>(a, v, m, s_c[wave], L);
    mine = r.idx;
    double x = r.w;
    if (a.renorm) {
      const double all = wave_total(x);
      x = all > 0.0 ? x / all : 0.0;
    }
    w = (float)(x * (double)a.scale);
  }
  if (lane < a.k) {
    a.idx[(size_t)t * a.k + lane] = mine;
    a.weights[(size_t)t * a.k + lane] = mine < 0 ? 0.f : w;  // also where scale is not finite
  }
}

// The plain choice (no bias, no groups), two tokens a wave: a token has 32 lanes, expert e in lane
// e % 32 as its value e / 32, and one step of the maximum serves both. Up to 256 experts and 32
// slots (30011 tokens of 160 experts, 6 slots: 17 us; 22 us with a wave a token).
template <typename T, int J>
__global__ __launch_bounds__(TPB) void k_route_pair(RouteArgs a) {
  const int lane = threadIdx.x & 63, l32 = lane & 31;
  const bool second = lane >= 32;
  const int64_t t = ((int64_t)blockIdx.x * RWAVES + (threadIdx.x >> 6)) * 2 + (second ? 1 : 0);
  const float NINF = -__builtin_inff();
  const T* l = static_cast<const T*>(a.logits) + (size_t)(t < a.T ? t : 0) * a.ld;
  float v[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = l32 + 32 * j;
    const float x = t < a.T && e < a.E ? (float)l[e] : NINF;
    v[j] = x == x ? x : NINF;  // NaN: off
  }
  // each token's largest and total, in its lanes
  auto most = [&](float x) {
    x = dpp_max<DPP_QP_XOR1>(x);
    x = dpp_max<DPP_QP_XOR2>(x);
    x = dpp_max<DPP_HALF_MIRROR>(x);
    x = dpp_max<DPP_MIRROR>(x);
    x = dpp_max<DPP_BCAST15, 0xA>(x);
    return second ? from_lane(x, 63) : from_lane(x, 31);
  };
  auto total = [&](float x) {
    x = dpp_add<DPP_QP_XOR1>(x);
    x = dpp_add<DPP_QP_XOR2>(x);
    x = dpp_add<DPP_HALF_MIRROR>(x);
    x = dpp_add<DPP_MIRROR>(x);
    x = dpp_add<DPP_BCAST15, 0xA>(x);
    return second ? from_lane(x, 63) : from_lane(x, 31);
  };
  const bool soft = a.score == 0;
  int mine = -1;
  float won = NINF, m = NINF, sum = 1.f;
  for (int s = 0; s < a.k; ++s) {
    float best = v[0];
#pragma unroll
    for (int j = 1; j < J; ++j) best = fmaxf(best, v[j]);
    best = most(best);
    if (s == 0) {
      m = best;
      if (soft && !a.renorm) {
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) x += v[j] == NINF ? 0.f : v[j] == m ? 1.f : expf(v[j] - m);
        sum = fmaxf(total(x), 1.f);
      }
    }
    if (__ballot(best > NINF) == 0) break;
    // the lowest index that has it: lowest value, then lowest lane
    unsigned has0 = 0, has1 = 0;
    int j0 = 0, j1 = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint64_t eq = __ballot(v[j] == best);
      if (has0 == 0) {
        has0 = (unsigned)eq;
        j0 = j;
      }
      if (has1 == 0) {
        has1 = (unsigned)(eq >> 32);
        j1 = j;
      }
    }
    const int at = second ? __builtin_ctz(has1) : __builtin_ctz(has0), jat = second ? j1 : j0;
    if (l32 == s && best > NINF) {
      mine = at + 32 * jat;
      won = best;
    }
    const int gone = l32 == at ? jat : -1;
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = gone == j ? NINF : v[j];
  }
  float w;
  if (soft) {
    w = won == m ? 1.f : expf(won - m);
    if (!a.renorm) w = w / sum;
  } else {
    // sigmoids that are divided by their sum: those of low logits together times e^-m, which keeps
    // them in range
    const float low = a.renorm && m < 0.f ? m : 0.f;
    w = won < 0.f ? expf(won - low) / (1.f + expf(won)) : expf(-low) / (1.f + expf(-won));
    if (won <= ZERO_SIGMOID) w = 0.f;
  }
  if (mine < 0) w = 0.f;
  if (a.renorm) {
    const float all = total(w);
    w = all > 0.f ? w / all : 0.f;
  }
  if (l32 < a.k && t < a.T) {
    a.idx[(size_t)t * a.k + l32] = mine;
    a.weights[(size_t)t * a.k + l32] = mine < 0 ? 0.f : w * a.scale;
  }
}

template <typename T, int J>
void route_launch(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)a.T + RWAVES - 1) / RWAVES)), block(TPB);
  if (a.bias) k_route<T, J, true><<<grid, block, 0, s>>>(a);
  else k_route<T, J, false><<<grid, block, 0, s>>>(a);
}

template <typename T, int J>
void pair_launch(const RouteArgs& a, hipStream_t s) {
  k_route_pair<T, J><<<dim3((unsigned)(((int64_t)a.T + 2 * RWAVES - 1) / (2 * RWAVES))), dim3(TPB), 0, s>>>(a);
}

template <typename T>
void route_launch(const RouteArgs& a, hipStream_t s) {
  // few tokens leave lanes to spare (1 token of 64 experts: 2.8 us with a wave a token, 3.4 here)
  if (!a.bias && a.groups == 1 && a.E <= 256 && a.k <= 32 && a.T >= 2048) {
    if (a.E <= 64) pair_launch<T, 2>(a, s);
    else if (a.E <= 128) pair_launch<T, 4>(a, s);
    else if (a.E <= 160) pair_launch<T, 5>(a, s);
    else pair_launch<T, 8>(a, s);
    return;
  }
  if (a.E <= 64) route_launch<T, 1>(a, s);
  else if (a.E <= 128) route_launch<T, 2>(a, s);
  else if (a.E <= 192) route_launch<T, 3>(a, s);
  else if (a.E <= 256) route_launch<T, 4>(a, s);
  else if (a.E <= 512) route_launch<T, 8>(a, s);
  else route_launch<T, 16>(a, s);
}

}  // namespace

// In pieces: a launch holds less than 2^32 threads, and a token takes up to 64.
hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t s) {
  constexpr int PIECE = 1 << 25;
  for (int64_t t0 = 0; t0 < a.T; t0 += PIECE) {
    RouteArgs p = a;
    p.T = (int)std::min<int64_t>(PIECE, a.T - t0);
    p.logits = static_cast<const char*>(a.logits) + (size_t)t0 * a.ld * (dtype == T_F32 ? 4 : 2);
    p.idx = a.idx + (size_t)t0 * a.k;
    p.weights = a.weights + (size_t)t0 * a.k;
    if (dtype == T_F32) route_launch<float>(p, s);
    else if (dtype == T_F16) route_launch<_Float16>(p, s);
    else route_launch<__bf16>(p, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sffn
