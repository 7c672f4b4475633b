// Routing of tokens to experts for any score, bias, groups and top-k, and the
// gradient of its weights.
//
//   s_e = softmax(l)_e or 1 / (1 + e^-l_e),  c_e = s_e + b_e
//   the top_groups groups with the highest sums of their best c stay, the k
//   highest c of those are chosen, w_j = scale s_ej (/ sum_j s_ej)
#include "ops.h"

#include <float.h>

#include <algorithm>

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxRouteExperts = 256, kMaxK = 8, kMaxGroups = 16;
constexpr uint32_t kManyTokens = 16384;  // fewer lanes a token from here on

struct RouteArgs {
  const float* logits;
  const float* bias;
  const uint8_t* valid;
  int32_t* experts;
  float* weights;
  const float* dweights;
  const float* add;
  float* dlogits;
  uint32_t tokens, E, k;
  uint32_t groups, top_groups, group_best;
  uint32_t by_group;  // 1: some groups are left out
  uint32_t renorm;
  float scale;
  uint32_t names;      // the low bits of a key that name its expert: at least E - 1
  float cut;           // what the others are relatively off by, at most
  uint32_t per_group;  // 2^16 / experts of a group, rounded up
};

// A logit as it is used: +infinity is the largest finite value, NaN is none.
__device__ __forceinline__ float usable(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

// Weights of the chosen logits: lane j of each aligned group of 8 lanes holds
// the j-th (-infinity: no expert). u_j = s_j e^-m with m = min(0, the largest
// logit) keeps the ratios of scores that underflow.
template <bool kSigmoid>
__device__ __forceinline__ float chosen_score(float l, bool renorm) {
  float m = lanes_max<8>(l);
  if (m == -INFINITY) return 0.0f;
  if constexpr (kSigmoid) {
    m = renorm ? fminf(m, 0.0f) : 0.0f;
    return expf(fminf(l, 0.0f) - m) / (1.0f + expf(-fabsf(l)));
  }
  return expf(l - m);
}

// ---- the choice -------------------------------------------------------------------
//
// L lanes a token, C times four neighbouring experts a lane. The choice is that
// of 64-bit scores, but few tokens need them: the values that order the experts
// (logits where nothing is added to their scores and no group is marked, else
// c in fp32) are cut to the bits that leave room for the expert's number, so
// that one 32-bit integer orders and names an expert, and the k + 2 best are
// found with integer maxima. Where two of them are so close that the cut or
// the fp32 evaluation might have changed their order, the k + 1 best are
// compared in 64 bits (`settle`), and where even the (k + 2)-th might belong to
// the k best, or two groups' marks are that close, all of the token's scores are
// computed in 64 bits (`choose_slowly`).

// Order-preserving integers of floats.
__device__ __forceinline__ int32_t ordered(float f) {
  const int32_t b = __builtin_bit_cast(int32_t, f + 0.0f);  // no negative zero
  return b ^ (b >> 31 & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int32_t i) { return __builtin_bit_cast(float, i ^ (i >> 31 & 0x7fffffff)); }
constexpr int32_t kNone = INT32_MIN;  // below every value's

template <int M>
__device__ __forceinline__ int32_t across_int(int32_t v) {
  return __builtin_bit_cast(int32_t, across<M>(__builtin_bit_cast(float, v)));
}
template <int L, int M = 1>
__device__ __forceinline__ int32_t lanes_max_int(int32_t v) {
  if constexpr (M < L) return lanes_max_int<L, 2 * M>(max(v, across_int<M>(v)));
  return v;
}
template <int L, int M = 1>
__device__ __forceinline__ uint32_t lanes_or(uint32_t v) {
  if constexpr (M < L) return lanes_or<L, 2 * M>(v | (uint32_t)across_int<M>((int32_t)v));
  return v;
}

// Score of a logit in 64 bits: l - top's exponential over `total`, or the sigmoid.
template <bool kSigmoid>
__device__ __forceinline__ double score64(float l, float top, double total) {
  if constexpr (kSigmoid) return 1.0 / (1.0 + exp(-(double)l));
  return exp((double)l - (double)top) / total;
}

// What a token's lanes know of it. at(i): the first of the four experts of the
// lane's i-th chunk; elements before 4 chunk(i) are the chunk's before.
template <int L, int C>
struct Token {
  const float* in;
  float l[4 * C];
  uint32_t E, sub;
  __device__ __forceinline__ uint32_t expert(int i, int v) const {
    const uint32_t c = 4 * (i * L + sub);
    return min(c, max(E, 4u) - 4) + v;
  }
  // E >= 4: rows of any count in 16-byte loads, the last chunk moved back
  __device__ __forceinline__ void load(bool live) {
    typedef float At __attribute__((ext_vector_type(4), aligned(4)));
    typedef float Vec __attribute__((ext_vector_type(4)));
    Vec x[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (E >= 4) {
        x[i] = *reinterpret_cast<const At*>(in + expert(i, 0));
      } else {
#pragma unroll
        for (uint32_t v = 0; v < 4; ++v) x[i][v] = in[min(v, E - 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t e = expert(i, v);
        l[4 * i + v] = live && e < E && e >= 4 * (i * L + sub) ? usable(x[i][v]) : -INFINITY;
      }
  }
};

// Softmax statistics in 64 bits.
template <int L, int C>
__device__ __forceinline__ double total64(const Token<L, C>& t, float top) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < 4 * C; ++i) sum += t.l[i] == -INFINITY ? 0.0 : exp((double)t.l[i] - (double)top);
#pragma unroll
  for (int m = 1; m < L; m *= 2) sum += __shfl_xor(sum, m);
  return sum;
}

// The kept groups as bits from the marks in s_c, the row's c (missing: -infinity);
// *close: a kept and a left one differ by `margin` of the larger or less.
template <int L, typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, const F* c, uint32_t sub, F margin, bool* close) {
  constexpr int kEach = L >= (int)kMaxGroups ? 1 : (int)kMaxGroups / L;  // groups of a lane
  const uint32_t size = a.E / a.groups;
  const F low = -(F)INFINITY;
  F mark[kEach];
#pragma unroll
  for (int h = 0; h < kEach; ++h) {
    const uint32_t g = h * L + sub;
    F m1 = low, m2 = low;
    if (g < a.groups) {
      for (uint32_t i = 0; i < size; ++i) {
        const F x = c[g * size + i];
        m2 = max(m2, min(m1, x));
        m1 = max(m1, x);
      }
    }
    mark[h] = a.group_best == 2 && m2 > low ? m1 + m2 : m1;
  }
  uint32_t better[kEach] = {}, kept = 0;
  const int base = (int)(threadIdx.x & 63) / L * L;
  for (uint32_t g = 0; g < a.groups; ++g) {
    F m = mark[0];
#pragma unroll
    for (int h = 1; h < kEach; ++h)
      if (g / L == (uint32_t)h) m = mark[h];
    m = __shfl(m, base + (int)(g % L));
#pragma unroll
    for (int h = 0; h < kEach; ++h) better[h] += m > mark[h] || (m == mark[h] && g < h * L + sub);
  }
  F least = (F)INFINITY, most = low;  // of the kept, of the left
#pragma unroll
  for (int h = 0; h < kEach; ++h) {
    const uint32_t g = h * L + sub;
    const bool keep = g < a.groups && better[h] < a.top_groups;
    kept |= keep ? 1u << g : 0u;
    if (keep) least = min(least, mark[h]);
    else if (g < a.groups) most = max(most, mark[h]);
  }
  kept = lanes_or<L>(kept);
#pragma unroll
  for (int m = 1; m < L; m *= 2) {
    least = min(least, (F)__shfl_xor(least, m));
    most = max(most, (F)__shfl_xor(most, m));
  }
  *close = most > low && !(least - most > margin * (1 + max(fabs(least), fabs(most))));
  return kept;
}

// Lane q of the first eight of a token's (or of its four) has the q-th expert, with
// four lanes a token also the (q + 4)-th.
template <int L>
struct Places {
  static constexpr int kLanes = L < 8 ? L : 8, kEach = 8 / kLanes;
  int32_t id[kEach];  // E: none
};

// The k best by 64-bit values, everything computed anew.
template <int L, int C, bool kSigmoid>
__device__ __forceinline__ void choose_slowly(const RouteArgs& a, const Token<L, C>& t, bool scored, double* s_c, Places<L>& to) {
  typedef Places<L> P;
  double c[4 * C];
  float top = t.l[0];
#pragma unroll
  for (int i = 1; i < 4 * C; ++i) top = fmaxf(top, t.l[i]);
  top = lanes_max<L>(top);
  const double total = kSigmoid || !scored ? 1.0 : total64<L, C>(t, top);
#pragma unroll
  for (int i = 0; i < 4 * C; ++i) {
    c[i] = -(double)INFINITY;
    if (t.l[i] != -INFINITY) {
      c[i] = scored ? score64<kSigmoid>(t.l[i], top, total) : (double)t.l[i];
      if (a.bias) c[i] += (double)a.bias[t.expert(i / 4, i % 4)];
      if (!(c[i] > -(double)INFINITY)) c[i] = -(double)INFINITY;
    }
  }
  if (a.by_group) {
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) {
      const uint32_t e = t.expert(i / 4, i % 4);
      if (e < a.E && e >= 4 * (i / 4 * L + t.sub)) s_c[e] = c[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    bool close;
    const uint32_t kept = keep_groups<L, double>(a, s_c, t.sub, 0.0, &close), size = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < 4 * C; ++i)
      if (!(kept >> min(t.expert(i / 4, i % 4) / size, 31u) & 1)) c[i] = -(double)INFINITY;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
#pragma unroll 1
  for (int j = 0; j < (int)a.k; ++j) {
    double best = -(double)INFINITY;
    int32_t at = (int32_t)a.E;
#pragma unroll
    for (int i = 0; i < 4 * C; ++i)
      if (c[i] > best) best = c[i], at = (int32_t)t.expert(i / 4, i % 4);
#pragma unroll
    for (int m = 1; m < L; m *= 2) {
      const double o = __shfl_xor(best, m);
      const int32_t n = __shfl_xor(at, m);
      if (o > best || (o == best && n < at)) best = o, at = n;
    }
#pragma unroll
    for (int h = 0; h < P::kEach; ++h)
      if (h * P::kLanes + (int)t.sub % P::kLanes == j) to.id[h] = at;
#pragma unroll
    for (int i = 0; i < 4 * C; ++i)
      if ((int32_t)t.expert(i / 4, i % 4) == at) c[i] = -(double)INFINITY;
  }
}

// Puts the N candidates of keys[] (of a sigmoid, or plain logits) in the order of
// their 64-bit values.
template <int L, int C, bool kSigmoid, int N>
__device__ __forceinline__ void settle(const RouteArgs& a, const Token<L, C>& t, bool scored, uint32_t names, int32_t (&keys)[N]) {
  constexpr int kEach = (N + L - 1) / L;
  double c[kEach];
  int32_t key[kEach];
  uint32_t before[kEach] = {};
#pragma unroll
  for (int h = 0; h < kEach; ++h) {
    key[h] = kNone;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (h * L + (int)t.sub == j) key[h] = keys[j];
    c[h] = -(double)INFINITY;
    if (key[h] != kNone) {
      const uint32_t e = names - ((uint32_t)key[h] & names);
      const float l = usable(t.in[e]);
      c[h] = scored ? score64<kSigmoid>(l, 0.0f, 1.0) : (double)l;
      if (a.bias) c[h] += (double)a.bias[e];
    }
  }
  const int base = (int)(threadIdx.x & 63) / L * L;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const double o = __shfl(c[j / L], base + j % L);
    const int32_t other = __shfl(key[j / L], base + j % L);
    if (other == kNone) continue;
#pragma unroll
    for (int h = 0; h < kEach; ++h)  // equal values: the larger name bits are the lower index
      before[h] += o > c[h] || (o == c[h] && (other & names) > (key[h] & names));
  }
  int32_t to[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    int32_t mine = 0;
#pragma unroll
    for (int h = 0; h < kEach; ++h)
      if (key[h] != kNone && before[h] == (uint32_t)j) mine = key[h];
    to[j] = (int32_t)lanes_or<L>((uint32_t)mine);
    if (keys[j] == kNone) to[j] = kNone;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) keys[j] = to[j];
}

// K: the largest top_k of this instance.
template <int L, int C, int K, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a) {
  constexpr int kRows = kThreads / L, N = K + 2, kList = N < 4 * C ? N : 4 * C;
  // Two fp32 values of c are off by less than this, and their roundings by less than
  // a.cut of themselves. Sigmoid: the exponent is off by 1.5 x 2^-24 of itself, e^x by 2^-23, the
  // sum and the reciprocal by 2^-23 each, and s (1 - s) |l| is at most 0.224: 4.3 x 2^-23 of c
  // each. Softmax: (D + 4) 2^-24 of e^-D, 30 x 2^-24 of the sum and the quotient: 31 x 2^-24 each.
  constexpr float kOff = kSigmoid ? 0x1p-19f : 0x1p-17f;
  extern __shared__ __attribute__((aligned(16))) double s_row[];  // [rows][E] by group: c, in 32 or 64 bits
  Token<L, C> t;
  t.E = a.E;
  t.sub = threadIdx.x % L;
  const uint32_t row = threadIdx.x / L, names = a.names;
  const bool scored = a.bias || a.by_group;
  double* s_c = s_row + row * a.E;
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows; t0 < a.tokens; t0 += (uint64_t)gridDim.x * kRows) {
    const uint64_t at = min(t0 + row, (uint64_t)a.tokens - 1);
    const bool live = !a.valid || a.valid[at];
    t.in = a.logits + at * a.E;
    t.load(live);
    // what orders the experts
    float c[4 * C];
    float top = -INFINITY, total = 1.0f;
    if constexpr (!kSigmoid) {
      if (scored || !a.renorm) {
#pragma unroll
        for (int i = 0; i < 4 * C; ++i) top = fmaxf(top, t.l[i]);
        top = lanes_max<L>(top);
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * C; ++i) {
          c[i] = t.l[i] == -INFINITY ? 0.0f : expf(t.l[i] - top);
          total += c[i];
        }
        total = lanes_sum<L>(total);
      }
    }
    if (scored) {
      const float inv = 1.0f / total;
#pragma unroll
      for (int i = 0; i < 4 * C; ++i) {
        if constexpr (kSigmoid) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t.l[i] * -1.44269504f));
        else c[i] *= inv;
        if (a.bias) c[i] += a.bias[min(t.expert(i / 4, i % 4), a.E - 1)];
        if (t.l[i] == -INFINITY || !(c[i] > -INFINITY)) c[i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * C; ++i) c[i] = t.l[i];
    }
    bool slow = false;
    if (a.by_group) {
      float* s = reinterpret_cast<float*>(s_c);
#pragma unroll
      for (int i = 0; i < 4 * C; ++i) {
        const uint32_t e = t.expert(i / 4, i % 4);
        if (e < a.E && e >= 4 * (i / 4 * L + t.sub)) s[e] = c[i];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const uint32_t kept = keep_groups<L, float>(a, s, t.sub, 2 * kOff, &slow);
#pragma unroll
      for (int i = 0; i < 4 * C; ++i) {
        const uint32_t e = min(t.expert(i / 4, i % 4), a.E - 1);
        if (!(kept >> (e * a.per_group >> 16) & 1)) c[i] = -INFINITY;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the lane's best, in order: each new one moves the lesser ones down
    int32_t list[kList];
#pragma unroll
    for (int n = 0; n < kList; ++n) list[n] = kNone;
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) {
      const uint32_t e = t.expert(i / 4, i % 4);
      const int32_t x = c[i] == -INFINITY ? kNone : (int32_t)(((uint32_t)ordered(c[i]) & ~names) | (names - e));
#pragma unroll
      for (int n = kList - 1; n > 0; --n) list[n] = max(min(list[n - 1], x), list[n]);
      list[0] = max(list[0], x);
    }
    // the token's best
    int32_t keys[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t best = lanes_max_int<L>(list[0]);
      keys[j] = best;
      const bool pop = list[0] == best;
#pragma unroll
      for (int n = 0; n + 1 < kList; ++n) list[n] = pop ? list[n + 1] : list[n];
      if (pop) list[kList - 1] = kNone;
    }
    // are they in order?
    const uint32_t k = a.k;
    bool close = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      // (j, j + 1) inside the k + 1 best; the (k + 2)-th against the k-th
      const int i = j + 1 < N ? j + 1 : j;
      const int32_t x = keys[j] & (int32_t)~names, y = keys[i] & (int32_t)~names;
      const float u = unordered(x), v = unordered(y);
      const float margin = (fabsf(u) + fabsf(v)) * a.cut + kOff;
      const bool near = scored ? !(u - v > margin) : x == y;
      if ((uint32_t)j < k && i > j && keys[i] != kNone) close |= near;
    }
#pragma unroll
    for (int j = 0; j + 2 < N; ++j) {
      const int32_t x = keys[j] & (int32_t)~names, y = keys[j + 2] & (int32_t)~names;
      const float u = unordered(x), v = unordered(y);
      const float margin = (fabsf(u) + fabsf(v)) * a.cut + kOff;
      const bool near = scored ? !(u - v > margin) : x == y;
      if ((uint32_t)j + 1 == k && keys[j + 2] != kNone) slow |= near;
    }
    slow |= close && scored && !kSigmoid;  // a softmax needs all of its logits
    if (close && !slow) {
      // the (k + 2)-th stays where it is
#pragma unroll
      for (int j = 0; j < N; ++j)
        if ((uint32_t)j > k) keys[j] = kNone;
      settle<L, C, kSigmoid, N>(a, t, scored, names, keys);
    }
    typedef Places<L> P;
    constexpr int kLanes = P::kLanes, kEach = P::kEach;
    P place;
    int32_t(&id)[kEach] = place.id;
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      id[h] = (int32_t)a.E;
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (h * kLanes + (int)t.sub % kLanes == j && (uint32_t)j < k && keys[j] != kNone)
          id[h] = (int32_t)(names - ((uint32_t)keys[j] & names));
    }
    if (slow) choose_slowly<L, C, kSigmoid>(a, t, scored, s_c, place);
    // the weights
    float l[kEach], u[kEach], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int h = 0; h < kEach; ++h) l[h] = t.in[min((uint32_t)id[h], a.E - 1)];
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      l[h] = id[h] < (int32_t)a.E ? usable(l[h]) : -INFINITY;
      m = fmaxf(m, l[h]);
    }
    m = lanes_max<kLanes>(m);
    if constexpr (kSigmoid) m = a.renorm ? fminf(m, 0.0f) : 0.0f;
    else m = a.renorm ? m : top;
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      u[h] = 0.0f;
      if (l[h] != -INFINITY) {
        // s e^-m with m = min(0, the largest logit) keeps the ratios of scores that underflow
        if constexpr (kSigmoid) u[h] = expf(fminf(l[h], 0.0f) - m) / (1.0f + expf(-fabsf(l[h])));
        else u[h] = expf(l[h] - m);
      }
      sum += u[h];
    }
    sum = lanes_sum<kLanes>(sum);
    const float by = a.renorm ? sum : total;
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      const uint32_t j = h * kLanes + t.sub;
      if (t0 + row < a.tokens && t.sub < (uint32_t)kLanes && j < k) {
        a.experts[at * k + j] = id[h];
        a.weights[at * k + j] = id[h] < (int32_t)a.E ? a.scale * (u[h] / by) : 0.0f;
      }
    }
  }
}

template <int L, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void k_route_grad(RouteArgs a) {
  constexpr int kRows = kThreads / L;
  const int sub = threadIdx.x % L, row = threadIdx.x / L;
  const int base = (threadIdx.x & 63) / L * L;
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows; t0 < a.tokens; t0 += (uint64_t)gridDim.x * kRows) {
    const uint64_t t = t0 + row;
    const bool live = t < a.tokens && (!a.valid || a.valid[t]);
    const float* in = a.logits + (t < a.tokens ? t : 0) * a.E;
    int id = -1;
    float g = 0.0f, l = -INFINITY;
    if (live && (uint32_t)sub < a.k) {
      id = a.experts[t * a.k + sub];
      if ((uint32_t)id < a.E) {
        l = usable(in[id]);
        g = a.dweights[t * a.k + sub] * a.scale;
      }
    }
    float u = chosen_score<kSigmoid>(l, a.renorm), d[4] = {0, 0, 0, 0};
    if (!kSigmoid && !a.renorm) {  // the softmax over all experts
      float x[4], top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t e = 4 * sub + v;
        x[v] = live && e < a.E ? usable(in[e]) : -INFINITY;
        top = fmaxf(top, x[v]);
      }
      top = lanes_max<L>(top);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x[v] = x[v] == -INFINITY ? 0.0f : expf(x[v] - top);
        sum += x[v];
      }
      sum = lanes_sum<L>(sum);
      const float inv = sum > 0 ? 1.0f / sum : 0.0f;
      u = l == -INFINITY ? 0.0f : expf(l - top) * inv;
      const float dot = __shfl(lanes_sum<8>(u * g), base);  // lanes from 8 on hold no expert
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] = -x[v] * inv * dot;
      u *= g;
    } else if (a.renorm) {
      const float sum = lanes_sum<8>(u);
      u = sum > 0 ? u / sum : 0.0f;
      u *= g - lanes_sum<8>(u * g);
      if constexpr (kSigmoid) u /= 1.0f + expf(l);
    } else {
      u *= g / (1.0f + expf(l));
    }
    for (uint32_t j = 0; j < a.k; ++j) {
      const int e = __shfl(id, base + (int)j);
      const float x = __shfl(u, base + (int)j);
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] += e == 4 * sub + v ? x : 0.0f;
    }
    if (t < a.tokens) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t e = 4 * sub + v;
        if (e >= a.E) continue;
        if (a.add && live) d[v] += a.add[t * a.E + e];
        a.dlogits[t * a.E + e] = live ? d[v] : 0.0f;
      }
    }
  }
}

int validate(const pw_route_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->tokens > (1ull << 28)) return fail(PW_ERR_INVALID, "tokens must be at most 2^28");
  if (d->num_experts < 2 || d->num_experts > kMaxRouteExperts)
    return fail(PW_ERR_INVALID, "num_experts must be in [2, %u]", kMaxRouteExperts);
  if (d->top_k < 1 || d->top_k > kMaxK || d->top_k > d->num_experts)
    return fail(PW_ERR_INVALID, "top_k must be in [1, 8] and at most num_experts");
  if (d->tokens * d->top_k > 0x7fffffffull) return fail(PW_ERR_INVALID, "tokens x top_k must stay below 2^31");
  if (d->score > PW_SCORE_SIGMOID) return fail(PW_ERR_INVALID, "unknown score %u", d->score);
  if (d->groups < 1 || d->groups > kMaxGroups || d->num_experts % d->groups)
    return fail(PW_ERR_INVALID, "groups must be in [1, %u] and divide num_experts", kMaxGroups);
  if (d->top_groups < 1 || d->top_groups > d->groups) return fail(PW_ERR_INVALID, "top_groups must be in [1, groups]");
  if (d->group_best < 1 || d->group_best > 2) return fail(PW_ERR_INVALID, "group_best must be 1 or 2");
  if (d->renorm > 1) return fail(PW_ERR_INVALID, "renorm must be 0 or 1");
  if (!isfinite(d->scale)) return fail(PW_ERR_INVALID, "the scale must be finite");
  return PW_OK;
}

RouteArgs args(const pw_route_desc& d, const pw_route_io& io) {
  RouteArgs a{};
  a.logits = io.logits;
  a.bias = io.bias;
  a.valid = io.valid;
  a.experts = io.experts;
  a.weights = io.weights;
  a.dweights = io.dweights;
  a.add = io.add;
  a.dlogits = io.dlogits;
  a.tokens = (uint32_t)d.tokens;
  a.E = d.num_experts;
  a.k = d.top_k;
  a.groups = d.groups;
  a.top_groups = d.top_groups;
  a.group_best = d.group_best;
  a.by_group = d.top_groups < d.groups;
  a.renorm = d.renorm;
  a.scale = d.scale;
  a.names = a.E <= 4 ? 3 : a.E <= 16 ? 15 : a.E <= 64 ? 63 : 255;
  a.cut = ldexpf((float)(a.names + 1), -23);
  const uint32_t size = a.E / a.groups;
  a.per_group = (65536 + size - 1) / size;
  return a;
}

template <int L, int C, int K, bool kSigmoid>
void launch_route_k(const RouteArgs& a, hipStream_t s) {
  constexpr uint32_t R = kThreads / L;
  const uint32_t lds = a.by_group ? R * a.E * sizeof(double) : 0;
  hipLaunchKernelGGL((k_route<L, C, K, kSigmoid>), dim3(std::min((a.tokens + R - 1) / R, kMaxGrid)), dim3(kThreads), lds, s, a);
}

template <int L, int C, bool kSigmoid>
void launch_route_lanes(const RouteArgs& a, hipStream_t s) {
  if (a.k <= 2) launch_route_k<L, C, 2, kSigmoid>(a, s);
  else if (a.k <= 4) launch_route_k<L, C, 4, kSigmoid>(a, s);
  else if (a.k <= 6) launch_route_k<L, C, 6, kSigmoid>(a, s);
  else launch_route_k<L, C, 8, kSigmoid>(a, s);
}

template <bool kSigmoid>
void launch_route(const RouteArgs& a, hipStream_t s) {
  const bool many = a.tokens >= kManyTokens;
  if (a.E <= 16) launch_route_lanes<4, 1, kSigmoid>(a, s);
  else if (a.E <= 64) many ? launch_route_lanes<4, 4, kSigmoid>(a, s) : launch_route_lanes<16, 1, kSigmoid>(a, s);
  else many ? launch_route_lanes<16, 4, kSigmoid>(a, s) : launch_route_lanes<64, 1, kSigmoid>(a, s);
}

template <int L, bool kSigmoid>
void launch_grad(const RouteArgs& a, hipStream_t s) {
  constexpr uint32_t R = kThreads / L;
  hipLaunchKernelGGL((k_route_grad<L, kSigmoid>), dim3(std::min((a.tokens + R - 1) / R, kMaxGrid)), dim3(kThreads), 0, s,
                     a);
}

#define PW_BY_SCORE(fn, score, a, s)                                                                 \
  do {                                                                                               \
    if ((a).E <= 64) (score) == PW_SCORE_SIGMOID ? fn<16, true>(a, s) : fn<16, false>(a, s);         \
    else (score) == PW_SCORE_SIGMOID ? fn<64, true>(a, s) : fn<64, false>(a, s);                     \
  } while (0)

}  // namespace

}  // namespace pw

using namespace pw;

extern "C" int pw_route(const pw_route_desc* d, const pw_route_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->tokens == 0) return PW_OK;
  if (!io->logits || !io->experts || !io->weights)
    return fail(PW_ERR_INVALID, "logits, experts and weights are required");
  if (misaligned({io->logits, io->bias, io->experts, io->weights}, 4))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const RouteArgs a = args(*d, *io);
  d->score == PW_SCORE_SIGMOID ? launch_route<true>(a, s) : launch_route<false>(a, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch route");
}

extern "C" int pw_route_grad(const pw_route_desc* d, const pw_route_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->tokens == 0) return PW_OK;
  if (!io->logits || !io->experts || !io->dweights || !io->dlogits)
    return fail(PW_ERR_INVALID, "logits, experts, dweights and dlogits are required");
  if (misaligned({io->logits, io->experts, io->dweights, io->add, io->dlogits}, 4))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const RouteArgs a = args(*d, *io);
  PW_BY_SCORE(launch_grad, d->score, a, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch route_grad");
}
