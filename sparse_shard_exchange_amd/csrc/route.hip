// Routing of tokens to experts for any score, bias, groups and top-k, and the
// gradient of its weights.
//
//   s_e = softmax(l)_e or 1 / (1 + e^-l_e),  c_e = s_e + b_e
//   the top_groups groups with the highest sums of their best c stay, the k
//   highest c of those are chosen, w_j = scale s_ej (/ sum_j s_ej)
#include "ops.h"

#include <float.h>

#include <algorithm>

#include "route_key.h"

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxRouteExperts = 256, kMaxK = 8, kMaxGroups = 16;
// Fewer lanes a token, and a second launch, from so many logits on (of more than 16
// experts; 64 experts, k = 6: 16384 tokens 11.3 us so and 10.0 us in one launch, 131072 27
// and 54; 256 experts in groups, k = 8: 4096 tokens 16.6 and 13.2 us, 8192 17.8 and 21.9;
// 131072 tokens of 8 experts 8.9 and 7.0).
constexpr uint64_t kManyLogits = 1ull << 21;

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

// A logit as it is used: +infinity is the largest finite value, NaN is none (the
// larger of a NaN and a number is the number).
__device__ __forceinline__ float usable(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

// ---- the choice -------------------------------------------------------------------
//
// L lanes a token, C times four neighbouring experts a lane. The choice is that
// of 64-bit scores, but few tokens need them: the values that order the experts
// (logits where nothing is added to their scores and no group is marked, else
// c in fp32) are cut to the bits that leave room for the expert's number, so
// that one 32-bit integer orders and names an expert, and the k + 2 best are
// found with integer maxima. Tokens of whose order this leaves a doubt are listed
// and seen to at the end: where two of the k + 1 best are so close that the cut or
// the fp32 evaluation might have exchanged them, these are compared in 64 bits (16
// lanes a token); where even the (k + 2)-th might belong to the k best, or two
// groups' marks are that close, or the scores are a softmax, whose 64-bit value
// needs all logits, a wave takes the token anew in 64 bits. Where logits alone order
// the experts, those of fewer bits than are cut (bf16 ones) leave no doubt. Equal scores do,
// and so do scores that fp32 cannot tell apart.
//
// What doubt costs, 131072 x 64, k = 6, softmax / sigmoid. Random fp32 logits: 22 / 21 us by
// logits alone, 35 / 27 with a bias, 45 / 43 in groups. Every token taken anew, one after the
// other by its wave (equal logits and a zero bias; a softmax whose lesser half fp32 sees as
// one value; sigmoids of logits about 30): 420 / 400, in groups 480 / 455, less than the plain form's
// 1570. bf16 logits and a zero bias: 137 / 47, in groups 156 / 54; with a bias of random bits as
// fp32 ones. 4096 x 64: 5.5, 9.3 / 6.3, 11 without, 28 / 27, 31 with every token in doubt.
//
// What bounds it: 32 x 256 in groups takes 7.7 us, a launch and one chain of dependent
// steps (the row, its scores, the groups' marks, eight maxima, the weights); 131072 x 64,
// k = 6, sigmoid with bias 23.7 us, of vector instructions (three of four cycles of a SIMD issue one, with
// 2.7 waves; its 40 MB would take 6.1), and 4.4 to 5 of the second launch. All in 64 bits, as a simple kernel does it, takes 51.6.

constexpr int32_t kLowest = (int32_t)0x80800000;  // of the finite values; those below are no experts

template <int M>
__device__ __forceinline__ int32_t across_int(int32_t v) {
  return __builtin_bit_cast(int32_t, across<M>(__builtin_bit_cast(float, v)));
}
template <int L, int M = 1>
__device__ __forceinline__ int32_t lanes_max_int(int32_t v) {
  if constexpr (M >= L) return v;
  else if constexpr (M < 16) return lanes_max_int<L, 2 * M>(max(v, across_int<M>(v)));
  else if constexpr (M == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);  // rows 0 0 2 2 and 1 1 3 3
    return lanes_max_int<L, 32>(max((int32_t)r[0], (int32_t)r[1]));
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max((int32_t)r[0], (int32_t)r[1]);
  }
}
template <int L, int M = 1>
__device__ __forceinline__ uint32_t lanes_or(uint32_t v) {
  if constexpr (M < L) return lanes_or<L, 2 * M>(v | (uint32_t)across_int<M>((int32_t)v));
  return v;
}
__device__ __forceinline__ int32_t middle(int32_t a, int32_t b, int32_t c) { return max(min(a, b), min(max(a, b), c)); }

// A token's logits in its lanes: element v of the lane's chunk i is expert
// first(i) + v. The last chunk is moved back to end with the row; what the chunk
// before has of it counts as no expert, as does what lies behind the row.
template <int L, int C>
struct Token {
  const float* in;
  float l[4 * C];
  uint32_t E, sub;
  __device__ __forceinline__ uint32_t first(int i) const { return min(4 * (i * L + sub), max(E, 4u) - 4); }
  __device__ __forceinline__ uint32_t expert(int i) const { return first(i / 4) + i % 4; }  // of l[i]
  __device__ __forceinline__ uint32_t skipped(int i, bool live) const {  // of chunk i's elements
    const uint32_t c = 4 * (i * L + sub);
    return live && c < E ? c - first(i) : 4u;
  }
  __device__ __forceinline__ void load(const RouteArgs& a, uint64_t at, bool live) {
    typedef float At __attribute__((ext_vector_type(4), aligned(4)));
    typedef float Vec __attribute__((ext_vector_type(4)));
    in = a.logits + at * a.E;
    E = a.E;
    Vec x[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      if (E >= 4) {
        x[i] = *reinterpret_cast<const At*>(in + first(i));
      } else {
#pragma unroll
        for (uint32_t v = 0; v < 4; ++v) x[i][v] = in[min(v, E - 1)];
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const uint32_t skip = skipped(i, live);
#pragma unroll
      for (uint32_t v = 0; v < 4; ++v) l[4 * i + v] = v >= skip && v < E ? usable(x[i][v]) : -INFINITY;
    }
  }
  __device__ __forceinline__ float top() const {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < 4 * C; ++i) m = fmaxf(m, l[i]);
    return lanes_max<L>(m);
  }
};

// The kept groups as bits, from the row's c in LDS (no expert: -infinity); *close:
// the marks of a kept and a left one differ by `margin` (relatively, or of one) and
// the rounding of their members or less. A member is off by 2^-24 of itself, which may be far
// more than of their sum, the mark: four of them, two a mark, by 2^-22 of the largest. A mark
// of two lowest values that passes the range of fp32 tells nothing.
template <int L, typename F>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, const F* c, uint32_t sub, F margin, bool* close) {
  constexpr int kEach = L >= (int)kMaxGroups ? 1 : (int)kMaxGroups / L;  // groups of a lane
  constexpr int kShare = L > (int)kMaxGroups ? L / (int)kMaxGroups : 1;   // neighbouring lanes of a group
  const uint32_t size = a.E / a.groups;
  const F low = -(F)INFINITY;
  F mark[kEach], largest = 0;
  uint32_t lost = 0;
#pragma unroll
  for (int h = 0; h < kEach; ++h) {
    const uint32_t g = (h * L + sub) / kShare;
    F m1 = low, m2 = low;
    if (g < a.groups) {
      uint32_t at = (g + sub % kShare) % size;  // lanes begin in different banks
      for (uint32_t i = sub % kShare; i < size; i += kShare) {
        const F x = c[g * size + at];
        at = at + kShare < size ? at + kShare : at + kShare - size;
        m2 = max(m2, min(m1, x));
        m1 = max(m1, x);
      }
    }
#pragma unroll
    for (int m = 1; m < kShare; m *= 2) {
      const F o1 = __shfl_xor(m1, m), o2 = __shfl_xor(m2, m);
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    }
    const bool two = a.group_best == 2 && m2 > low;
    mark[h] = two ? m1 + m2 : m1;
    if (m1 > low) largest = max(largest, max((F)fabs(m1), two ? (F)fabs(m2) : (F)0));
    lost |= m1 > low && !(mark[h] > low);
  }
  uint32_t better[kEach] = {}, kept = 0;
  const int base = (int)(threadIdx.x & 63) / L * L;
  for (uint32_t g = 0; g < a.groups; ++g) {
    F m = mark[0];
#pragma unroll
    for (int h = 1; h < kEach; ++h)
      if (g / L == (uint32_t)h) m = mark[h];
    m = __shfl(m, base + (int)(g * kShare % L));
#pragma unroll
    for (int h = 0; h < kEach; ++h) better[h] += m > mark[h] || (m == mark[h] && g < (h * L + sub) / kShare);
  }
  F least = (F)INFINITY, most = low;  // of the kept, of the left
#pragma unroll
  for (int h = 0; h < kEach; ++h) {
    const uint32_t g = (h * L + sub) / kShare;
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
    largest = max(largest, (F)__shfl_xor(largest, m));
  }
  *close = lanes_or<L>(lost) || (most > low && !(least - most > margin * (1 + max(fabs(least), fabs(most))) + (F)0x1p-22 * largest));
  return kept;
}

// c in LDS, then the experts of left groups out of it.
template <int L, int C, typename F>
__device__ __forceinline__ void leave_groups(const RouteArgs& a, const Token<L, C>& t, F* s_c, F (&c)[4 * C], F margin, bool* close) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const uint32_t skip = t.skipped(i, true);
#pragma unroll
    for (uint32_t v = 0; v < 4; ++v)
      if (v >= skip && v < t.E) s_c[t.first(i) + v] = c[4 * i + v];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const uint32_t kept = keep_groups<L, F>(a, s_c, t.sub, margin, close);
#pragma unroll
  for (int i = 0; i < 4 * C; ++i)
    if (!(kept >> (min(t.expert(i), a.E - 1) * a.per_group >> 16) & 1)) c[i] = -(F)INFINITY;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Lane q of the first eight of a token's (or of its four) has the q-th expert, with
// four lanes a token also the (q + 4)-th.
template <int L>
struct Places {
  static constexpr int kLanes = L < 8 ? L : 8, kEach = 8 / kLanes;
  int32_t id[kEach];  // E: none
};

// Experts and weights of token `at`; top and total: of its softmax (without renorm). Unlike
// the scores that order the experts, the weights take expf and divisions: a sigmoid's is a few
// 2^-24 off whatever its logit, a softmax's as many as logits are apart more, by
// the rounding of their difference.
template <int L, bool kSigmoid>
__device__ __forceinline__ void store_token(const RouteArgs& a, const float* in, uint64_t at, uint32_t sub, bool live,
                                            const Places<L>& p, float top, float total) {
  constexpr int kLanes = Places<L>::kLanes, kEach = Places<L>::kEach;
  float l[kEach], u[kEach], m = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int h = 0; h < kEach; ++h) l[h] = in[min((uint32_t)p.id[h], a.E - 1)];
#pragma unroll
  for (int h = 0; h < kEach; ++h) {
    l[h] = p.id[h] < (int32_t)a.E ? usable(l[h]) : -INFINITY;
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
    const uint32_t j = h * kLanes + sub;
    if (live && sub < (uint32_t)kLanes && j < a.k) {
      a.experts[at * a.k + j] = p.id[h];
      a.weights[at * a.k + j] = p.id[h] < (int32_t)a.E ? u[h] / by * a.scale : 0.0f;
    }
  }
}

// A token in 64 bits, by a wave.
template <bool kSigmoid>
__device__ __forceinline__ void route_exactly(const RouteArgs& a, uint64_t at, double* s_c) {
  typedef Places<64> P;
  Token<64, 1> t;
  t.sub = threadIdx.x & 63;
  t.load(a, at, true);
  const float top = t.top();
  double c[4], total = 1.0;
  if constexpr (!kSigmoid) {
    total = 0.0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      c[v] = t.l[v] == -INFINITY ? 0.0 : exp((double)t.l[v] - (double)top);
      total += c[v];
    }
#pragma unroll
    for (int m = 1; m < 64; m *= 2) total += __shfl_xor(total, m);
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if constexpr (kSigmoid) c[v] = 1.0 / (1.0 + exp(-(double)t.l[v]));
    else c[v] /= total;
    if (!a.bias && !a.by_group) c[v] = (double)t.l[v];
    if (a.bias) c[v] += (double)a.bias[min(t.expert(v), a.E - 1)];
    if (t.l[v] == -INFINITY || !(c[v] > -(double)INFINITY)) c[v] = -(double)INFINITY;
  }
  if (a.by_group) {
    bool close;
    leave_groups<64, 1, double>(a, t, s_c, c, 0.0, &close);
  }
  P place;
  place.id[0] = (int32_t)a.E;
#pragma unroll 1
  for (int j = 0; j < (int)a.k; ++j) {
    double best = -(double)INFINITY;
    int32_t e = (int32_t)a.E;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (c[v] > best) best = c[v], e = (int32_t)t.expert(v);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_xor(best, m);
      const int32_t n = __shfl_xor(e, m);
      if (o > best || (o == best && n < e)) best = o, e = n;
    }
    if ((int)t.sub % P::kLanes == j) place.id[0] = e;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if ((int32_t)t.expert(v) == e) c[v] = -(double)INFINITY;
  }
  store_token<64, kSigmoid>(a, t.in, at, t.sub, true, place, top, (float)total);
}

// The k best of k + 1 candidates, by 64-bit scores of a sigmoid, or by logits; 16
// lanes a token, lane q has the q-th candidate's key.
template <bool kSigmoid>
__device__ __forceinline__ void settle(const RouteArgs& a, uint64_t at, int32_t key) {
  typedef Places<16> P;
  const int q = threadIdx.x & 15, base = (int)(threadIdx.x & 48);
  const float* in = a.logits + at * a.E;
  const bool some = (uint32_t)q <= a.k && key >= kLowest;
  const uint32_t e = min(a.names - ((uint32_t)key & a.names), a.E - 1);
  double c = (double)usable(in[e]);
  if (a.bias || a.by_group) c = 1.0 / (1.0 + exp(-c));
  if (a.bias) c += (double)a.bias[e];
  if (!some) c = -(double)INFINITY;
  uint32_t before = 0;
  for (uint32_t j = 0; j <= a.k; ++j) {
    const double o = __shfl(c, base + (int)j);
    const uint32_t n = (uint32_t)__shfl((int)e, base + (int)j);
    before += o > c || (o == c && n < e);
  }
  const uint32_t mine = some ? before << 16 | e : ~0u;
  P place;
  place.id[0] = (int32_t)a.E;
  for (uint32_t j = 0; j <= a.k; ++j) {
    const uint32_t o = (uint32_t)__shfl((int)mine, base + (int)j);
    if (o >> 16 == (uint32_t)(q & 7) && o >> 16 < a.k) place.id[0] = (int32_t)(o & 0xffff);
  }
  float top = 0.0f, total = 1.0f;
  if (!kSigmoid && !a.renorm) {
    top = -INFINITY, total = 0.0f;
    for (uint32_t i = q; i < a.E; i += 16) top = fmaxf(top, usable(in[i]));
    top = lanes_max<16>(top);
    for (uint32_t i = q; i < a.E; i += 16) total += usable(in[i]) == -INFINITY ? 0.0f : expf(usable(in[i]) - top);
    total = lanes_sum<16>(total);
  }
  store_token<16, kSigmoid>(a, in, at, q, true, place, top, total);
}

// What k_route leaves in the first place of a token that k_route_rest sees to: one
// to be settled, whose other places and weights hold the k + 1 keys, or one to be
// taken anew.
constexpr int32_t kSettle = INT32_MIN, kAnew = INT32_MIN + 1;

// K: the largest top_k of this instance. kScored: c orders the experts, not their logits.
// kWhole: tokens in doubt are seen to here, else left for k_route_rest. The latter takes
// fewer registers (131072 x 64, k = 6, sigmoid with bias: 3 waves a SIMD instead of 2,
// 23 us instead of 41), for a launch more.
template <int L, int C, int K, bool kSigmoid, bool kScored, bool kWhole>
__global__ __launch_bounds__(kThreads, kWhole ? 2 : 3) void k_route(RouteArgs a) {
  constexpr int kRows = kThreads / L, N = K + 2, kList = N < 4 * C ? N : 4 * C;
  extern __shared__ __attribute__((aligned(16))) float s_rows[];  // by group: [rows][E], c
  constexpr bool kSettled = kSigmoid || !kScored;  // (a softmax needs all of its logits)
  __shared__ double s_c[kWhole && kScored ? kThreads / 64 : 1][kWhole && kScored ? kMaxRouteExperts : 1];
  __shared__ uint32_t s_listed[2];  // to be settled, to be taken anew
  __shared__ uint8_t s_list[2][kRows];
  __shared__ int32_t s_key[kWhole && kSettled ? kRows : 1][N];
  const uint32_t row = threadIdx.x / L, names = a.names, k = a.k;
  if constexpr (kWhole) {
    if (threadIdx.x < 2) s_listed[threadIdx.x] = 0;
    __syncthreads();
  }
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows; t0 < a.tokens; t0 += (uint64_t)gridDim.x * kRows) {
    const uint64_t at = min(t0 + row, (uint64_t)a.tokens - 1);
    const bool mine = t0 + row < a.tokens, live = !a.valid || a.valid[at];
    Token<L, C> t;
    t.sub = threadIdx.x % L;
    t.load(a, at, live);
    float c[4 * C], top = 0.0f, total = 1.0f;
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) c[i] = t.l[i];
    if constexpr (!kSigmoid) {
      if (kScored || !a.renorm) {
        top = t.top();
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < 4 * C; ++i) {
          const float z = t.l[i] == -INFINITY ? 0.0f : expf(t.l[i] - top);
          total += z;
          if (kScored) c[i] = z;
        }
        total = lanes_sum<L>(total);
      }
    }
    bool doubt = false, anew = false;
    // What two fp32 values of c are off by together, beside their last bits. Sigmoid:
    // the exponent is off by 1.5 x 2^-24 of itself, e^x, the sum and the reciprocal by 2^-23
    // each, and s (1 - s) |l| is at most 0.224: 4.3 x 2^-23 each. Softmax, with p the largest:
    // (D + 4) 2^-24 of e^-D p (D e^-D is at most 0.37) and 30 x 2^-24 of the sum and the
    // quotient: 35 p 2^-24 each.
    float off = 0x1p-19f;
    if constexpr (kScored) {
      const float inv = 1.0f / total;
      if constexpr (!kSigmoid) off = (1.0f + 70.0f * inv) * 0x1p-24f;
#pragma unroll
      for (int i = 0; i < 4 * C; ++i) {
        if constexpr (kSigmoid) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t.l[i] * -1.44269504f));
        else c[i] *= inv;
        if (a.bias) c[i] += fmaxf(a.bias[min(t.expert(i), a.E - 1)], -INFINITY);  // (of a NaN: -infinity)
        if (t.l[i] == -INFINITY) c[i] = -INFINITY;
      }
      if (a.by_group) leave_groups<L, C, float>(a, t, s_rows + row * a.E, c, 4 * off, &anew);
    }
    // the lane's best in order: each new one moves the lesser ones down
    int32_t list[kList];
    uint32_t cut = 0;  // bits that the keys lack
#pragma unroll
    for (int n = 0; n < kList; ++n) list[n] = INT32_MIN;
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) {
      const float v = kScored ? c[i] : c[i] + 0.0f;  // (s + b is no negative zero)
      if (!kScored) cut |= v == -INFINITY ? 0u : key_lacks(v, names);
      const int32_t x = route_key(v, t.expert(i), names);
#pragma unroll
      for (int n = (i < kList - 1 ? i : kList - 1); n > 0; --n) list[n] = middle(list[n - 1], x, list[n]);
      list[0] = max(list[0], x);
    }
    // the token's best, and whether they are in order
    if (!kScored) cut = lanes_or<L>(cut);
    typedef Places<L> P;
    P place;
#pragma unroll
    for (int h = 0; h < P::kEach; ++h) place.id[h] = INT32_MIN;
    int32_t one = 0, two = 0, keys[N];  // one, two: the keys before
    float u1 = 0.0f, u2 = 0.0f;         // and their values
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t best = lanes_max_int<L>(list[0]);
      if (j < K && (int)t.sub % P::kLanes == j % P::kLanes) place.id[j / P::kLanes] = best;
      const float v = unordered(best & (int32_t)~names);
      // (j - 1, j) up to the (k + 1)-th, and the (k + 2)-th against the k-th
      if (j > 0 && (uint32_t)j <= k + 1) {
        bool near;
        if constexpr (kScored) {
          // the lesser one may be a whole cut higher
          const float u = (uint32_t)j <= k ? u1 : u2;
          near = !(u - v > fmaf(fmaxf(fabsf(u), fabsf(v)), a.cut + 0x1p-22f, off));
        } else {
          near = cut && ((uint32_t)(((uint32_t)j <= k ? one : two) ^ best) & ~names) == 0;
        }
        near &= best >= kLowest;
        if ((uint32_t)j <= k && kSettled) doubt |= near;
        else anew |= near;
      }
      keys[j] = best;
      two = one;
      one = best;
      u2 = u1;
      u1 = v;
      const bool pop = list[0] == best;
#pragma unroll
      for (int n = 0; n + 1 < kList; ++n)
        if (n + j + 1 < N) list[n] = pop ? list[n + 1] : list[n];
      if (pop) list[kList - 1] = INT32_MIN;
    }
#pragma unroll
    for (int h = 0; h < P::kEach; ++h) {
      const bool some = (uint32_t)h * P::kLanes + t.sub % P::kLanes < k && place.id[h] >= kLowest;
      place.id[h] = some ? (int32_t)(names - ((uint32_t)place.id[h] & names)) : (int32_t)a.E;
    }
    store_token<L, kSigmoid>(a, t.in, at, t.sub, mine && !doubt && !anew, place, top, total);
    if constexpr (!kWhole) {
      if (doubt || anew) {
        if (k == 1) anew = true;  // no room for two keys
        if (mine && t.sub == 0) {
          a.experts[at * k] = anew ? kAnew : kSettle;
          if (kSettled && !anew) {
#pragma unroll
            for (int j = 0; j < N - 1; ++j)
              if ((uint32_t)j <= k) {
                int32_t* to = (uint32_t)j + 1 < k ? a.experts + at * k + j + 1 : reinterpret_cast<int32_t*>(a.weights) + at * k + j + 1 - k;
                *to = keys[j];
              }
          }
        }
      }
    } else {
      if ((doubt || anew) && mine && t.sub == 0) {
        s_list[anew][atomicAdd(&s_listed[anew], 1u)] = (uint8_t)row;
        if constexpr (kSettled) {
#pragma unroll
          for (int j = 0; j < N; ++j) s_key[row][j] = keys[j];
        }
      }
      __syncthreads();
      const uint32_t settled = s_listed[0], again = s_listed[1];
      __syncthreads();  // before the next tokens are listed
      if (settled | again) {
        if constexpr (kSettled) {
          for (uint32_t i = threadIdx.x / 16; i < settled; i += kThreads / 16)
            settle<kSigmoid>(a, t0 + s_list[0][i], s_key[s_list[0][i]][min(threadIdx.x & 15, k)]);
        }
        for (uint32_t i = threadIdx.x / 64; i < again; i += kThreads / 64)
          route_exactly<kSigmoid>(a, t0 + s_list[1][i], s_c[kScored ? threadIdx.x / 64 : 0]);
        __syncthreads();
        if (threadIdx.x < 2) s_listed[threadIdx.x] = 0;
        __syncthreads();
      }
    }
  }
}

// The tokens that k_route left, out of 64 a wave: their marks are found in one load and
// a vote, so tokens without doubt cost this launch four bytes each.
template <bool kSigmoid>
__global__ __launch_bounds__(kThreads) void k_route_rest(RouteArgs a) {
  __shared__ double s_c[kThreads / 64][kMaxRouteExperts];
  const uint32_t lane = threadIdx.x & 63, w = threadIdx.x / 64;
  for (uint64_t t0 = ((uint64_t)blockIdx.x * (kThreads / 64) + w) * 64; t0 < a.tokens; t0 += (uint64_t)gridDim.x * kThreads) {
    const int32_t place = t0 + lane < a.tokens ? a.experts[(t0 + lane) * a.k] : 0;
    uint64_t settled = __ballot(place == kSettle), again = __ballot(place == kAnew);
    while (settled) {  // four at a time, 16 lanes each
      int mine = -1;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if ((int)lane / 16 == g && settled) mine = __builtin_ctzll(settled);
        settled &= settled - 1;
      }
      if (mine >= 0) {
        const uint64_t at = t0 + mine;
        const uint32_t j = min(lane & 15, a.k);
        const int32_t* from = j + 1 < a.k ? a.experts + at * a.k + j + 1 : reinterpret_cast<const int32_t*>(a.weights) + at * a.k + j + 1 - a.k;
        settle<kSigmoid>(a, at, *from);
      }
    }
    while (again) {
      const int mine = __builtin_ctzll(again);
      again &= again - 1;
      route_exactly<kSigmoid>(a, t0 + mine, s_c[w]);
    }
  }
}

// ---- the gradient -----------------------------------------------------------------
//
// With v_j = s_ej / sum s over the chosen and g_j = scale dw_j:
//   renorm:     dl_ej = v_j (g_j - sum_i g_i v_i), times 1 - s_ej for a sigmoid (the sum
//               over the chosen drops out, so ratios that underflow keep their gradient)
//   otherwise:  dl_ej = g_j s_ej (1 - s_ej) for a sigmoid,
//               dl_e = s_e (sum of the g_j with e_j = e - sum_j g_j s_ej) for a softmax
// L lanes a token, four neighbouring experts a lane; the chosen ones' logits are gathered,
// each by its own lane, all at once. Bound by vector instructions (one in nearly every cycle) and
// memory alike: 131072 x 64, k = 6, with add, in 18.4 us (77 MB needed; the gathered logits bring
// whole lines, 110 MB: 6 TB/s); a softmax without renorm or add 17.8. Four lanes a token up to 16 experts, not 16: 131072 x 16 7.4 us instead of 14.1.
template <int L, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void k_route_grad(RouteArgs a) {
  typedef float At __attribute__((ext_vector_type(4), aligned(4)));
  typedef float Vec __attribute__((ext_vector_type(4)));
  constexpr int kRows = kThreads / L, kLanes = Places<L>::kLanes, kEach = Places<L>::kEach;
  const uint32_t sub = threadIdx.x % L, row = threadIdx.x / L;
  const int base = (threadIdx.x & 63) / L * L;
  const bool whole = 4 * sub + 4 <= a.E;
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows; t0 < a.tokens; t0 += (uint64_t)gridDim.x * kRows) {
    const uint64_t t = t0 + row;
    const bool live = t < a.tokens && (!a.valid || a.valid[t]);
    const float* in = a.logits + (t < a.tokens ? t : 0) * a.E;
    int id[kEach];
    float g[kEach], l[kEach], u[kEach], m = -INFINITY;
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      const uint32_t j = h * kLanes + sub;
      id[h] = -1;
      g[h] = 0.0f, l[h] = -INFINITY;
      if (live && sub < (uint32_t)kLanes && j < a.k) {
        id[h] = a.experts[t * a.k + j];
        if ((uint32_t)id[h] < a.E) {
          l[h] = usable(in[id[h]]);
          g[h] = a.dweights[t * a.k + j] * a.scale;
        }
      }
      if (l[h] == -INFINITY) g[h] = 0.0f;  // no expert
      m = fmaxf(m, l[h]);
    }
    // s, or s e^-m with m = min(0, the largest logit): the ratios of scores that underflow
    m = lanes_max<kLanes>(m);
    if constexpr (kSigmoid) m = a.renorm ? fminf(m, 0.0f) : 0.0f;
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      u[h] = 0.0f;
      if (l[h] == -INFINITY) continue;
      if constexpr (kSigmoid) u[h] = expf(fminf(l[h], 0.0f) - m) / (1.0f + expf(-fabsf(l[h])));
      else u[h] = expf(l[h] - m);
    }
    auto sum_of = [&](auto f) {
      float s = 0.0f;
#pragma unroll
      for (int h = 0; h < kEach; ++h) s += f(h);
      return lanes_sum<kLanes>(s);
    };
    float d[4] = {0, 0, 0, 0};
    if (!kSigmoid && !a.renorm) {  // the softmax over all experts
      float x[4], top = -INFINITY, sum = 0.0f;
      if (whole) {
        const Vec q = *reinterpret_cast<const At*>(in + 4 * sub);
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = live ? usable(q[v]) : -INFINITY;
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = live && 4 * sub + v < a.E ? usable(in[4 * sub + v]) : -INFINITY;
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) top = fmaxf(top, x[v]);
      top = lanes_max<L>(top);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x[v] = x[v] == -INFINITY ? 0.0f : expf(x[v] - top);
        sum += x[v];
      }
      sum = lanes_sum<L>(sum);
      const float inv = sum > 0 ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int h = 0; h < kEach; ++h) u[h] = l[h] == -INFINITY ? 0.0f : expf(l[h] - top) * inv * g[h];
      const float dot = __shfl(sum_of([&](int h) { return u[h]; }), base);  // lanes from 8 on hold no expert
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] = -x[v] * inv * dot;
    } else if (a.renorm) {
      const float sum = sum_of([&](int h) { return u[h]; });
#pragma unroll
      for (int h = 0; h < kEach; ++h) u[h] = sum > 0 ? u[h] / sum : 0.0f;
      const float dot = sum_of([&](int h) { return u[h] * g[h]; });
#pragma unroll
      for (int h = 0; h < kEach; ++h) {
        u[h] *= g[h] - dot;
        if constexpr (kSigmoid) u[h] /= 1.0f + expf(l[h]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < kEach; ++h) u[h] *= g[h] / (1.0f + expf(l[h]));
    }
    for (uint32_t j = 0; j < a.k; ++j) {
      const int at = base + (int)j % kLanes;
      int e = __shfl(id[0], at);
      float x = __shfl(u[0], at);
#pragma unroll
      for (int h = 1; h < kEach; ++h) {
        const int eh = __shfl(id[h], at);
        const float xh = __shfl(u[h], at);
        if ((int)j / kLanes == h) e = eh, x = xh;
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] += e == (int)(4 * sub + v) ? x : 0.0f;
    }
    if (t >= a.tokens) continue;
    float* out = a.dlogits + t * a.E + 4 * sub;
    if (whole) {
      Vec r = {d[0], d[1], d[2], d[3]};
      if (a.add) r += *reinterpret_cast<const At*>(a.add + t * a.E + 4 * sub);
      __builtin_nontemporal_store(live ? r : Vec{}, reinterpret_cast<At*>(out));
    } else {
#pragma unroll
      for (uint32_t v = 0; v < 4; ++v) {
        if (4 * sub + v >= a.E) continue;
        if (a.add) d[v] += a.add[t * a.E + 4 * sub + v];
        out[v] = live ? d[v] : 0.0f;
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

template <int L, int C, int K, bool kSigmoid, bool kWhole>
void launch_route_k(const RouteArgs& a, hipStream_t s) {
  constexpr uint32_t R = kThreads / L;
  const dim3 grid(std::min((a.tokens + R - 1) / R, kMaxGrid));
  if (a.bias || a.by_group)
    hipLaunchKernelGGL((k_route<L, C, K, kSigmoid, true, kWhole>), grid, dim3(kThreads), a.by_group ? R * a.E * sizeof(float) : 0, s, a);
  else
    hipLaunchKernelGGL((k_route<L, C, K, kSigmoid, false, kWhole>), grid, dim3(kThreads), 0, s, a);
}

template <int L, int C, bool kSigmoid, bool kWhole>
void launch_route_lanes(const RouteArgs& a, hipStream_t s) {
  if (a.k <= 2) launch_route_k<L, C, 2, kSigmoid, kWhole>(a, s);
  else if (a.k <= 4) launch_route_k<L, C, 4, kSigmoid, kWhole>(a, s);
  else if (a.k <= 6) launch_route_k<L, C, 6, kSigmoid, kWhole>(a, s);
  else launch_route_k<L, C, 8, kSigmoid, kWhole>(a, s);
}

template <bool kSigmoid>
hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.E <= 16 || (uint64_t)a.tokens * a.E < kManyLogits) {
    if (a.E <= 16) launch_route_lanes<4, 1, kSigmoid, true>(a, s);
    else if (a.E <= 64) launch_route_lanes<16, 1, kSigmoid, true>(a, s);
    else launch_route_lanes<64, 1, kSigmoid, true>(a, s);
    return hipGetLastError();
  }
  if (a.E <= 64) launch_route_lanes<4, 4, kSigmoid, false>(a, s);
  else launch_route_lanes<16, 4, kSigmoid, false>(a, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const uint32_t blocks = (a.tokens + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(k_route_rest<kSigmoid>, dim3(std::min(blocks, kMaxGrid)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int L, bool kSigmoid>
void launch_grad(const RouteArgs& a, hipStream_t s) {
  constexpr uint32_t R = kThreads / L;
  hipLaunchKernelGGL((k_route_grad<L, kSigmoid>), dim3(std::min((a.tokens + R - 1) / R, kMaxGrid)), dim3(kThreads), 0, s,
                     a);
}

#define PW_BY_SCORE(fn, score, a, s)                                                                 \
  do {                                                                                               \
    if ((a).E <= 16) (score) == PW_SCORE_SIGMOID ? fn<4, true>(a, s) : fn<4, false>(a, s);          \
    else if ((a).E <= 64) (score) == PW_SCORE_SIGMOID ? fn<16, true>(a, s) : fn<16, false>(a, s);         \
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
  const hipError_t e = d->score == PW_SCORE_SIGMOID ? launch_route<true>(a, s) : launch_route<false>(a, s);
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
