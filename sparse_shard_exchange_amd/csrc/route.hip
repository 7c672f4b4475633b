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
};

// A logit as it is used: +infinity is the largest finite value, NaN is none.
__device__ __forceinline__ float usable(float l) { return l == l ? fminf(l, FLT_MAX) : -INFINITY; }

__device__ __forceinline__ double shuffle_xor(double v, int m) { return __shfl_xor(v, m); }

// The larger of two (value, index) pairs; equal values: the lower index.
__device__ __forceinline__ bool beats(double a, int i, double b, int j) { return a > b || (a == b && i < j); }

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

// L lanes a token, four neighbouring experts a lane.
template <int L, bool kSigmoid>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a) {
  constexpr int kRows = kThreads / L;
  __shared__ double s_c[kRows][4 * L];
  const int sub = threadIdx.x % L, row = threadIdx.x / L;
  for (uint64_t t0 = (uint64_t)blockIdx.x * kRows; t0 < a.tokens; t0 += (uint64_t)gridDim.x * kRows) {
    const uint64_t t = t0 + row;
    const bool live = t < a.tokens && (!a.valid || a.valid[t]);
    const float* in = a.logits + (t < a.tokens ? t : 0) * a.E;
    float l[4];
    double c[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t e = 4 * sub + v;
      l[v] = live && e < a.E ? usable(in[e]) : -INFINITY;
    }
    float top = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
    top = lanes_max<L>(top);
    double total = 1.0;
    if constexpr (!kSigmoid) {
      double sum = 0.0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        c[v] = l[v] == -INFINITY ? 0.0 : exp((double)l[v] - (double)top);
        sum += c[v];
      }
#pragma unroll
      for (int m = 1; m < L; m *= 2) sum += shuffle_xor(sum, m);
      total = sum;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t e = 4 * sub + v;
      if constexpr (kSigmoid) c[v] = 1.0 / (1.0 + exp(-(double)l[v]));
      else c[v] = c[v] / total;
      if (a.bias && e < a.E) c[v] += (double)a.bias[e];
      if (l[v] == -INFINITY || !(c[v] > -(double)INFINITY)) c[v] = -(double)INFINITY;
    }
    if (a.by_group) {
#pragma unroll
      for (int v = 0; v < 4; ++v) s_c[row][4 * sub + v] = c[v];
      __syncthreads();
      const uint32_t size = a.E / a.groups;
      double mark = -(double)INFINITY;
      if ((uint32_t)sub < a.groups) {
        double m1 = mark, m2 = mark;
        for (uint32_t i = 0; i < size; ++i) {
          const double x = s_c[row][sub * size + i];
          m2 = fmax(m2, fmin(m1, x));
          m1 = fmax(m1, x);
        }
        mark = a.group_best == 2 && m2 > -(double)INFINITY ? m1 + m2 : m1;
      }
      uint32_t better = 0;
      const int base = (threadIdx.x & 63) / L * L;
      for (uint32_t g = 0; g < a.groups; ++g) {
        const double m = __shfl(mark, base + (int)g);
        better += beats(m, g, mark, sub);
      }
      const bool kept = (uint32_t)sub < a.groups && better < a.top_groups;
      const uint64_t mask = __ballot(kept) >> base;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (!(mask >> ((4 * sub + v) / size) & 1)) c[v] = -(double)INFINITY;
      __syncthreads();
    }
    int mine = (int)a.E;         // lane j: the j-th expert
    float logit = -INFINITY;     // and its logit
    for (uint32_t j = 0; j < a.k; ++j) {
      double best = c[0];
      int at = 4 * sub;
#pragma unroll
      for (int v = 1; v < 4; ++v)
        if (c[v] > best) best = c[v], at = 4 * sub + v;
#pragma unroll
      for (int m = 1; m < L; m *= 2) {
        const double o = shuffle_xor(best, m);
        const int i = __shfl_xor(at, m);
        if (beats(o, i, best, at)) best = o, at = i;
      }
      const bool some = best > -(double)INFINITY;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * sub + v == at) c[v] = -(double)INFINITY;
      if ((uint32_t)sub == j && some) {
        mine = at;
        logit = usable(in[at]);
      }
    }
    float u = chosen_score<kSigmoid>((uint32_t)sub < a.k ? logit : -INFINITY, a.renorm);
    if (a.renorm) {
      const float sum = lanes_sum<8>(u);
      u = sum > 0 ? u / sum : 0.0f;
    } else if constexpr (!kSigmoid) {
      u = logit == -INFINITY ? 0.0f : (float)(exp((double)logit - (double)top) / total);
    }
    if (t < a.tokens && (uint32_t)sub < a.k) {
      a.experts[t * a.k + sub] = mine;
      a.weights[t * a.k + sub] = mine < (int)a.E ? a.scale * u : 0.0f;
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
  return a;
}

template <int L, bool kSigmoid>
void launch_route(const RouteArgs& a, hipStream_t s) {
  constexpr uint32_t R = kThreads / L;
  hipLaunchKernelGGL((k_route<L, kSigmoid>), dim3(std::min((a.tokens + R - 1) / R, kMaxGrid)), dim3(kThreads), 0, s, a);
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
  PW_BY_SCORE(launch_route, d->score, a, s);
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
