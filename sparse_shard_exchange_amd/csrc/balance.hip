// Router balance: the loss that keeps a router's load even, per-expert tuple
// counts, and the whole gradient of the router logits.
//
//   p = softmax(l_t), n = valid tokens, c_e = tuples routed to e
//   L0 = a E sum_e c_e / (k n) * (1/n sum_t p_te)      L1 = b / n sum_t lse_t^2
//   dl_te = u0 a E / (k n^2) p_te (c_e - sum_j c_j p_tj) + u1 2 b / n lse_t p_te
//           + sum_s [expert_ts = e] g_ts (dg_ts - sum_j g_tj dg_tj)
//
// Both kernels read each logit once: a token's row is spread over a group of
// L lanes of 4 experts each (L = 4, 16, 64 for E <= 16, 64, 256), so a wave's
// load covers 64 / L whole rows, and the row's maximum, sum and dot product
// are lane exchanges inside the group.
#include "ops.h"

#include <algorithm>

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxBalanceExperts = 256;
constexpr uint32_t kParts = 256;        // partial sums at most (workgroups of k_balance)
constexpr uint32_t kAlone = 2048;       // tokens up to which one workgroup does all
constexpr uint32_t kRows = 4;           // rows of a group in flight

struct BalanceArgs {
  const float* logits;
  const int32_t* experts;
  const uint8_t* valid;
  int32_t* counts;
  float* prob_mean;
  float* loss;
  const float* gates;
  const float* dgates;
  const float* grad_loss;
  float* dlogits;
  float* part_p;    // [parts][E] sums of probabilities
  int32_t* part_c;  // [parts][E + 1] tuples per expert; valid tokens
  float* part_z;    // [parts] sums of squared logarithms
  uint32_t parts;
  uint32_t tokens, E, k;
  float balance_coef, z_coef;
};

// Four logits of one row, -infinity where there is no expert.
template <bool kVec>
__device__ __forceinline__ void load4(const float* row, uint32_t e0, uint32_t E, float (&v)[4]) {
  if (kVec) {
    typedef __attribute__((ext_vector_type(4))) float f32x4;
    f32x4 q = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (e0 < E) q = *reinterpret_cast<const f32x4*>(row + e0);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = q[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
  }
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Probabilities of a row (in place) and its logarithm of the sum of
// exponentials. A row of -infinity alone gives zeros; NaN stays NaN.
template <int L>
__device__ __forceinline__ float softmax_row(float (&v)[4]) {
  const float top = group_max<L>(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
  const float m = top == -INFINITY ? 0.f : top;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = expf(v[j] - m);
    s += v[j];
  }
  s = group_sum<L>(s);
  const float inv = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= inv;
  return s == 0.f ? 0.f : m + logf(s);
}

// The losses from whole sums; all threads of the workgroup (kThreads or more)
// call it, thread e holding expert e's sums. red: kThreads doubles.
__device__ __forceinline__ void finish(const BalanceArgs& a, double p, int c, double z, int n, double* red) {
  const uint32_t t = threadIdx.x;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  const double mean = p * inv;
  if (t < (uint32_t)kThreads) red[t] = t < a.E ? (double)c * mean : 0.0;
  __syncthreads();
  for (uint32_t m = kThreads / 2; m > 0; m >>= 1) {
    if (t < m) red[t] += red[t + m];
    __syncthreads();
  }
  if (t < a.E) {
    a.counts[t] = c;
    if (a.prob_mean) a.prob_mean[t] = (float)mean;
  }
  if (t == 0) {
    a.counts[a.E] = n;
    a.loss[0] = (float)((double)a.balance_coef * a.E * red[0] * inv / a.k);
    a.loss[1] = (float)((double)a.z_coef * z * inv);
  }
}

// Sums over the workgroup's tokens: probabilities per expert (fp32 per lane
// over its rows, then across lanes and waves in a fixed order), squared
// logarithms, tuples per expert (whole numbers, in LDS), valid tokens. With
// kLast the one workgroup writes the results, else its partial sums.
template <int L, bool kVec, bool kLast>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs a) {
  constexpr uint32_t G = kThreads / L;  // groups: rows of one pass
  __shared__ int s_cnt[kMaxBalanceExperts + 1];
  __shared__ float s_p[kThreads / 64][4 * L];
  __shared__ float s_z[kThreads / 64];
  __shared__ double s_red[kLast ? kThreads : 1];
  const uint32_t tid = threadIdx.x, lane = tid % L, grp = tid / L;
  for (uint32_t i = tid; i <= a.E; i += kThreads) s_cnt[i] = 0;
  __syncthreads();
  float p[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f;
  int n = 0;
  const uint32_t step = G * kRows;
  for (uint32_t t0 = blockIdx.x * step; t0 < a.tokens; t0 += gridDim.x * step) {
    const uint32_t here = min(step, a.tokens - t0);
    float v[kRows][4];
    bool ok[kRows];
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      const uint32_t t = t0 + u * G + grp;
      const uint32_t tc = min(t, a.tokens - 1);
      load4<kVec>(a.logits + (uint64_t)tc * a.E, lane * 4, a.E, v[u]);
      ok[u] = t < a.tokens && (!a.valid || a.valid[tc]);
    }
    for (uint32_t i = tid; i < here * a.k; i += kThreads) {
      const uint32_t t = t0 + i / a.k;
      const uint32_t e = (uint32_t)a.experts[(uint64_t)t0 * a.k + i];
      if (e < a.E && (!a.valid || a.valid[t])) atomicAdd(&s_cnt[e], 1);
    }
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      const float lse = softmax_row<L>(v[u]);
      if (ok[u]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] += v[u][j];
        if (lane == 0) {
          z = fmaf(lse, lse, z);
          ++n;
        }
      }
    }
  }
  if (n) atomicAdd(&s_cnt[a.E], n);
  // across the groups of a wave, then across waves
#pragma unroll
  for (int j = 0; j < 4; ++j)
    for (int m = L; m < 64; m <<= 1) p[j] += __shfl_xor(p[j], m);
  for (int m = 1; m < 64; m <<= 1) z += __shfl_xor(z, m);
  const uint32_t w = tid / 64, l = tid % 64;
  if (l < L)
#pragma unroll
    for (int j = 0; j < 4; ++j) s_p[w][l * 4 + j] = p[j];
  if (l == 0) s_z[w] = z;
  __syncthreads();
  float sp = 0.f, sz = 0.f;
  for (uint32_t i = 0; i < kThreads / 64; ++i) {
    if (tid < a.E) sp += s_p[i][tid];
    sz += s_z[i];
  }
  if (kLast) {
    finish(a, (double)sp, tid < a.E ? s_cnt[tid] : 0, (double)sz, s_cnt[a.E], s_red);
  } else {
    if (tid < a.E) a.part_p[blockIdx.x * a.E + tid] = sp;
    for (uint32_t i = tid; i <= a.E; i += kThreads) a.part_c[blockIdx.x * (a.E + 1) + i] = s_cnt[i];
    if (tid == 0) a.part_z[blockIdx.x] = sz;
  }
}

// Joins the partial sums: thread (r, e) adds every R-th partial of expert e
// in double, then the R slices are added in order.
__global__ __launch_bounds__(1024) void k_balance_join(BalanceArgs a) {
  __shared__ double s_p[1024];
  __shared__ int s_c[1024];
  __shared__ double s_z[kThreads];
  __shared__ int s_n[kThreads];
  __shared__ double s_red[kThreads];
  const uint32_t tid = threadIdx.x;
  const uint32_t W = a.E <= 64 ? 64 : 256, R = 1024 / W;
  const uint32_t e = tid % W, r = tid / W;
  double p = 0.0;
  int c = 0;
  if (e < a.E)
    for (uint32_t i = r; i < a.parts; i += R) {
      p += (double)a.part_p[i * a.E + e];
      c += a.part_c[i * (a.E + 1) + e];
    }
  s_p[tid] = p;
  s_c[tid] = c;
  if (tid < kThreads) {
    double z = 0.0;
    int n = 0;
    for (uint32_t i = tid; i < a.parts; i += kThreads) {
      z += (double)a.part_z[i];
      n += a.part_c[i * (a.E + 1) + a.E];
    }
    s_z[tid] = z;
    s_n[tid] = n;
  }
  __syncthreads();
  for (uint32_t m = kThreads / 2; m > 0; m >>= 1) {
    if (tid < m) {
      s_z[tid] += s_z[tid + m];
      s_n[tid] += s_n[tid + m];
    }
    __syncthreads();
  }
  p = 0.0;
  c = 0;
  if (tid < a.E)
    for (uint32_t i = 0; i < R; ++i) {
      p += s_p[i * W + tid];
      c += s_c[i * W + tid];
    }
  finish(a, p, c, s_z[0], s_n[0], s_red);
}

// The gradient of the logits, one row per group. The counts enter centred on
// their mean k n / E, a difference of whole numbers (the probabilities sum to one,
// so a common part has no gradient): nearly even loads lose nothing in
// c_e - sum_j c_j p_j.
template <int L, bool kVec>
__global__ __launch_bounds__(kThreads) void k_router_grad(BalanceArgs a) {
  constexpr uint32_t G = kThreads / L;
  const uint32_t tid = threadIdx.x, lane = tid % L, grp = tid / L;
  const int n = a.counts[a.E];
  const float inv = n > 0 ? 1.0f / (float)n : 0.f;
  const float u0 = a.grad_loss ? a.grad_loss[0] : 1.f, u1 = a.grad_loss ? a.grad_loss[1] : 1.f;
  const float cb = u0 * a.balance_coef * (float)a.E / (float)a.k * inv, cz = u1 * 2.f * a.z_coef * inv;
  float c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t e = lane * 4 + j;
    c[j] = e < a.E ? (float)((int64_t)a.counts[e] * a.E - (int64_t)a.k * n) * (inv / (float)a.E) : 0.f;
  }
  const uint32_t t = blockIdx.x * G + grp;
  if (t >= a.tokens) return;  // whole groups leave: the exchanges below stay inside a group
  float v[4];
  load4<kVec>(a.logits + (uint64_t)t * a.E, lane * 4, a.E, v);
  const bool ok = !a.valid || a.valid[t];
  const float lse = softmax_row<L>(v);
  const float mean = group_sum<L>(fmaf(c[0], v[0], fmaf(c[1], v[1], fmaf(c[2], v[2], c[3] * v[3]))));
  float o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = v[j] * fmaf(cb, c[j] - mean, cz * lse);
  if (a.gates) {
    const float* g = a.gates + (uint64_t)t * a.k;
    const float* dg = a.dgates + (uint64_t)t * a.k;
    const int32_t* ex = a.experts + (uint64_t)t * a.k;
    float dot = 0.f;
    for (uint32_t s = 0; s < a.k; ++s) dot = fmaf(g[s], dg[s], dot);
    for (uint32_t s = 0; s < a.k; ++s) {
      const uint32_t e = (uint32_t)ex[s] - lane * 4;
      const float part = g[s] * (dg[s] - dot);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (e == j) o[j] += part;
    }
  }
  float* out = a.dlogits + (uint64_t)t * a.E;
  if (kVec) {
    typedef __attribute__((ext_vector_type(4))) float f32x4;
    const f32x4 q = {ok ? o[0] : 0.f, ok ? o[1] : 0.f, ok ? o[2] : 0.f, ok ? o[3] : 0.f};
    if (lane * 4 < a.E) *reinterpret_cast<f32x4*>(out + lane * 4) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane * 4 + j < a.E) out[lane * 4 + j] = ok ? o[j] : 0.f;
  }
}

struct BalanceLayout {
  size_t p = 0, c = 0, z = 0, total = 0;
  uint32_t parts = 0;  // 1: one workgroup, no partial sums
};

int group_lanes(uint32_t E) { return E <= 16 ? 4 : E <= 64 ? 16 : 64; }

BalanceLayout balance_layout(const pw_balance_desc& d) {
  BalanceLayout l;
  const uint32_t rows = kThreads / group_lanes(d.num_experts) * kRows;
  const uint64_t blocks = (d.tokens + rows - 1) / rows;
  l.parts = d.tokens <= kAlone ? 1u : (uint32_t)std::min<uint64_t>(blocks, kParts);
  if (l.parts <= 1) return l;
  l.p = 0;
  l.c = up256((size_t)l.parts * d.num_experts * 4);
  l.z = l.c + up256((size_t)l.parts * (d.num_experts + 1) * 4);
  l.total = l.z + up256((size_t)l.parts * 4);
  return l;
}

int validate(const pw_balance_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->tokens > (1ull << 28)) return fail(PW_ERR_INVALID, "tokens must be at most 2^28");
  if (d->num_experts < 2 || d->num_experts > kMaxBalanceExperts)
    return fail(PW_ERR_INVALID, "num_experts must be in [2, %u]", kMaxBalanceExperts);
  if (d->top_k < 1 || d->top_k > 8 || d->top_k > d->num_experts)
    return fail(PW_ERR_INVALID, "top_k must be in [1, 8] and at most num_experts");
  if (d->tokens * d->top_k > 0x7fffffffull) return fail(PW_ERR_INVALID, "tokens x top_k must stay below 2^31");
  if (!isfinite(d->balance_coef) || !isfinite(d->z_coef)) return fail(PW_ERR_INVALID, "the coefficients must be finite");
  return PW_OK;
}

BalanceArgs args(const pw_balance_desc& d, const pw_balance_io& io) {
  BalanceArgs a{};
  a.logits = io.logits;
  a.experts = io.experts;
  a.valid = io.valid;
  a.counts = io.counts;
  a.prob_mean = io.prob_mean;
  a.loss = io.loss;
  a.gates = io.gates;
  a.dgates = io.dgates;
  a.grad_loss = io.grad_loss;
  a.dlogits = io.dlogits;
  a.tokens = (uint32_t)d.tokens;
  a.E = d.num_experts;
  a.k = d.top_k;
  a.balance_coef = d.balance_coef;
  a.z_coef = d.z_coef;
  return a;
}

template <int L, bool kVec>
void launch_balance(const BalanceArgs& a, hipStream_t s) {
  if (a.parts <= 1) {
    hipLaunchKernelGGL((k_balance<L, kVec, true>), dim3(1), dim3(kThreads), 0, s, a);
    return;
  }
  hipLaunchKernelGGL((k_balance<L, kVec, false>), dim3(a.parts), dim3(kThreads), 0, s, a);
}

template <int L, bool kVec>
void launch_grad(const BalanceArgs& a, hipStream_t s) {
  constexpr uint32_t G = kThreads / L;
  hipLaunchKernelGGL((k_router_grad<L, kVec>), dim3((a.tokens + G - 1) / G), dim3(kThreads), 0, s, a);
}

#define PW_BY_EXPERTS(fn, a, vec, s)                                \
  do {                                                              \
    const int lanes = group_lanes((a).E);                           \
    if (lanes == 4) (vec) ? fn<4, true>(a, s) : fn<4, false>(a, s); \
    else if (lanes == 16) (vec) ? fn<16, true>(a, s) : fn<16, false>(a, s); \
    else (vec) ? fn<64, true>(a, s) : fn<64, false>(a, s);          \
  } while (0)

}  // namespace

}  // namespace pw

using namespace pw;

extern "C" int pw_router_balance_workspace(const pw_balance_desc* d, size_t* bytes) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!bytes) return fail(PW_ERR_INVALID, "bytes is NULL");
  *bytes = balance_layout(*d).total;
  return PW_OK;
}

extern "C" int pw_router_balance(const pw_balance_desc* d, const pw_balance_io* io, void* ws, size_t ws_bytes,
                                 void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io || !io->counts || !io->loss) return fail(PW_ERR_INVALID, "counts and loss are required");
  if (d->tokens && (!io->logits || !io->experts)) return fail(PW_ERR_INVALID, "logits and experts are required");
  const BalanceLayout l = balance_layout(*d);
  if ((st = check_workspace(ws, ws_bytes, l.total))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  BalanceArgs a = args(*d, *io);
  unsigned char* base = static_cast<unsigned char*>(ws);
  a.parts = l.parts;
  if (l.parts > 1) {
    a.part_p = reinterpret_cast<float*>(base + l.p);
    a.part_c = reinterpret_cast<int32_t*>(base + l.c);
    a.part_z = reinterpret_cast<float*>(base + l.z);
  }
  const bool vec = a.E % 4 == 0 && (uintptr_t)a.logits % 16 == 0;
  PW_BY_EXPERTS(launch_balance, a, vec, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "launch balance");
  if (l.parts > 1) {
    hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(1024), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "launch balance_join");
  }
  return PW_OK;
}

extern "C" int pw_router_grad(const pw_balance_desc* d, const pw_balance_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->tokens == 0) return PW_OK;
  if (!io->logits || !io->counts || !io->dlogits) return fail(PW_ERR_INVALID, "logits, counts and dlogits are required");
  if (!io->gates != !io->dgates) return fail(PW_ERR_INVALID, "gates and dgates are given together or not at all");
  if (io->gates && !io->experts) return fail(PW_ERR_INVALID, "gates need experts");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const BalanceArgs a = args(*d, *io);
  const bool vec = a.E % 4 == 0 && ((uintptr_t)a.logits | (uintptr_t)a.dlogits) % 16 == 0;
  PW_BY_EXPERTS(launch_grad, a, vec, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch router_grad");
}
