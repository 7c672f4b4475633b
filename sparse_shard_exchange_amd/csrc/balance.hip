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
// are lane exchanges inside the group. 131072 x 64: loss 11.0 + 4.5 us (35 MB,
// 3.2 TB/s), gradient 15.6 us (70 MB, 4.5 TB/s). At this size a workgroup of the loss
// makes two passes, the second's loads behind the first's arithmetic, and the join
// is a launch's latency. 48 x 8: 4.1 us, a few memory latencies.
#include "ops.h"

#include <algorithm>

namespace pw {

namespace {

constexpr int kThreads = 1024;     // k_balance, its join
constexpr int kGradThreads = 256;  // k_router_grad
constexpr uint32_t kMaxBalanceExperts = 256;
constexpr int kRed = 256;          // threads of the loss' last sum: one per expert
constexpr uint32_t kParts = 256;        // partial sums at most: a workgroup of 16 waves per CU
// Rows of a group up to which one workgroup does all, in one launch (E = 64, 512
// tokens: 9.5 us against 10.7 for two launches; 1024 tokens: 16.0 against 10.7;
// E = 8 and 256 cross over at the same count of 8 rows).
constexpr uint32_t kAlone = 8;
constexpr uint32_t rows_of(bool last) { return last ? 2 : 4; }  // rows of a group of k_balance in flight
// Passes of a run of k_balance: a lane adds 256 rows, then that sum to its sum of
// the runs (256 at most, for 2^28 tokens), so that no chain has more than 512
// additions (2^25 equal tokens, 8192 rows a lane in one chain: probabilities off by
// 1.1e-4). 2^20 tokens take one run up to 256 experts, 2^22 up to 64.
constexpr uint32_t kRun = 64;
// Workgroups up to which k_router_grad takes one row a group (16000 x 64, 1000
// workgroups: 4.8 us against 5.1 with 4 rows; 32000 x 64: 6.9 against 6.6).
constexpr uint32_t kGradWide = 1024;

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
  uint2* part;      // [parts][E + 1] sums of probabilities (fp32 bits), tuples; last: squared logarithms, valid tokens
  uint32_t parts;
  uint32_t tokens, E, k;
  float balance_coef, z_coef;
};

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4), aligned(4))) float f32x4_at4;

// The first of a lane's four experts: 4 lane, or, where fewer than four are left
// (kFour, at least four experts), moved back to the row's last four, so that
// every row goes in 16-byte accesses (131072 x 61: loss 19.5 us with four loads
// a lane, logit gradient 22.1).
template <bool kFour>
__device__ __forceinline__ uint32_t first_of(uint32_t lane, uint32_t E) { return kFour ? min(lane * 4, E - 4) : lane * 4; }

// A lane's logits of one row from expert e0 on; -infinity where another lane
// has the expert, or there is none.
template <bool kFour>
__device__ __forceinline__ void load4(const float* row, uint32_t e0, uint32_t lane, uint32_t E, float (&v)[4]) {
  if (kFour) {
    const f32x4 q = *reinterpret_cast<const f32x4_at4*>(row + e0);
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) v[j] = e0 + j >= lane * 4 ? q[j] : -INFINITY;
  } else {
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) v[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
  }
}

// Whether a token counts, as a byte loaded without a branch (under one, the
// compiler waits for it before the next row's load: the loss of 131072 x 64 took
// 15.4 us). With no mask it reads a byte of the logits, which counts as nothing.
struct Mask {
  const uint8_t* p;
  uint32_t every, index;  // no mask: 1, 0; else 0, all ones
  __device__ __forceinline__ explicit Mask(const BalanceArgs& a)
      : p(a.valid ? a.valid : reinterpret_cast<const uint8_t*>(a.logits)), every(a.valid ? 0 : 1), index(every - 1) {}
  __device__ __forceinline__ uint32_t load(uint32_t t) const { return p[t & index]; }
  __device__ __forceinline__ bool has(uint32_t v) const { return v | every; }
};

// e^x for x <= 0 (and NaN): the hardware's 2^t with t = x log2(e), and what the
// product's rounding and log2(e)'s own left out put back to first order, so the
// result is off by the rounding of x and two units in the last place. 8
// instructions where expf takes 14; half of both kernels' arithmetic is this.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e430p-1f;
  x = x < -150.f ? -150.f : x;  // e^-150 is zero in fp32; keeps -infinity out of the rest
  const float t = x * kLog2e;
  const float rest = fmaf(x, kLog2e, -t) + x * kRest;
  const float y = __builtin_amdgcn_exp2f(t);
  return fmaf(y, rest * kLn2, y);
}

// Probabilities of a row (in place) and its logarithm of the sum of
// exponentials. A row of -infinity alone gives zeros; NaN stays NaN.
template <int L>
__device__ __forceinline__ float softmax_row(float (&v)[4]) {
  const float top = lanes_max<L>(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
  const float m = top == -INFINITY ? 0.f : top;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = exp_neg(v[j] - m);
    s += v[j];
  }
  s = lanes_sum<L>(s);
  const float inv = s == 0.f ? 0.f : __builtin_amdgcn_rcpf(s);  // s is in [1, E]: a unit in the last place
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= inv;
  return s == 0.f ? 0.f : fmaf(__builtin_amdgcn_logf(s), 0x1.62e430p-1f, m);  // log2(s) ln 2
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// The losses from whole sums; all threads of the workgroup call it, thread e
// holding expert e's sums. red: kRed / 64 doubles.
__device__ __forceinline__ void finish(const BalanceArgs& a, double p, int c, double z, int n, double* red) {
  const uint32_t t = threadIdx.x;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  const double mean = p * inv;
  if (t < (uint32_t)kRed) {  // whole waves
    const double s = wave_sum(t < a.E ? (double)c * mean : 0.0);
    if (t % 64 == 0) red[t / 64] = s;
  }
  __syncthreads();
  if (t < a.E) {
    a.counts[t] = c;
    if (a.prob_mean) a.prob_mean[t] = (float)mean;
  }
  if (t == 0) {
    double s = 0.0;
    for (int w = 0; w < kRed / 64; ++w) s += red[w];
    a.counts[a.E] = n;
    a.loss[0] = (float)((double)a.balance_coef * a.E * s * inv / a.k);
    a.loss[1] = a.z_coef == 0.f ? 0.f : (float)((double)a.z_coef * z * inv);  // (z may have overflowed)
  }
}

// Sums over the workgroup's tokens: probabilities per expert (fp32 per lane
// over its rows, in runs, then across lanes and waves in a fixed order), squared
// logarithms, tuples per expert (whole numbers, in LDS), valid tokens. With
// kLast the one workgroup writes the results, else its partial sums.
template <int L, bool kFour, bool kLast>
__global__ __launch_bounds__(kThreads) void k_balance(BalanceArgs a) {
  constexpr uint32_t G = kThreads / L, kRows = rows_of(kLast);  // groups: rows of one pass
  __shared__ int s_cnt[kMaxBalanceExperts + 1];
  __shared__ float s_p[kThreads / 64][4 * L];
  __shared__ float s_z[kThreads / 64];
  __shared__ double s_red[kRed / 64];
  const uint32_t tid = threadIdx.x, lane = tid % L, grp = tid / L, e0 = first_of<kFour>(lane, a.E);
  for (uint32_t i = tid; i <= a.E; i += kThreads) s_cnt[i] = 0;
  __syncthreads();
  const Mask mask(a);
  float p[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f;
  float runs_p[4] = {0.f, 0.f, 0.f, 0.f}, runs_z = 0.f;
  int n = 0;
  const uint32_t step = G * kRows;
  uint32_t pass = 0;
  for (uint32_t t0 = blockIdx.x * step; t0 < a.tokens; t0 += gridDim.x * step) {
    const uint32_t here = min(step, a.tokens - t0);
    float v[kRows][4];
    uint32_t ok[kRows];
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      const uint32_t t = min(t0 + u * G + grp, a.tokens - 1);
      load4<kFour>(a.logits + (uint64_t)t * a.E, e0, lane, a.E, v[u]);
      ok[u] = mask.load(t);
    }
    for (uint32_t i = tid; i < here * a.k; i += kThreads) {
      const uint32_t e = (uint32_t)a.experts[(uint64_t)t0 * a.k + i], in = mask.load(t0 + i / a.k);
      if ((e < a.E) & mask.has(in)) atomicAdd(&s_cnt[e], 1);
    }
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      const float lse = softmax_row<L>(v[u]);
      if (mask.has(ok[u]) && t0 + u * G + grp < a.tokens) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] += v[u][j];
        if (lane == 0) {
          z = fmaf(lse, lse, z);
          ++n;
        }
      }
    }
    if (!kLast && ++pass == kRun) {  // uniform; (kLast has kAlone rows a group at most)
      pass = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        runs_p[j] += p[j];
        p[j] = 0.f;
      }
      runs_z += z;
      z = 0.f;
    }
  }
  if (!kLast) {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] += runs_p[j];
    z += runs_z;
  }
  if (n) atomicAdd(&s_cnt[a.E], n);
  // across the groups of a wave, then across waves
#pragma unroll
  for (int j = 0; j < 4; ++j)
    for (int m = L; m < 64; m <<= 1) p[j] += __shfl_xor(p[j], m);
  z = lanes_sum<64>(z);
  const uint32_t w = tid / 64, l = tid % 64;
  if (l < L)
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (e0 + j >= l * 4) s_p[w][e0 + j] = p[j];
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
    uint2* part = a.part + (uint64_t)blockIdx.x * (a.E + 1);
    if (tid <= a.E) part[tid] = uint2{__builtin_bit_cast(uint32_t, tid < a.E ? sp : sz), (uint32_t)s_cnt[tid]};
  }
}

// Joins the partial sums: thread (r, e) adds every R-th partial of column e,
// then the R slices are added in order; the last column goes to 16 threads.
// 16 loads of a thread in flight and no branch between them: the kernel is a
// few memory latencies long, whatever it adds.
__device__ __forceinline__ void add_parts(const BalanceArgs& a, uint32_t e, uint32_t i0, uint32_t step, float& p, int& c) {
  uint2 v[16];
#pragma unroll
  for (uint32_t q = 0; q < 16; ++q) v[q] = a.part[min(i0 + q * step, a.parts - 1) * (a.E + 1) + e];
#pragma unroll
  for (uint32_t q = 0; q < 16; ++q) {
    const bool in = i0 + q * step < a.parts;
    p += in ? __builtin_bit_cast(float, v[q].x) : 0.f;
    c += in ? (int)v[q].y : 0;
  }
}

__global__ __launch_bounds__(kThreads) void k_balance_join(BalanceArgs a) {
  static_assert(kParts == 256, "16 slices of 16 partial sums, or 4 of 64");
  __shared__ float s_p[kThreads], s_z[16];
  __shared__ int s_c[kThreads], s_n[16];
  __shared__ double s_red[kRed / 64];
  const uint32_t tid = threadIdx.x, W = a.E <= 64 ? 64 : 256, R = kThreads / W;
  float p = 0.f;
  int c = 0;
  for (uint32_t i = 0; i < kParts / R; i += 16) add_parts(a, min(tid % W, a.E), tid / W + i * R, R, p, c);
  s_p[tid] = p;
  s_c[tid] = c;
  if (tid < 16) {
    p = 0.f;
    c = 0;
    add_parts(a, a.E, tid, 16, p, c);
    s_z[tid] = p;
    s_n[tid] = c;
  }
  __syncthreads();
  double sum = 0.0, z = 0.0;
  int count = 0, n = 0;
  if (tid < a.E)
    for (uint32_t i = 0; i < R; ++i) {
      sum += (double)s_p[i * W + tid];
      count += s_c[i * W + tid];
    }
  for (uint32_t i = 0; i < 16; ++i) {
    z += (double)s_z[i];
    n += s_n[i];
  }
  finish(a, sum, count, z, n, s_red);
}

// The gradient of the logits, kRows rows per group in flight. The counts enter centred on
// their mean k n / E, a difference of whole numbers (the probabilities sum to
// one, so a common part has no gradient): nearly even loads lose nothing in
// c_e - sum_j c_j p_j. A row's gates are loaded by its group's first k lanes (two
// each where there are 4 lanes) and handed round, picked by constant indices: an
// array that is indexed at run time goes to LDS (131072 x 8: 20 us against 6).
template <int L, bool kFour, uint32_t kRows>
__global__ __launch_bounds__(kGradThreads) void k_router_grad(BalanceArgs a) {
  constexpr uint32_t G = kGradThreads / L, S = L < 8 ? L : 8;  // lanes that hold gates
  constexpr uint32_t kOf = 8 / S;                              // gates of such a lane
  const uint32_t tid = threadIdx.x, lane = tid % L, grp = tid / L, e0 = first_of<kFour>(lane, a.E);
  const Mask mask(a);
  for (uint32_t t0 = blockIdx.x * G * kRows + grp; t0 - grp < a.tokens; t0 += gridDim.x * G * kRows) {
    float v[kRows][4], g[kRows][kOf], dg[kRows][kOf];
    uint32_t ex[kRows][kOf], ok[kRows];
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      const uint32_t t = min(t0 + u * G, a.tokens - 1);
      load4<kFour>(a.logits + (uint64_t)t * a.E, e0, lane, a.E, v[u]);
      ok[u] = mask.load(t);
    }
    if (a.gates)  // uniform
#pragma unroll
      for (uint32_t u = 0; u < kRows; ++u)
#pragma unroll
        for (uint32_t q = 0; q < kOf; ++q) {
          const uint64_t o = (uint64_t)min(t0 + u * G, a.tokens - 1) * a.k + min(lane * kOf + q, a.k - 1);
          g[u][q] = a.gates[o];
          dg[u][q] = a.dgates[o];
          ex[u][q] = (uint32_t)a.experts[o];
        }
    // all without branches, so that one wait covers these and the rows
    const int n = a.counts[a.E];
    const float* up = a.grad_loss ? a.grad_loss : reinterpret_cast<const float*>(a.counts);  // (then not used)
    const float up0 = up[0], up1 = up[1];
    int count[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) count[j] = a.counts[min(e0 + j, a.E)];
    const float inv = n > 0 ? 1.0f / (float)n : 0.f;
    const float u0 = a.grad_loss ? up0 : 1.f, u1 = a.grad_loss ? up1 : 1.f;
    const float cb = u0 * a.balance_coef * (float)a.E / (float)a.k * inv, cz = u1 * 2.f * a.z_coef * inv;
    float c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t e = e0 + j;
      c[j] = e < a.E ? (float)((int64_t)count[j] * a.E - (int64_t)a.k * n) * (inv / (float)a.E) : 0.f;
    }
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      const uint32_t t = t0 + u * G;
      const float lse = softmax_row<L>(v[u]);
      const float mean = lanes_sum<L>(fmaf(c[0], v[u][0], fmaf(c[1], v[u][1], fmaf(c[2], v[u][2], c[3] * v[u][3]))));
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = v[u][j] * fmaf(cb, c[j] - mean, cz * lse);
      if (a.gates) {  // uniform
        float dot = 0.f, part[kOf];
#pragma unroll
        for (uint32_t q = 0; q < kOf; ++q)
          if (lane * kOf + q < a.k) dot = fmaf(g[u][q], dg[u][q], dot);
        dot = lanes_sum<S>(dot);
#pragma unroll
        for (uint32_t q = 0; q < kOf; ++q) part[q] = g[u][q] * (dg[u][q] - dot);
        for (uint32_t s = 0; s < a.k; s += kOf) {
          const int from = (int)(tid % 64 - lane + s / kOf);
#pragma unroll
          for (uint32_t q = 0; q < kOf; ++q) {
            const float p = __shfl(s + q < a.k ? part[q] : 0.f, from);
            const uint32_t e = (uint32_t)__shfl((int)ex[u][q], from) - e0;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
              if (e == j) o[j] += p;
          }
        }
      }
      if (t >= a.tokens) continue;
      float* out = a.dlogits + (uint64_t)t * a.E;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = mask.has(ok[u]) ? o[j] : 0.f;
      if (kFour && e0 == lane * 4) {
        *reinterpret_cast<f32x4_at4*>(out + e0) = f32x4{o[0], o[1], o[2], o[3]};
      } else {
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
          if (e0 + j >= lane * 4 && e0 + j < a.E) out[e0 + j] = o[j];
      }
    }
  }
}

struct BalanceLayout {
  size_t total = 0;
  uint32_t parts = 0;  // 1: one workgroup, no partial sums
};

int group_lanes(uint32_t E) { return E <= 16 ? 4 : E <= 64 ? 16 : 64; }

BalanceLayout balance_layout(const pw_balance_desc& d) {
  BalanceLayout l;
  const uint32_t G = kThreads / group_lanes(d.num_experts), rows = G * rows_of(false);
  const uint64_t blocks = (d.tokens + rows - 1) / rows;
  l.parts = d.tokens <= kAlone * G ? 1u : (uint32_t)std::min<uint64_t>(blocks, kParts);
  if (l.parts > 1) l.total = up256((size_t)l.parts * (d.num_experts + 1) * sizeof(uint2));
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

int check_aligned(const pw_balance_io& io) {
  if (misaligned({io.logits, io.experts, io.counts, io.prob_mean, io.loss, io.gates, io.dgates, io.grad_loss,
                  io.dlogits}, 4))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
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

template <int L, bool kFour>
void launch_balance(const BalanceArgs& a, hipStream_t s) {
  if (a.parts <= 1) {
    hipLaunchKernelGGL((k_balance<L, kFour, true>), dim3(1), dim3(kThreads), 0, s, a);
    return;
  }
  hipLaunchKernelGGL((k_balance<L, kFour, false>), dim3(a.parts), dim3(kThreads), 0, s, a);
}

template <int L, bool kFour>
void launch_grad(const BalanceArgs& a, hipStream_t s) {
  constexpr uint32_t G = kGradThreads / L;
  const uint32_t groups = (a.tokens + G - 1) / G;
  if (groups <= kGradWide) hipLaunchKernelGGL((k_router_grad<L, kFour, 1>), dim3(groups), dim3(kGradThreads), 0, s, a);
  else hipLaunchKernelGGL((k_router_grad<L, kFour, 4>), dim3(std::min((groups + 3) / 4, kMaxGrid)), dim3(kGradThreads), 0, s, a);
}

#define PW_BY_EXPERTS(fn, a, s)                          \
  do {                                                   \
    const int lanes = group_lanes((a).E);                \
    if (lanes == 4) (a).E < 4 ? fn<4, false>(a, s) : fn<4, true>(a, s); \
    else if (lanes == 16) fn<16, true>(a, s);            \
    else fn<64, true>(a, s);                             \
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
  if ((st = check_aligned(*io))) return st;
  const BalanceLayout l = balance_layout(*d);
  if ((st = check_workspace(ws, ws_bytes, l.total))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  BalanceArgs a = args(*d, *io);
  a.parts = l.parts;
  a.part = static_cast<uint2*>(ws);
  PW_BY_EXPERTS(launch_balance, a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, "launch balance");
  if (l.parts > 1) {
    hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(kThreads), 0, s, a);
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
  if ((st = check_aligned(*io))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const BalanceArgs a = args(*d, *io);
  PW_BY_EXPERTS(launch_grad, a, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch router_grad");
}
