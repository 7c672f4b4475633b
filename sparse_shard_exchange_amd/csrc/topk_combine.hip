// out[t] = add[t] + sum_j w[t][j] y[t][j]: the expert rows of each token, in
// tuple order, joined by their routing weights. Bound by memory: every row of y is
// read once and past the caches (nothing reads it again), every row of out written so.
#include "ops.h"

#include <algorithm>

namespace pw {

namespace {

constexpr int kThreads = 256;

struct CombineArgs {
  const void* y;
  const float* weights;
  const void* add;
  void* out;
  uint32_t tokens, d;
};

// Sixteen bytes of a row, or one element; At: in memory, aligned to its elements.
template <typename T, int V>
struct Chunk {
  typedef T Vec __attribute__((ext_vector_type(V)));
  typedef T At __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};

// L lanes a token, K rows of y in flight a lane. The last chunk of a row is moved
// back to end with it and stores its own elements alone (out may be add). A row of
// weight 0 is not read: its lanes read the buffer's first row instead, a line
// that is in the caches, since loads under a branch would wait one for another.
// bf16 with add, d = 1024: 131072 tokens of 6 in 343 us, a tenth of the tokens masked (2.0 GB
// moved, 5.8 TB/s; a large copy reaches 5.1). Nontemporal neither way / stores only / both,
// without add: 131072 x 6 x 1024 381 / 362 / 304 us, 131072 x 2 x 1024 136 / 133 / 121, 16384 x 2 x 4096 70 / 57 / 63.
template <typename T, int V, int L, int K>
__global__ __launch_bounds__(kThreads) void k_topk_combine(CombineArgs a) {
  typedef Chunk<T, V> C;
  constexpr int kTeams = kThreads / L;
  const uint32_t lane = threadIdx.x % L, team = threadIdx.x / L;
  const T* y = static_cast<const T*>(a.y);
  const T* add = static_cast<const T*>(a.add);
  T* out = static_cast<T*>(a.out);
  const uint32_t chunks = (a.d + V - 1) / V;
  for (uint64_t t = (uint64_t)blockIdx.x * kTeams + team; t < a.tokens; t += (uint64_t)gridDim.x * kTeams) {
    float w[K];
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = a.weights[t * K + j];
    for (uint32_t c = lane; c < chunks; c += L) {
      const uint32_t at = min(c * V, a.d - V), over = c * V - at;  // over: elements of the chunk before
      typename C::Vec v[K], r = {};
#pragma unroll
      for (int j = 0; j < K; ++j)
        v[j] = __builtin_nontemporal_load(
            reinterpret_cast<const typename C::At*>(y + (w[j] != 0.0f ? (t * K + j) * a.d + at : 0)));
      if (add) r = *reinterpret_cast<const typename C::At*>(add + t * a.d + at);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float sum = (float)r[e];
#pragma unroll
        for (int j = 0; j < K; ++j) sum = w[j] != 0.0f ? fmaf(w[j], (float)v[j][e], sum) : sum;
        r[e] = (T)sum;
      }
      T* to = out + t * a.d + at;
      if (over == 0) {
        __builtin_nontemporal_store(r, reinterpret_cast<typename C::At*>(to));
      } else {
#pragma unroll
        for (int e = 1; e < V; ++e)
          if ((uint32_t)e >= over) to[e] = r[e];
      }
    }
  }
}

template <typename T, int V, int L, int K>
void launch(const CombineArgs& a, hipStream_t s) {
  constexpr uint32_t kTeams = kThreads / L;
  hipLaunchKernelGGL((k_topk_combine<T, V, L, K>), dim3(std::min((a.tokens + kTeams - 1) / kTeams, kMaxGrid)), dim3(kThreads),
                     0, s, a);
}

// Lanes a token: a row in one turn of 16-byte chunks, up to a workgroup. K is a
// constant so that a lane's rows are all in registers, on their way at once.
template <typename T, int K>
void launch_width(const CombineArgs& a, hipStream_t s) {
  constexpr uint32_t V = 16 / sizeof(T);
  if (a.d < V) launch<T, 1, 8, K>(a, s);
  else if (a.d <= 16 * V) launch<T, V, 16, K>(a, s);
  else if (a.d <= 64 * V) launch<T, V, 64, K>(a, s);
  else if (a.d <= 128 * V) launch<T, V, 128, K>(a, s);
  else launch<T, V, 256, K>(a, s);
}

template <typename T>
void launch_combine(const CombineArgs& a, uint32_t k, hipStream_t s) {
  switch (k) {
    case 1: return launch_width<T, 1>(a, s);
    case 2: return launch_width<T, 2>(a, s);
    case 3: return launch_width<T, 3>(a, s);
    case 4: return launch_width<T, 4>(a, s);
    case 5: return launch_width<T, 5>(a, s);
    case 6: return launch_width<T, 6>(a, s);
    case 7: return launch_width<T, 7>(a, s);
    default: return launch_width<T, 8>(a, s);
  }
}

int validate(const pw_combine_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->tokens > 0x7fffffffull) return fail(PW_ERR_INVALID, "tokens must be at most 2^31 - 1");
  if (d->d < 1 || d->d > 65536) return fail(PW_ERR_INVALID, "d must be in [1, 65536]");
  if (d->top_k < 1 || d->top_k > 8) return fail(PW_ERR_INVALID, "top_k must be in [1, 8]");
  if (d->dtype != PW_F32 && d->dtype != PW_BF16) return fail(PW_ERR_INVALID, "unknown dtype %u", d->dtype);
  return PW_OK;
}

}  // namespace

}  // namespace pw

using namespace pw;

extern "C" int pw_topk_combine(const pw_combine_desc* d, const pw_topk_combine_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->tokens == 0) return PW_OK;
  if (!io->y || !io->weights || !io->out) return fail(PW_ERR_INVALID, "y, weights and out are required");
  if (misaligned({io->y, io->add, io->out}, d->dtype == PW_F32 ? 4 : 2) || misaligned({io->weights}, 4))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const CombineArgs a{io->y, io->weights, io->add, io->out, (uint32_t)d->tokens, d->d};
  if (d->dtype == PW_F32) launch_combine<float>(a, d->top_k, s);
  else launch_combine<__bf16>(a, d->top_k, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch topk_combine");
}
