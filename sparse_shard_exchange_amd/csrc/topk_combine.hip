// out[t] = add[t] + sum_j w[t][j] y[t][j]: the expert rows of each token, in
// tuple order, joined by their routing weights.
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
  uint32_t tokens, d, k;
};

template <typename T>
__global__ __launch_bounds__(kThreads) void k_topk_combine(CombineArgs a) {
  const T* y = static_cast<const T*>(a.y);
  const T* add = static_cast<const T*>(a.add);
  T* out = static_cast<T*>(a.out);
  for (uint64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    for (uint32_t c = threadIdx.x; c < a.d; c += kThreads) {
      float sum = add ? (float)add[t * a.d + c] : 0.0f;
      for (uint32_t j = 0; j < a.k; ++j) {
        const float w = a.weights[t * a.k + j];
        if (w != 0.0f) sum = fmaf(w, (float)y[(t * a.k + j) * a.d + c], sum);
      }
      out[t * a.d + c] = (T)sum;
    }
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
  CombineArgs a{io->y, io->weights, io->add, io->out, (uint32_t)d->tokens, d->d, d->top_k};
  const dim3 grid(std::min(a.tokens, kMaxGrid));
  if (d->dtype == PW_F32) hipLaunchKernelGGL(k_topk_combine<float>, grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(k_topk_combine<__bf16>, grid, dim3(kThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch topk_combine");
}
