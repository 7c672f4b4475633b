// Products of an expert's rows in 8-bit integers: rows as codes with a scale
// each, and the matrix product of codes by expert segments.
//
//   s_t = max |x_t| / 127,  q = rint(x / s)
//   out = act(s_t ws_en sum_k q_tk w_enk)
#include "ops.h"

#include <float.h>

#include <algorithm>

#include "gemm.h"

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxWidth = 65536, kMaxQ8Experts = 256;

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(16))) int i32x16;

// ---- rows as codes -----------------------------------------------------------

struct QuantArgs {
  const void* x;
  const int64_t* limit;
  int8_t* q;
  float* scale;
  uint32_t rows, d, stride;
};

// The largest |x| as bits: NaN and infinity are the largest of all.
__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

template <typename T>
__global__ __launch_bounds__(kThreads) void k_quant_rows(QuantArgs a) {
  __shared__ uint32_t s_top[kThreads / 64];
  const int64_t limit = a.limit ? *a.limit : (int64_t)a.rows;
  const uint32_t rows = limit < 0 ? 0u : limit < (int64_t)a.rows ? (uint32_t)limit : a.rows;
  for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + r * a.d;
    uint32_t top = 0;
    for (uint32_t c = threadIdx.x; c < a.d; c += kThreads) top = max(top, magnitude((float)x[c]));
    for (int m = 1; m < 64; m *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    __syncthreads();
    if (threadIdx.x % 64 == 0) s_top[threadIdx.x / 64] = top;
    __syncthreads();
    top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    const float scale = top < 0x7f800000u ? __builtin_bit_cast(float, top) / 127.0f : NAN;
    const bool some = scale > 0.0f;
    for (uint32_t c = threadIdx.x; c < a.stride; c += kThreads) {
      float q = 0.0f;
      if (some && c < a.d) q = fminf(fmaxf(rintf((float)x[c] / scale), -127.0f), 127.0f);
      a.q[r * a.stride + c] = (int8_t)q;
    }
    if (threadIdx.x == 0) a.scale[r] = scale;
  }
}

hipError_t launch_quant(const QuantArgs& a, bool f32, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const dim3 grid(std::min(a.rows, kMaxGrid));
  if (f32) hipLaunchKernelGGL(k_quant_rows<float>, grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(k_quant_rows<__bf16>, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

// ---- products ----------------------------------------------------------------

struct Q8Args {
  const int8_t* q;
  const float* q_scale;
  const int8_t* w;
  const float* w_scale;
  const int64_t* offsets;    // or null: one expert, every row
  const int32_t* src_index;  // or null
  void* out;
  uint64_t tiles;
  uint32_t tuples;           // ids of src_index are below this
  uint32_t rows, n, E, stride;
  uint32_t gather;           // tuples of a row of q; 0: dispatched order
  uint32_t scatter;
  uint32_t col_tiles;
};

// Where a workgroup works: `rows` rows from row0 on, of expert e.
struct Segment {
  uint32_t e, row0, rows;
};

// The rb-th block of at most M rows, blocks counted over the experts' segments
// in turn; rows == 0: there is none. Every lane of the wave takes part.
template <uint32_t M>
__device__ __forceinline__ Segment segment_of(const Q8Args& a, uint32_t rb) {
  if (!a.offsets) {
    const uint32_t row0 = rb * M;
    return {0, row0, row0 < a.rows ? min(M, a.rows - row0) : 0u};
  }
  const uint32_t lane = threadIdx.x & 63;
  uint32_t done = 0, from = 0;  // blocks and rows of the experts before
  for (uint32_t e0 = 0; e0 < a.E; e0 += 64) {
    // where the lane's expert ends, and where the one before it did
    const uint32_t e = e0 + lane;
    if (e0 == 0) from = (uint32_t)min(max(a.offsets[0], (int64_t)0), (int64_t)a.rows);
    uint32_t end = (uint32_t)min(max(a.offsets[min(e + 1, a.E)], (int64_t)0), (int64_t)a.rows);
    end = max(end, from);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) end = max(end, (uint32_t)__shfl_up((int)end, m));  // a lane too low keeps its own
    uint32_t begin = (uint32_t)__shfl_up((int)end, 1);
    if (lane == 0) begin = from;
    const uint32_t blocks = (end - begin + M - 1) / M;
    uint32_t upto = blocks;  // blocks of this expert and those before it
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const uint32_t o = (uint32_t)__shfl_up((int)upto, m);
      if ((int)lane >= m) upto += o;
    }
    const uint64_t has = __ballot(rb < done + upto);
    if (has) {
      const int at = __builtin_ctzll(has);
      const uint32_t first = done + (uint32_t)__builtin_amdgcn_readlane((int)(upto - blocks), at);
      const uint32_t row0 = (uint32_t)__builtin_amdgcn_readlane((int)begin, at) + (rb - first) * M;
      return {e0 + (uint32_t)at, row0, min(M, (uint32_t)__builtin_amdgcn_readlane((int)end, at) - row0)};
    }
    done += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    from = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
  }
  return {0, 0, 0};
}

// Row of q that dispatched row i multiplies, and row of out that it gives (-1: none).
struct RowOf {
  uint32_t in;
  int64_t out;
};
__device__ __forceinline__ RowOf row_of(const Q8Args& a, uint32_t i) {
  if (!a.src_index) return {i, (int64_t)i};
  const int32_t g = a.src_index[i];
  if (g < 0 || (uint32_t)g >= a.tuples) return {0, -1};
  return {a.gather ? (uint32_t)g / a.gather : i, a.scatter ? (int64_t)g : (int64_t)i};
}

// bf16 results take the GELU of gemm.h (5.1e-5 of its value off, a seventieth of
// the rounding that follows), fp32 ones the library's error function.
template <typename T, bool kGelu>
__device__ __forceinline__ float finish(int sum, float s, float ws) {
  const float z = (float)sum * s * ws;
  if constexpr (!kGelu) return z;
  else if constexpr (sizeof(T) == 2) return mm::gelu(z);
  else return 0.5f * z * erfcf(z * -0.70710678f);
}

constexpr int kTile = 64, kStep = 64;

// One 64 x 64 tile a workgroup: operands through LDS in steps of 64 bytes, wave
// w the rows from 16 w on.
template <typename T, bool kGelu>
__global__ __launch_bounds__(kThreads) void k_q8_product(Q8Args a) {
  __shared__ __attribute__((aligned(16))) int8_t s_a[kTile][kStep + 16], s_b[kTile][kStep + 16];
  __shared__ float s_scale[kTile];
  __shared__ int64_t s_out[kTile];
  for (uint64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const Segment g = segment_of<kTile>(a, (uint32_t)(tile / a.col_tiles));
    if (g.rows == 0) return;  // nor is there a later one
    const uint32_t col0 = (uint32_t)(tile % a.col_tiles) * kTile;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const uint32_t ra = tid / 4, chunk = tid % 4 * 16;
    const RowOf row = row_of(a, g.row0 + min(ra, g.rows - 1));
    __syncthreads();
    if (tid % 4 == 0) {
      s_scale[ra] = a.q_scale[row.in];
      s_out[ra] = ra < g.rows ? row.out : -1;
    }
    const int8_t* pa = a.q + (uint64_t)row.in * a.stride + chunk;
    const int8_t* pb = a.w + ((uint64_t)g.e * a.n + min(col0 + ra, a.n - 1)) * a.stride + chunk;
    i32x4 acc[4] = {};
    for (uint32_t k = 0; k < a.stride; k += kStep) {
      __syncthreads();
      *reinterpret_cast<i32x4*>(&s_a[ra][chunk]) = *reinterpret_cast<const i32x4*>(pa + k);
      *reinterpret_cast<i32x4*>(&s_b[ra][chunk]) = *reinterpret_cast<const i32x4*>(pb + k);
      __syncthreads();
      const i32x4 x = *reinterpret_cast<const i32x4*>(&s_a[16 * w + lane % 16][lane / 16 * 16]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const i32x4 y = *reinterpret_cast<const i32x4*>(&s_b[16 * j + lane % 16][lane / 16 * 16]);
        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(y, x, acc[j], 0, 0, 0);
      }
    }
    // the lane holds 4 columns from 16 j + 4 (lane / 16) on of row 16 w + lane % 16
    const int r = 16 * w + lane % 16;
    const int64_t o = s_out[r];
    if (o < 0) continue;
    const float s = s_scale[r];
    T* out = static_cast<T*>(a.out) + (uint64_t)o * a.n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t c = col0 + 16 * j + 4 * (lane / 16) + v;
        if (c < a.n) out[c] = (T)finish<T, kGelu>(acc[j][v], s, a.w_scale[(uint64_t)g.e * a.n + c]);
      }
  }
}

template <typename T, bool kGelu>
hipError_t launch_product(Q8Args a, hipStream_t s) {
  a.col_tiles = (a.n + kTile - 1) / kTile;
  const uint64_t full = (a.rows + kTile - 1) / kTile;
  const uint64_t blocks = a.offsets ? std::min<uint64_t>(a.rows, a.rows / kTile + a.E) : full;
  a.tiles = blocks * a.col_tiles;
  hipLaunchKernelGGL((k_q8_product<T, kGelu>), dim3((uint32_t)std::min<uint64_t>(a.tiles, kMaxGrid)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

// ---- host --------------------------------------------------------------------

int validate(const pw_quant_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->rows > 0x7fffffffull) return fail(PW_ERR_INVALID, "rows must be at most 2^31 - 1");
  if (d->d < 1 || d->d > kMaxWidth) return fail(PW_ERR_INVALID, "d must be in [1, %u]", kMaxWidth);
  if (d->dtype != PW_F32 && d->dtype != PW_BF16) return fail(PW_ERR_INVALID, "unknown dtype %u", d->dtype);
  return PW_OK;
}

int validate(const pw_q8_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->rows > 0x7fffffffull || d->x_rows > 0x7fffffffull)
    return fail(PW_ERR_INVALID, "rows and x_rows must be at most 2^31 - 1");
  if (d->d < 1 || d->d > kMaxWidth || d->n < 1 || d->n > kMaxWidth)
    return fail(PW_ERR_INVALID, "d and n must be in [1, %u]", kMaxWidth);
  if (d->num_experts < 1 || d->num_experts > kMaxQ8Experts)
    return fail(PW_ERR_INVALID, "num_experts must be in [1, %u]", kMaxQ8Experts);
  if (d->dtype != PW_F32 && d->dtype != PW_BF16) return fail(PW_ERR_INVALID, "unknown dtype %u", d->dtype);
  if (d->gather > 256) return fail(PW_ERR_INVALID, "gather must be at most 256");
  if (d->scatter > 1 || d->gelu > 1) return fail(PW_ERR_INVALID, "scatter and gelu must be 0 or 1");
  if (!d->gather && d->x_rows < d->rows) return fail(PW_ERR_INVALID, "x_rows must be at least rows (no gather)");
  if (d->gather && d->rows && !d->x_rows) return fail(PW_ERR_INVALID, "rows to gather, but x has none");
  return PW_OK;
}

size_t product_workspace(const pw_q8_desc& d) {
  return up256(d.x_rows * PW_Q8_ROW(d.d)) + up256(d.x_rows * sizeof(float));
}

}  // namespace

}  // namespace pw

using namespace pw;

extern "C" int pw_quant_rows(const pw_quant_desc* d, const pw_quant_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->rows == 0) return PW_OK;
  if (!io->x || !io->q || !io->scale) return fail(PW_ERR_INVALID, "x, q and scale are required");
  if (misaligned({io->x}, d->dtype == PW_F32 ? 4 : 2) || misaligned({io->scale}, 4) || misaligned({io->limit}, 8))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
  if (misaligned({io->q}, 16)) return fail(PW_ERR_INVALID, "q must be 16-byte aligned");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const QuantArgs a{io->x, io->limit, io->q, io->scale, (uint32_t)d->rows, d->d, (uint32_t)PW_Q8_ROW(d->d)};
  const hipError_t e = launch_quant(a, d->dtype == PW_F32, s);
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch quant_rows");
}

extern "C" int pw_q8_product_workspace(const pw_q8_desc* d, size_t* bytes) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!bytes) return fail(PW_ERR_INVALID, "bytes is NULL");
  *bytes = product_workspace(*d);
  return PW_OK;
}

extern "C" int pw_q8_product(const pw_q8_desc* d, const pw_q8_io* io, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->rows == 0) return PW_OK;
  if (!io->w || !io->w_scale || !io->out) return fail(PW_ERR_INVALID, "w, w_scale and out are required");
  if (!io->x == !io->q || !io->q != !io->q_scale) return fail(PW_ERR_INVALID, "either x, or q with q_scale, is required");
  if (!io->offsets && d->num_experts != 1) return fail(PW_ERR_INVALID, "several experts need offsets");
  if (!io->src_index != (!d->gather && !d->scatter))
    return fail(PW_ERR_INVALID, "src_index is given with gather or scatter, and only then");
  if (misaligned({io->x, io->out}, d->dtype == PW_F32 ? 4 : 2) ||
      misaligned({io->q_scale, io->w_scale, io->src_index}, 4) || misaligned({io->offsets}, 8))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
  if (misaligned({io->q, io->w}, 16)) return fail(PW_ERR_INVALID, "codes must be 16-byte aligned");
  if (io->x && (st = check_workspace(ws, ws_bytes, product_workspace(*d)))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  Q8Args a{};
  a.q = io->q;
  a.q_scale = io->q_scale;
  a.w = io->w;
  a.w_scale = io->w_scale;
  a.offsets = io->offsets;
  a.src_index = io->src_index;
  a.out = io->out;
  a.rows = (uint32_t)d->rows;
  uint64_t tuples = d->gather ? d->x_rows * d->gather : d->rows;
  if (d->scatter) tuples = std::min(tuples, d->rows);
  a.tuples = (uint32_t)std::min<uint64_t>(tuples, 1u << 31);
  a.n = d->n;
  a.E = d->num_experts;
  a.stride = (uint32_t)PW_Q8_ROW(d->d);
  a.gather = d->gather;
  a.scatter = d->scatter;
  hipError_t e;
  if (io->x) {
    int8_t* q = static_cast<int8_t*>(ws);
    float* scale = reinterpret_cast<float*>(q + up256(d->x_rows * a.stride));
    // rows behind the last segment are not looked at
    const QuantArgs qa{io->x, d->gather ? nullptr : io->offsets ? io->offsets + a.E : nullptr, q, scale,
                       (uint32_t)d->x_rows, d->d, a.stride};
    if ((e = launch_quant(qa, d->dtype == PW_F32, s)) != hipSuccess) return hip_fail(e, "launch quant_rows");
    a.q = q;
    a.q_scale = scale;
  }
  if (d->dtype == PW_F32) e = d->gelu ? launch_product<float, true>(a, s) : launch_product<float, false>(a, s);
  else e = d->gelu ? launch_product<__bf16, true>(a, s) : launch_product<__bf16, false>(a, s);
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch q8_product");
}
