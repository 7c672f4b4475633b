// Products of an expert's rows in 8-bit integers: rows as codes with a scale
// each, and the matrix product of codes by expert segments.
//
//   s_t = max |x_t| fp32(1 / 127),  q = rint(fp32(x / s))
//   out = act(s_t ws_en sum_k q_tk w_enk)
//
// The sum is of whole numbers and exact in 32 bits (127^2 65536 < 2^31), in any
// order, so every shape below gives the same bits. Many rows an expert: bound by the
// matrix instructions (v_mfma_i32_32x32x32_i8; a library product of 8192^3 reaches
// 2.08 P operations/s here); few: by reading the weights once, from memory
// (5.7 TB/s once they stream, 4.0 to 4.5 with the start and end of a call).
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

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) float f32x8;
typedef __attribute__((ext_vector_type(8))) uint16_t u16x8;
typedef __attribute__((ext_vector_type(8))) uint32_t u32x8;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// Eight elements of a row, as loaded; At: in memory, aligned to its elements.
template <typename T>
struct Eight;
template <>
struct Eight<__bf16> {
  typedef __attribute__((ext_vector_type(8), aligned(2))) __bf16 At;
  typedef bf16x8 Vec;
  // the largest magnitude as the bits of an fp32 number: NaN and infinity are the largest of all
  static __device__ __forceinline__ uint32_t top(const Vec& v) {
    const u16x8 m = __builtin_bit_cast(u16x8, v) & (uint16_t)0x7fff;
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
    const u16x2 a = __builtin_elementwise_max(m.s01, m.s23), b = __builtin_elementwise_max(m.s45, m.s67);
    const u16x2 c = __builtin_elementwise_max(a, b);
    return (uint32_t)max(c.x, c.y) << 16;
  }
};
template <>
struct Eight<float> {
  typedef __attribute__((ext_vector_type(8), aligned(4))) float At;
  typedef f32x8 Vec;
  static __device__ __forceinline__ uint32_t top(const Vec& v) {
    const u32x8 m = __builtin_bit_cast(u32x8, v) & 0x7fffffffu;
    return max(max(max(m.s0, m.s1), max(m.s2, m.s3)), max(max(m.s4, m.s5), max(m.s6, m.s7)));
  }
};

// Eight codes. x / s as fp32 rounds it, without a division: with r = 1 / s
// correctly rounded, q + r (x - q s) is within an ulp of x / s after one step
// from q = x r, and the correctly rounded quotient after another (Markstein's
// theorem on division by a correctly rounded reciprocal; the remainders are exact
// where nothing leaves the normal numbers, so for s from 2^-100 to 2^100:
// quotients below 1/4, whose remainders might, are 0 either way). 1.5 x 2^23 added
// rounds to the nearest whole number, ties to even, and leaves it in the low byte.
template <typename T>
__device__ __forceinline__ u32x2 codes(const typename Eight<T>::Vec& v, float s, float r) {
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (float)v[e];
    float q = x * r;
    q = fmaf(fmaf(-q, s, x), r, q);
    q = fmaf(fmaf(-q, s, x), r, q);
    c[e] = __builtin_bit_cast(uint32_t, q + 12582912.0f);
  }
  u32x2 out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x04000c0cu);
    out[h] = lo | hi;
  }
  return out;
}

// The same for any scale above zero.
template <typename T>
__device__ __forceinline__ u32x2 codes_any(const typename Eight<T>::Vec& v, float s) {
  u32x2 out = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float q = fminf(fmaxf(rintf((float)v[e] / s), -127.0f), 127.0f);
    out[e / 4] |= ((uint32_t)(int)q & 0xff) << e % 4 * 8;
  }
  return out;
}

// A row's scale from its largest magnitude (as bits).
struct CodeScale {
  float scale, rcp;
  bool usual;  // codes() holds
};
__device__ __forceinline__ CodeScale code_scale(uint32_t top) {
  const float scale = top < 0x7f800000u ? __builtin_bit_cast(float, top) * (1.0f / 127.0f) : NAN;
  return {scale, 1.0f / scale, scale >= 0x1p-100f && scale <= 0x1p100f};
}

template <typename T>
__device__ __forceinline__ u32x2 codes_of(const typename Eight<T>::Vec& v, const CodeScale& s) {
  if (s.usual) return codes<T>(v, s.scale, s.rcp);
  return s.scale > 0.0f ? codes_any<T>(v, s.scale) : u32x2{0, 0};
}

// Elements 8 c to 8 c + 7 of a row of d, zeros behind the row.
template <typename T>
__device__ __forceinline__ typename Eight<T>::Vec eight_of(const T* row, uint32_t c, uint32_t d) {
  typename Eight<T>::Vec v = {};
  if (8 * c + 8 <= d) v = *reinterpret_cast<const typename Eight<T>::At*>(row + 8 * c);
  else if (8 * c < d) {
#pragma unroll
    for (uint32_t e = 0; e < 7; ++e)
      if (8 * c + e < d) v[e] = row[8 * c + e];
  }
  return v;
}

// A team of L lanes takes a row into registers, C times eight elements a lane
// (C == 0: a wider row, read twice), finds its largest magnitude and writes its
// codes. Bound by memory: 236000 rows of 4096 in bf16 take 480 us (6.0 TB/s), 65536 of
// 1024 31 us. One vector a lane leaves too few bytes in flight and too
// many workgroups to start: of bf16 (two or four vectors / one) 32768 x 2048 takes
// 31 / 71 us, 65536 x 512 17.3 / 35, 262144 x 64 10.5 / 18.6. From 2049 elements on
// a workgroup takes a row: eight vectors a lane of a wave take 146 us for 65536 x
// 4096, two a lane of four waves 136. With few rows it is all one launch.
template <typename T, int L, int C>
__global__ __launch_bounds__(kThreads) void k_quant_rows(QuantArgs a) {
  constexpr int kTeams = kThreads / L, kHold = C ? C : 1;
  __shared__ uint32_t s_top[2][kThreads / 64];
  const int64_t limit = a.limit ? *a.limit : (int64_t)a.rows;
  const uint32_t rows = limit < 0 ? 0u : limit < (int64_t)a.rows ? (uint32_t)limit : a.rows;
  const uint32_t lane = threadIdx.x % L, team = threadIdx.x / L;
  uint32_t turn = 0;
  for (uint64_t r0 = (uint64_t)blockIdx.x * kTeams; r0 < rows; r0 += (uint64_t)gridDim.x * kTeams, turn ^= 1) {
    const uint64_t r = min(r0 + team, (uint64_t)rows - 1);  // a team without a row repeats the last one
    const T* x = static_cast<const T*>(a.x) + r * a.d;
    typename Eight<T>::Vec v[kHold];
    uint32_t top = 0;
    if constexpr (C > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = eight_of<T>(x, c * L + lane, a.d);
#pragma unroll
      for (int c = 0; c < C; ++c) top = max(top, Eight<T>::top(v[c]));
    } else {
      for (uint32_t c = lane; 8 * c < a.d; c += L) top = max(top, Eight<T>::top(eight_of<T>(x, c, a.d)));
    }
#pragma unroll
    for (int m = 1; m < (L < 64 ? L : 64); m *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if constexpr (L > 64) {
      if (threadIdx.x % 64 == 0) s_top[turn][threadIdx.x / 64] = top;
      __syncthreads();
      top = max(max(s_top[turn][0], s_top[turn][1]), max(s_top[turn][2], s_top[turn][3]));
    }
    const CodeScale s = code_scale(top);
    int8_t* q = a.q + r * a.stride;
#pragma unroll
    for (int i = 0; i < (C ? C : 1); ++i) {
      for (uint32_t c = i * L + lane; 8 * c < a.stride; c += L) {
        if constexpr (C == 0) v[0] = eight_of<T>(x, c, a.d);
        *reinterpret_cast<u32x2*>(q + 8 * c) = codes_of<T>(v[i], s);
        if constexpr (C > 0) break;
      }
    }
    if (lane == 0) a.scale[r] = s.scale;
  }
}

template <typename T, int L, int C>
void launch_quant_rows(const QuantArgs& a, hipStream_t s) {
  constexpr uint32_t kTeams = kThreads / L;
  const uint32_t blocks = (a.rows + kTeams - 1) / kTeams;
  hipLaunchKernelGGL((k_quant_rows<T, L, C>), dim3(std::min(blocks, kMaxGrid)), dim3(kThreads), 0, s, a);
}

template <typename T>
hipError_t launch_quant(const QuantArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  if (a.d <= 64) launch_quant_rows<T, 4, 2>(a, s);
  else if (a.d <= 128) launch_quant_rows<T, 8, 2>(a, s);
  else if (a.d <= 256) launch_quant_rows<T, 8, 4>(a, s);
  else if (a.d <= 512) launch_quant_rows<T, 16, 4>(a, s);
  else if (a.d <= 1024) launch_quant_rows<T, 32, 4>(a, s);
  else if (a.d <= 2048) launch_quant_rows<T, 64, 4>(a, s);
  else if (a.d <= 4096) launch_quant_rows<T, 256, 2>(a, s);
  else if (a.d <= 8192) launch_quant_rows<T, 256, 4>(a, s);
  else launch_quant_rows<T, 256, 0>(a, s);
  return hipGetLastError();
}

hipError_t launch_quant(const QuantArgs& a, bool f32, hipStream_t s) {
  return f32 ? launch_quant<float>(a, s) : launch_quant<__bf16>(a, s);
}

// ---- products ----------------------------------------------------------------

struct Q8Args {
  const void* x;             // rows to be coded in the call (k_q8_few)
  uint32_t d;
  const int8_t* q;
  const float* q_scale;
  const int8_t* w;
  const float* w_scale;
  const int64_t* offsets;    // or null: one expert, every row
  const int32_t* src_index;  // or null
  void* out;
  uint32_t tuples;           // ids of src_index are below this
  uint32_t rows, n, E, stride;
  uint32_t gather;           // tuples of a row of q; 0: dispatched order
  uint32_t scatter;
  uint32_t col_tiles;
};

// Where a workgroup works: `rows` rows from row0 on, of expert e, and the
// columns from col0 on; rows == 0: there is no such tile.
struct Piece {
  uint32_t e, row0, rows, col0;
};

// The b-th tile of M rows and N columns. Row blocks are counted over the experts'
// segments in turn, a block's column tiles one after the other, and each XCD takes
// a contiguous range of them. Every lane of the wave takes part.
template <uint32_t M, uint32_t N>
__device__ __forceinline__ Piece piece_of(const Q8Args& a, uint64_t b) {
  if (!a.offsets) {
    const uint64_t total = (uint64_t)((a.rows + M - 1) / M) * a.col_tiles;
    if (b >= total) return {0, 0, 0, 0};
    if (total <= 0x7fffffffu) b = xcd_contiguous((uint32_t)b, (uint32_t)total);
    const uint32_t row0 = (uint32_t)(b / a.col_tiles) * M;
    return {0, row0, min(M, a.rows - row0), (uint32_t)(b % a.col_tiles) * N};
  }
  constexpr uint32_t kChunks = kMaxQ8Experts / 64;
  const uint32_t lane = threadIdx.x & 63;
  const int64_t most = min(max(a.offsets[a.E], (int64_t)0), (int64_t)a.rows);  // no row lies behind offsets[E]
  // the rows where the lane's experts (64 c + lane) begin and end, and the blocks up to theirs
  uint32_t begin[kChunks], end[kChunks], upto[kChunks];
  uint32_t from = (uint32_t)min(max(a.offsets[0], (int64_t)0), most), done = 0;
#pragma unroll
  for (uint32_t c = 0; c < kChunks; ++c)
    if (64 * c < a.E) end[c] = (uint32_t)min(max(a.offsets[min(64 * c + lane + 1, a.E)], (int64_t)0), most);
#pragma unroll
  for (uint32_t c = 0; c < kChunks; ++c) {
    if (64 * c >= a.E) break;
    uint32_t v = max(end[c], from);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v = max(v, (uint32_t)__shfl_up((int)v, m));  // a lane too low keeps its own
    uint32_t o = (uint32_t)__shfl_up((int)v, 1);
    begin[c] = lane == 0 ? from : o;
    end[c] = v;
    uint32_t n = (v - begin[c] + M - 1) / M;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      o = (uint32_t)__shfl_up((int)n, m);
      if ((int)lane >= m) n += o;
    }
    upto[c] = done + n;
    done = (uint32_t)__builtin_amdgcn_readlane((int)upto[c], 63);
    from = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
  const uint64_t total = (uint64_t)done * a.col_tiles;
  if (b >= total) return {0, 0, 0, 0};
  if (total <= 0x7fffffffu) b = xcd_contiguous((uint32_t)b, (uint32_t)total);
  const uint32_t rb = (uint32_t)(b / a.col_tiles), col0 = (uint32_t)(b % a.col_tiles) * N;
#pragma unroll
  for (uint32_t c = 0; c < kChunks; ++c) {
    if (64 * c >= a.E) break;
    const uint64_t has = __ballot(rb < upto[c]);
    if (!has) continue;
    const int at = __builtin_ctzll(has);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)begin[c], at);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)end[c], at);
    const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)upto[c], at);
    const uint32_t row0 = lo + (rb + (hi - lo + M - 1) / M - last) * M;
    return {64 * c + (uint32_t)at, row0, min(M, hi - row0), col0};
  }
  return {0, 0, 0, 0};
}

// Row of q that dispatched row i multiplies, and row of out that it gives (-1: none).
struct RowOf {
  uint32_t in;
  int64_t out;
};
// (without branches: it stands between products and what is done with them)
__device__ __forceinline__ RowOf row_from(const Q8Args& a, uint32_t i, int32_t g) {
  const bool indexed = a.src_index != nullptr, none = indexed && (g < 0 || (uint32_t)g >= a.tuples);
  const uint32_t in = indexed && a.gather ? (uint32_t)g / max(a.gather, 1u) : i;
  const uint32_t out = indexed && a.scatter ? (uint32_t)g : i;
  return {none ? 0u : in, none ? (int64_t)-1 : (int64_t)out};
}
__device__ __forceinline__ RowOf row_of(const Q8Args& a, uint32_t i) {
  return row_from(a, i, a.src_index ? a.src_index[i] : 0);
}

// GELU(z) = z Phi(z) = max(z, 0) - a h with a = |z| and h = Phi(-a) = t 2^(P(t) - a^2 log2(e) / 2),
// t = 1 / (1 + p a), of the form of gemm.h's gelu(), with a polynomial P of degree 7 instead of 4
// (gelu_fit.py 7: h is 2.9e-7 of itself off, not 3.8e-5). Rounding takes (2 z^2 + 26) 2^-24 of
// the result together, so that one bf16 result in 23000 is not the one nearest to z Phi(z), with
// degree 4 one in 330. In turn on one card, 131072 x 2 1024 -> 4096 takes 1.93 ms, with degree 4 1.86; one
// token's 8 experts 11.7 us and 11.4.
__device__ __forceinline__ float gelu_bf16(float z) {
  const float a = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.338f, a, 1.0f));
  float q = fmaf(-0.28095758f, t, 1.20971f);
  q = fmaf(q, t, -1.8158277f);
  q = fmaf(q, t, 0.9169416f);
  q = fmaf(q, t, -0.20344722f);
  q = fmaf(q, t, 0.62913746f);
  q = fmaf(q, t, 1.4347367f);
  q = fmaf(q, t, -2.8902936f);
  const float e = __builtin_amdgcn_exp2f(fmaf(z * z, -0.72134752f, q));  // -log2(e) / 2
  // (behind 20 the tail is zero; an infinite factor would make it NaN. NaN stays, by t)
  return fmaf(-fminf(a, 20.0f), t * e, fmaxf(z, 0.0f));
}

// bf16 results take the GELU above, fp32 ones the library's error function (-infinity
// gives zero, by a finite factor).
// A row's scale in two factors. A sum reaches 2^30, so that sum x scale of a scale from
// 2^97 on may pass the range of fp32 where the result, times the column's scale, does not;
// such a scale is divided by 2^32 and the product multiplied by that in the end. (No result
// loses bits on the way down: the sum times the least scales is a multiple of the least number.)
struct RowScale {
  float s, up;
};
__device__ __forceinline__ RowScale row_scale(float s) {
  const bool large = fabsf(s) >= 0x1p97f;
  return {large ? s * 0x1p-32f : s, large ? 0x1p32f : 1.0f};
}

template <typename T, bool kGelu>
__device__ __forceinline__ float finish(int sum, const RowScale& s, float ws) {
  const float z = (float)sum * s.s * ws * s.up;
  if constexpr (!kGelu) return z;
  else if constexpr (sizeof(T) == 2) return gelu_bf16(z);
  else return 0.5f * fmaxf(z, -FLT_MAX) * erfcf(z * -0.70710678f);
}

// A lane's 16 results of 32 columns of a row, rounded, in runs of 16 bytes: every
// other one, the rest is the other half wave's.
template <typename T>
struct Run {
  static constexpr int V = 16 / sizeof(T);
  typedef T Vec __attribute__((ext_vector_type(V)));
  typedef T At __attribute__((ext_vector_type(V), aligned(sizeof(T))));  // rows may begin anywhere
  Vec v[16 / V];
};

// Scale, activation and the one rounding; ws: of the lane's first column.
template <typename T, bool kGelu>
__device__ __forceinline__ Run<T> finish_run(const i32x16& acc, const RowScale& s, const float* ws) {
  constexpr int V = Run<T>::V;
  Run<T> r;
#pragma unroll
  for (int e = 0; e < 16; ++e) r.v[e / V][e % V] = (T)finish<T, kGelu>(acc[e], s, ws[e / V * 2 * V + e % V]);
  return r;
}

// Four chunks of each of four rows, a row's in the lanes that differ from one of them in
// bits 4 and 2 alone, change places: element k = 2 j + i of lane (bit 4: m, bit 2: n)
// becomes element 2 n + m of lane (bit 4: i, bit 2: j). A store of one element then
// writes whole lines. By whole waves.
template <typename Vec>
__device__ __forceinline__ void turn_rows(Vec* x) {
  i32x4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __builtin_bit_cast(i32x4, x[k]);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const auto both = __builtin_amdgcn_permlane16_swap((uint32_t)v[k][d], (uint32_t)v[k + 1][d], false, false);
      v[k][d] = (int)both[0];
      v[k + 1][d] = (int)both[1];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int lo = v[k][d], hi = v[k + 2][d];
      v[k][d] = __builtin_amdgcn_update_dpp(lo, hi, 0x114, 15, 10, false);      // lanes of bit 2: from 4 lanes below
      v[k + 2][d] = __builtin_amdgcn_update_dpp(hi, lo, 0x104, 15, 5, false);   // the others: from 4 above
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = __builtin_bit_cast(Vec, v[k]);
}

// Rows of results: of any length, of whole 16-byte chunks (k_q8_stay turns those into
// whole lines), of whole lines that go past the caches.
enum { kAnyRow, kWholeChunks, kPastCaches };

// Stores 16 bytes of results from column c on, of a row of n (0: it is not stored).
template <typename T, int kRow>
__device__ __forceinline__ void store_chunk(const typename Run<T>::Vec& v, T* row, uint32_t c, uint32_t n) {
  constexpr int V = Run<T>::V;
  if (c + V <= n) {
    typename Run<T>::At* to = reinterpret_cast<typename Run<T>::At*>(row + c);
    if constexpr (kRow == kPastCaches) __builtin_nontemporal_store(v, to);
    else *to = v;
  } else if constexpr (kRow == kAnyRow) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e < n) row[c + e] = v[e];
  }
}

// Stores a lane's results of 32 columns, its first one c, of a row of n (0: it is not stored).
template <typename T>
__device__ __forceinline__ void store_run(const Run<T>& r, T* row, uint32_t c, uint32_t n) {
  constexpr int V = Run<T>::V;
#pragma unroll
  for (int p = 0; p < 16 / V; ++p) store_chunk<T, kAnyRow>(r.v[p], row, c + p * 2 * V, n);
}

// Shape of a tile: BM x BN results by WM x WN waves, each MI x NI blocks of
// v_mfma_i32_32x32x32_i8; operands pass through a ring of S stages of D bytes of
// each row in LDS. KS such groups of waves share a tile, each with a ring and a
// part of the rows' length of its own.
template <int BM_, int BN_, int WM_, int WN_, int D_, int S_, int KS_ = 1, int kWaves_ = 2>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, D = D_, S = S_, KS = KS_;
  static constexpr int NT = 64 * WM * WN, MI = BM / WM / 32, NI = BN / WN / 32;
  static constexpr int kChunks = D / 16, kRows = 64 / kChunks;  // 16-byte chunks of a row; rows of a wave-wide load
  static constexpr int LA = BM * kChunks / NT, LB = BN * kChunks / NT;  // 16-byte loads of a lane and stage
  static constexpr int kB = BM * D, kStage = (BM + BN) * D;
  static constexpr int kRing = S * kStage, kLds = KS * kRing;
  static constexpr int kWaves = kWaves_;  // of a SIMD at once: they share its registers
};

// A thread's wave inside its group.
template <typename P>
__device__ __forceinline__ int wave_of(uint32_t tid) {
  return (int)(tid % P::NT >> 6);
}

// Slot of a row of D bytes in LDS that holds chunk c: an LDS read serves 16 lanes
// (256 bytes) at a time, here 16 rows at one chunk, which so lie in all the banks.
template <typename P>
__device__ __forceinline__ int slot_of(int c, int row) {
  return c ^ (P::D == 64 ? row >> 2 & 3 : row >> 1 & 7);
}

// Column of a tile that row r of B's LDS block holds. Register 4 q + e of lane l is
// MFMA row 8 q + 4 (l / 32) + e; of each 32 columns a lane gets the runs of V (16
// bytes of results) that begin at V (l / 32), so that one store instruction writes
// 32 neighbouring bytes of every row.
template <int V>
__device__ __forceinline__ int column_of(int r) {
  if constexpr (V == 4) return r;
  return (r & ~15) | (r >> 2 & 1) << 3 | (r >> 3 & 1) << 2 | (r & 3);
}

// What one lane loads: the chunk of its rows that its slot of each stage holds.
template <typename P>
struct Feed {
  const int8_t* a[P::LA];
  const int8_t* b[P::LB];
};

// 16 bytes a lane into 1 KiB of LDS, past the registers.
__device__ __forceinline__ void load_direct(const int8_t* from, unsigned char* to) {
  __builtin_amdgcn_global_load_lds(from, (mm::lds_ptr)to, 16, 0, 0);
}

// 4 bytes a lane into 256 bytes of LDS, past the registers.
__device__ __forceinline__ void load_words(const void* from, void* to) {
  __builtin_amdgcn_global_load_lds(from, (mm::lds_ptr)to, 4, 0, 0);
}

// Loads stage ks. Rows of 64 bytes more than whole stages of 128 end in half a
// stage: lanes whose chunk would lie behind the row repeat the one 64 bytes before
// (the chunk's number has bit 2 set: of the lane's slots in even rows of eight, or odd).
template <typename P>
__device__ __forceinline__ void load_stage(const Feed<P>& f, uint32_t ks, uint32_t stride, unsigned char* stage) {
  static_assert(P::D == 64 || (P::D == 128 && P::LA % 2 == 0 && P::LB % 2 == 0), "see slot_of");
  const int w = wave_of<P>(threadIdx.x);
  const uint32_t k = ks * P::D;
  int32_t even = (int32_t)k, odd = (int32_t)k;
  if constexpr (P::D == 128) {
    const int32_t back = k + P::D > stride ? 64 : 0, high = -(int32_t)(threadIdx.x >> 2 & 1);
    even -= back & high;
    odd -= back & ~high;
  }
#pragma unroll
  for (int i = 0; i < P::LA; ++i) load_direct(f.a[i] + (i % 2 ? odd : even), stage + (w * P::LA + i) * 1024);
#pragma unroll
  for (int i = 0; i < P::LB; ++i) load_direct(f.b[i] + (i % 2 ? odd : even), stage + P::kB + (w * P::LB + i) * 1024);
}

template <typename P>
struct Frags {
  i32x4 a[P::MI], b[P::NI];
};

// Byte offsets in a stage of the lane's operands in each 32 of its columns
// (those of the wave's other blocks follow in steps of 32 rows).
template <typename P>
struct Places {
  int a[P::D / 32], b[P::D / 32];
};

template <typename P>
__device__ __forceinline__ Places<P> places() {
  const uint32_t tid = mm::opaque_tid();
  const int lane = tid & 63, w = wave_of<P>(tid);
  const int ra = w / P::WN * (P::BM / P::WM) + (lane & 31), rb = w % P::WN * (P::BN / P::WN) + (lane & 31);
  Places<P> p;
#pragma unroll
  for (int kk = 0; kk < P::D / 32; ++kk) {
    const int c = 2 * kk + (lane >> 5);
    p.a[kk] = ra * P::D + (slot_of<P>(c, ra) << 4);
    p.b[kk] = P::kB + rb * P::D + (slot_of<P>(c, rb) << 4);
  }
  return p;
}

template <typename P>
__device__ __forceinline__ void read_frags(const unsigned char* stage, const Places<P>& p, int kk, Frags<P>& f) {
#pragma unroll
  for (int i = 0; i < P::MI; ++i) f.a[i] = *reinterpret_cast<const i32x4*>(stage + p.a[kk] + i * 32 * P::D);
#pragma unroll
  for (int j = 0; j < P::NI; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(stage + p.b[kk] + j * 32 * P::D);
}

template <typename P>
__device__ __forceinline__ void multiply(const Frags<P>& f, i32x16 (&acc)[P::MI][P::NI]) {
#pragma unroll
  for (int i = 0; i < P::MI; ++i)
#pragma unroll
    for (int j = 0; j < P::NI; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
}

// Instruction order of 32 columns: the reads of the next ones' operands (kRead)
// follow the first products, the loads of a stage (kLoad) the others (the
// compiler keeps loads that write LDS behind earlier reads of it).
template <typename P, bool kRead, bool kLoad>
__device__ __forceinline__ void schedule() {
  constexpr int M = P::MI * P::NI, R = kRead ? P::MI + P::NI : 0, L = kLoad ? P::LA + P::LB : 0;
  constexpr int kReads = kLoad && M > 2 ? (M - 1) / 2 : M;  // products among which the reads are spread
  constexpr int kLoads = M > kReads ? M - kReads : 1;       // and the loads
#pragma unroll
  for (int m = 0; m < M; ++m) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (m < kReads) {
#pragma unroll
      for (int r = (R * m + kReads - 1) / kReads; r < (R * (m + 1) + kReads - 1) / kReads; ++r)
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    } else {
#pragma unroll
      for (int l = L * (m - kReads) / kLoads; l < L * (m + 1 - kReads) / kLoads; ++l)
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

// The slots of the ring that a stage and the next one take.
struct Ring {
  uint32_t cur, next;
};

template <typename P>
__device__ __forceinline__ uint32_t after(uint32_t slot) {
  return slot + P::kStage == P::S * P::kStage ? 0u : slot + P::kStage;
}

// Stage ks, 32 columns after 32: each one's operands are read while the ones
// before multiply. Before the last ones multiply, a barrier publishes stage
// ks + 1 and, every wave having read all of stage ks, frees its slot, which stage
// ks + S (kLoad) takes. kWait: loads that may still be in flight then (63:
// any), -1: there is no stage ks + 1. On entry and on exit f[0] holds the next 32 columns.
template <typename P, bool kLoad, int kWait>
__device__ __forceinline__ void stage_step(const Feed<P>& f, const Places<P>& p, unsigned char* lds, uint32_t ks,
                                           uint32_t own, uint32_t stride, Ring& slot, Frags<P> (&g)[2],
                                           i32x16 (&acc)[P::MI][P::NI]) {
  constexpr int N = P::D / 32;
  static_assert(P::KS == 1 || N == 2, "both halves of a stage are here before it multiplies");
  // (a group whose part is shorter than the others' repeats its last stage, times zero)
  const int mine = P::KS == 1 || ks < own ? ~0 : 0;
#pragma unroll
  for (int kk = 0; kk + 1 < N; ++kk) {
    read_frags<P>(lds + slot.cur, p, kk + 1, g[(kk + 1) % 2]);
    if (P::D == 128 && kWait < 0 && kk >= 1) {  // half a stage: the rest of it multiplies with zeros
      const int keep = stride % 128 ? 0 : ~0;
#pragma unroll
      for (int i = 0; i < P::MI; ++i) g[(kk + 1) % 2].a[i] &= keep;
    }
    if (P::KS > 1) {
#pragma unroll
      for (int i = 0; i < P::MI; ++i) g[0].a[i] &= mine, g[1].a[i] &= mine;
    }
    multiply<P>(g[kk % 2], acc);
    schedule<P, true, false>();
  }
  if constexpr (kWait >= 0) {
    __builtin_amdgcn_s_waitcnt((kWait & 15) | ((kWait >> 4) << 14) | (7 << 4));  // vmcnt(kWait), lgkmcnt(0)
    mm::ring_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_frags<P>(lds + slot.next, p, 0, g[0]);
    if constexpr (kLoad) load_stage<P>(f, P::KS == 1 ? ks + P::S : min(ks + P::S, max(own, 1u) - 1), stride, lds + slot.cur);
  }
  multiply<P>(g[1], acc);
  schedule<P, (kWait >= 0), kLoad>();
  slot = {slot.next, after<P>(slot.next)};
}

// The products of a tile whose first S stages are in flight or in LDS, the first
// one published (read by every wave after a barrier); kHere: all of them, and the
// end of the first stage waits for no load nor for stores before this call. On
// return every wave has read all of the ring (barrier) and no load is in flight.
// nk: stages; own: those of them that are the group's.
template <typename P, bool kHere>
__device__ __forceinline__ void multiply_tile(const Feed<P>& f, unsigned char* lds, uint32_t nk, uint32_t own, uint32_t stride,
                                              i32x16 (&acc)[P::MI][P::NI]) {
  constexpr int LD = P::LA + P::LB;
#pragma unroll
  for (int i = 0; i < P::MI; ++i)
#pragma unroll
    for (int j = 0; j < P::NI; ++j) acc[i][j] = i32x16{};
  const Places<P> p = places<P>();
  Ring slot = {0, after<P>(0)};
  Frags<P> g[2];
  read_frags<P>(lds, p, 0, g[0]);
  uint32_t ks = 0;
  if (kHere && P::S < nk) stage_step<P, true, 63>(f, p, lds, ks++, own, stride, slot, g, acc);
  for (; ks + P::S < nk; ++ks) stage_step<P, true, (P::S - 2) * LD>(f, p, lds, ks, own, stride, slot, g, acc);
  for (; ks + 1 < nk; ++ks) stage_step<P, false, 0>(f, p, lds, ks, own, stride, slot, g, acc);
  stage_step<P, false, -1>(f, p, lds, ks, own, stride, slot, g, acc);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  mm::ring_barrier();
}

// The lane's part of B's rows: of expert e, columns from col0 on.
template <typename P, int V>
__device__ __forceinline__ void feed_b(const Q8Args& a, const Piece& g, Feed<P>& f) {
  const uint32_t tid = mm::opaque_tid(), lane = tid & 63, w = wave_of<P>(tid);
#pragma unroll
  for (int i = 0; i < P::LB; ++i) {
    const uint32_t r = (w * P::LB + i) * P::kRows + lane / P::kChunks;
    const uint32_t c = min(g.col0 + column_of<V>((int)r), a.n - 1);
    f.b[i] = a.w + ((uint64_t)g.e * a.n + c) * a.stride + (slot_of<P>(lane % P::kChunks, (int)r) << 4);
  }
}

// One tile a workgroup; while one multiplies, others of its CU start or end. Results
// go out as they are finished, 32 bytes of a row from each lane pair, past no cache:
// nontemporal stores of such parts of lines reach memory one by one (131072 x 2
// 1024 -> 4096 with 64 experts: 2194 us instead of 1804).
template <typename P, typename T, bool kGelu>
__global__ __launch_bounds__(P::NT * P::KS, P::kWaves) void k_q8_tile(Q8Args a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float s_scale[(P::BM + 63) / 64 * 64], s_ws[P::BN];
  __shared__ int64_t s_out[P::BM];
  constexpr int NT = P::NT * P::KS;
  for (uint64_t b = blockIdx.x;; b += gridDim.x) {
    const Piece g = piece_of<P::BM, P::BN>(a, b);
    if (g.rows == 0) return;  // nor is there a later one
    const int tid = threadIdx.x, lane = tid & 63, w = wave_of<P>(tid), group = tid / P::NT;
    const uint32_t stages = (a.stride + P::D - 1) / P::D, nk = (stages + P::KS - 1) / P::KS;  // of the rows; of a group at most
    const uint32_t first = min(group * nk, stages - 1), own = min(stages - min(group * nk, stages), nk);
    unsigned char* ring = lds + group * P::kRing;
    Feed<P> f;
    RowOf row[P::LA];
#pragma unroll
    for (int i = 0; i < P::LA; ++i) {
      const uint32_t r = (w * P::LA + i) * P::kRows + lane / P::kChunks;
      row[i] = row_of(a, g.row0 + min(r, g.rows - 1));
      f.a[i] = a.q + (uint64_t)row[i].in * a.stride + (slot_of<P>(lane % P::kChunks, (int)r) << 4) + first * P::D;
    }
    feed_b<P, Run<T>::V>(a, g, f);
#pragma unroll
    for (int i = 0; i < P::LB; ++i) f.b[i] += first * P::D;
    // the scales before the stages: who waits for a stage has waited for them
    const int wave = tid / 64;
    for (int c = wave; c < (P::BM + 63) / 64; c += NT / 64)
      load_words(a.q_scale + row_of(a, g.row0 + min((uint32_t)(64 * c + lane), g.rows - 1)).in, s_scale + 64 * c);
    for (int c = wave; c < P::BN / 64; c += NT / 64)
      load_words(a.w_scale + (uint64_t)g.e * a.n + min(g.col0 + 64 * c + lane, a.n - 1), s_ws + 64 * c);
#pragma unroll
    for (uint32_t s = 0; s < P::S; ++s)
      if (s < nk) load_stage<P>(f, P::KS == 1 ? s : min(s, max(own, 1u) - 1), a.stride, ring + s * P::kStage);
#pragma unroll
    for (int i = 0; i < P::LA; ++i) {
      const uint32_t r = (w * P::LA + i) * P::kRows + lane / P::kChunks;
      if (lane % P::kChunks == 0 && group == 0) s_out[r] = r < g.rows ? row[i].out : -1;
    }
    if (nk >= P::S) mm::wait_vmem<(P::S - 1) * (P::LA + P::LB)>();
    else mm::wait_vmem<0>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // s_out is written
    mm::ring_barrier();
    i32x16 acc[P::MI][P::NI];
    multiply_tile<P, false>(f, ring, nk, own, a.stride, acc);
    if constexpr (P::KS > 1) {  // the groups' sums meet in the first one, in the place of its stages
      i32x4* part = reinterpret_cast<i32x4*>(lds);
      constexpr int Q = P::MI * P::NI * 4;
      static_assert((P::KS - 1) * Q * P::NT * 16 <= P::kLds, "the sums fit");
      if (group > 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const i32x16& v = acc[q / 4 / P::NI][q / 4 % P::NI];
          part[((group - 1) * Q + q) * P::NT + tid % P::NT] = i32x4{v[q % 4 * 4], v[q % 4 * 4 + 1], v[q % 4 * 4 + 2], v[q % 4 * 4 + 3]};
        }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int p = 0; p < P::KS - 1; ++p)
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const i32x4 v = part[(p * Q + q) * P::NT + tid % P::NT];
            i32x16& to = acc[q / 4 / P::NI][q / 4 % P::NI];
#pragma unroll
            for (int e = 0; e < 4; ++e) to[q % 4 * 4 + e] += v[e];
          }
      }
    }
    T* out = static_cast<T*>(a.out);
    if (P::KS == 1 || group == 0) {
#pragma unroll
      for (int i = 0; i < P::MI; ++i) {
        const int r = w / P::WN * (P::BM / P::WM) + 32 * i + (lane & 31);
        const int64_t o = s_out[r];
        const RowScale s = row_scale(s_scale[r]);
#pragma unroll
        for (int j = 0; j < P::NI; ++j) {
          const uint32_t c = w % P::WN * (P::BN / P::WN) + 32 * j + Run<T>::V * (lane >> 5);
          store_run<T>(finish_run<T, kGelu>(acc[i][j], s, s_ws + c), out + (uint64_t)o * a.n, g.col0 + c, o < 0 ? 0u : a.n);
        }
      }
    }
    __syncthreads();  // before the next tile's scales and stages
  }
}

// ---- many tiles: workgroups that stay ------------------------------------------

// Where the experts' rows begin and how many blocks of M rows there are up to each
// one's end (s_upto, all ones behind the last); returns the blocks in all. By
// one wave; every lane takes part.
template <uint32_t M>
__device__ __forceinline__ uint32_t list_blocks(const Q8Args& a, uint32_t* s_begin, uint32_t* s_upto) {
  const uint32_t lane = threadIdx.x & 63;
  if (!a.offsets) {
    const uint32_t blocks = (a.rows + M - 1) / M;
    s_upto[lane] = lane ? ~0u : blocks;
    if (lane < 2) s_begin[lane] = lane * a.rows;
    return blocks;
  }
  const int64_t most = min(max(a.offsets[a.E], (int64_t)0), (int64_t)a.rows);
  uint32_t from = (uint32_t)min(max(a.offsets[0], (int64_t)0), most), done = 0;
  if (lane == 0) s_begin[0] = from;
  for (uint32_t e0 = 0; e0 < a.E; e0 += 64) {
    const uint32_t e = e0 + lane;
    uint32_t end = max((uint32_t)min(max(a.offsets[min(e + 1, a.E)], (int64_t)0), most), from);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) end = max(end, (uint32_t)__shfl_up((int)end, m));  // a lane too low keeps its own
    uint32_t begin = (uint32_t)__shfl_up((int)end, 1);
    if (lane == 0) begin = from;
    uint32_t upto = (end - begin + M - 1) / M;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const uint32_t o = (uint32_t)__shfl_up((int)upto, m);
      if ((int)lane >= m) upto += o;
    }
    upto += done;
    s_upto[e] = e < a.E ? upto : ~0u;
    if (e < a.E) s_begin[e + 1] = end;
    done = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    from = (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
  }
  return done;
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// The tile of workgroup turn b (below the total), from the list. An XCD's tiles are
// contiguous, in patches of kPatch row blocks by 4 column tiles, as many as its 32
// CUs work on at a time: they share what they load (262144 x 1024 -> 4096 with kPatch
// 2, 4, 8, 16: 1424, 1406, 1340, 1352 us).
constexpr uint32_t kPatch = 8;

template <typename P>
__device__ __forceinline__ Piece listed_piece(const Q8Args& a, uint32_t b, uint32_t total, const uint32_t* s_begin,
                                              const uint32_t* s_upto) {
  b = xcd_contiguous(b, total);
  const uint32_t band = b / (kPatch * a.col_tiles), high = min(kPatch, total / a.col_tiles - band * kPatch);
  uint32_t at = b % (kPatch * a.col_tiles);
  const uint32_t col = at / (high * 4) * 4, wide = min(4u, a.col_tiles - col);
  at -= col * high;
  const uint32_t rb = band * kPatch + at / wide, lane = threadIdx.x & 63;
  uint32_t e = 0;
  for (uint32_t e0 = 0; e0 < a.E; e0 += 64) e += __popcll(__ballot(s_upto[e0 + lane] <= rb));
  e = uniform(e);
  const uint32_t lo = uniform(s_begin[e]), hi = uniform(s_begin[e + 1]), before = e ? uniform(s_upto[e - 1]) : 0u;
  const uint32_t row0 = lo + (rb - before) * P::BM;
  return {e, row0, min((uint32_t)P::BM, hi - row0), (col + at % wide) * P::BN};
}

// As k_q8_tile, with one workgroup a CU that walks over tiles: the next tile's
// rows are looked up while this one multiplies, and its first stages are on their
// way while this one's results are scaled and stored. No branch stands between
// the products and the stores (it would make the accumulators move): behind the
// last tile it is started once more, in vain. 131072 x 2 rows of 64 experts, codes given:
// 4096 -> 1024 in 1.0 to 1.1 ms (2.0 P operations/s, as the library's one large product),
// 1024 -> 4096 with GELU in 1.84 ms, without in 1.47: a tile multiplies for 8 stages only there, and
// what a CU's one workgroup does then (GELU 0.37 ms, stores 0.25) nothing covers. Results are turned
// among lanes so that a store writes whole lines, past the caches where they are many (whole
// lines / 32 bytes of each of 32 rows a store, in turn on one card: 1.95 and 2.01 ms with GELU, 1.49 and
// 1.57 without; 65536 x 2 of 8 experts in fp32 without GELU 0.94 and 1.36 ms; 32768 x 2 -> 2048 fp32
// 212 and 299 us, with GELU 385 and 412, bf16 with GELU 248 and 242; rows that end inside a chunk,
// 2001 long, 238 and 223 with a shorter GELU, so those stay as they are); the first use of an expert's
// weights costs 12 %, and the clock 15 % (so much less time do weights of zeros take). Two workgroups a
// CU with tiles of 128 x 256 cover it but load 768 rows of operands for the 512 of one 256 x 256 tile, 1.5
// times as much from the caches: 1.98 ms with GELU, 1.78 without; waves of 4 x 2 or of raised
// priority change nothing. 64-byte stages instead of 128: 8192^3 in 595 us instead of 571 (a CU's loads are then
// twice as many, of half a line each).
template <typename P, typename T, bool kGelu, int kRow>
__global__ __launch_bounds__(P::NT, P::kWaves) void k_q8_stay(Q8Args a) {
  static_assert(P::NT == P::BM + P::BN && P::BM % 64 == 0, "a thread for each scale");
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float s_scale[2][P::NT];  // of the rows, then of the columns
  __shared__ int32_t s_src[2][P::NT];  // of the rows; the rest is not looked at
  __shared__ uint32_t s_begin[kMaxQ8Experts + 1], s_upto[kMaxQ8Experts], s_total;
  if (threadIdx.x < 64) {
    const uint32_t blocks = list_blocks<P::BM>(a, s_begin, s_upto);
    if (threadIdx.x == 0) s_total = blocks * a.col_tiles;
  }
  __syncthreads();
  const uint32_t total = uniform(s_total), stages = (a.stride + P::D - 1) / P::D;
  uint32_t b = blockIdx.x;
  if (b >= total) return;

  // ids of a tile's rows (without an index: any words)
  auto load_ids = [&](const Piece& g, int32_t* to) {
    const uint32_t tid = mm::opaque_tid(), i = g.row0 + min(tid & (P::BM - 1), g.rows - 1);
    load_words(a.src_index ? (const void*)(a.src_index + i) : (const void*)a.w_scale, to + (tid & ~63u));
  };
  auto row_at = [&](const Piece& g, const int32_t* ids, uint32_t r) { return row_from(a, g.row0 + min(r, g.rows - 1), ids[r]); };
  // a tile's scales, then its first stages
  auto start = [&](const Piece& g, const int32_t* ids, float* scale, Feed<P>& f) {
    const uint32_t tid = mm::opaque_tid(), lane = tid & 63, w = tid >> 6;
    const float* of_row = a.q_scale + row_at(g, ids, tid & (P::BM - 1)).in;
    const float* of_column = a.w_scale + (uint64_t)g.e * a.n + min(g.col0 + (tid & (P::BM - 1)), a.n - 1);
    load_words(tid < P::BM ? of_row : of_column, scale + (tid & ~63u));
#pragma unroll
    for (int i = 0; i < P::LA; ++i) {
      const uint32_t r = (w * P::LA + i) * P::kRows + lane / P::kChunks;
      f.a[i] = a.q + (uint64_t)row_at(g, ids, r).in * a.stride + (slot_of<P>(lane % P::kChunks, (int)r) << 4);
    }
    feed_b<P, Run<T>::V>(a, g, f);
#pragma unroll
    for (uint32_t s = 0; s < P::S; ++s) load_stage<P>(f, min(s, stages - 1), a.stride, lds + s * P::kStage);
  };

  Piece g = listed_piece<P>(a, b, total, s_begin, s_upto);
  load_ids(g, s_src[0]);
  mm::wait_vmem<0>();
  mm::ring_barrier();
  Feed<P> f;
  start(g, s_src[0], s_scale[0], f);
  mm::wait_vmem<0>();
  uint32_t turn = 0;
  while (true) {
    mm::ring_barrier();  // the tile's first stages and its scales are there
    const bool more = b + gridDim.x < total;
    const Piece next = more ? listed_piece<P>(a, b + gridDim.x, total, s_begin, s_upto) : g;
    load_ids(next, s_src[turn ^ 1]);
    i32x16 acc[P::MI][P::NI];
    multiply_tile<P, true>(f, lds, stages, stages, a.stride, acc);
    start(next, s_src[turn ^ 1], s_scale[turn ^ 1], f);
    const uint32_t tid = mm::opaque_tid(), lane = tid & 63, w = tid >> 6;
    T* out = static_cast<T*>(a.out);
    // half of the results are finished before the loads are waited for, and the
    // first store follows that wait: the counter then holds stores alone
    constexpr int H = (P::MI + 1) / 2, V = Run<T>::V, G = P::NI * 4 / V;  // groups of 4 chunks of a row
    constexpr bool kTurn = kRow != kAnyRow;
    static_assert(P::NI * 16 == G * 4 * V, "whole groups");
    typename Run<T>::Vec first[H][4 * G];
#pragma unroll
    for (int i = 0; i < P::MI; ++i) {
      const uint32_t r = w / P::WN * (P::BM / P::WM) + 32 * i + (lane & 31);
      const RowScale s = row_scale(s_scale[turn][r]);
      typename Run<T>::Vec chunk[4 * G];
#pragma unroll
      for (int j = 0; j < P::NI; ++j) {
        const uint32_t c = w % P::WN * (P::BN / P::WN) + 32 * j + V * (lane >> 5);
        const Run<T> run = finish_run<T, kGelu>(acc[i][j], s, &s_scale[turn][P::BM + c]);
#pragma unroll
        for (int p = 0; p < 16 / V; ++p) chunk[16 / V * j + p] = run.v[p];
      }
#pragma unroll
      for (int q = 0; q < G; ++q)
        if constexpr (kTurn) turn_rows(&chunk[4 * q]);
      if (i < H) {
#pragma unroll
        for (int q = 0; q < 4 * G; ++q) first[i][q] = chunk[q];
        if (i < H - 1) continue;
      }
      if (i == H - 1) mm::wait_vmem<0>();
#pragma unroll
      for (int i0 = i == H - 1 ? 0 : i; i0 <= i; ++i0) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t r0 = w / P::WN * (P::BM / P::WM) + 32 * i0 + (kTurn ? (lane & 11) | m / 2 << 2 | m % 2 << 4 : lane & 31);
          const RowOf row = row_at(g, s_src[turn], r0);
          const uint32_t n = r0 < g.rows && row.out >= 0 ? a.n : 0u;
          T* to = out + (uint64_t)row.out * a.n;
#pragma unroll
          for (int q = 0; q < G; ++q) {
            const uint32_t k = kTurn ? (lane >> 4 & 1) | (lane >> 2 & 1) << 1 : m;
            const uint32_t c0 = g.col0 + w % P::WN * (P::BN / P::WN) + 8 * V * q + 2 * V * k + V * (lane >> 5);
            store_chunk<T, kRow>(i0 < H ? first[i0 < H ? i0 : 0][4 * q + m] : chunk[4 * q + m], to, c0, n);
          }
        }
      }
    }
    if (!more) return;
    b += gridDim.x;
    g = next;
    turn ^= 1;
  }
}

// More LDS than 64 KiB has to be asked for.
hipError_t allow_lds(const void* kernel, uint32_t bytes) {
  return bytes > 60 * 1024 ? hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : hipSuccess;
}

// Results of so many bytes are not in the last-level cache (256 MiB) when they are read
// (past the caches / through them: 262144 x 1024 -> 4096 1.24 / 1.32 ms, 131072 x 1024 -> 4096 of
// 8 experts in fp32 0.79 / 0.96 ms).
constexpr uint64_t kManyBytes = 512ull << 20;

template <typename P, typename T, bool kGelu>
hipError_t launch_stay(Q8Args a, hipStream_t s) {
  a.col_tiles = (a.n + P::BN - 1) / P::BN;
  const uint64_t tiles = ((uint64_t)a.rows / P::BM + (a.offsets ? a.E : 1)) * a.col_tiles;  // at most
  int device = 0, cus = 0;
  hipError_t e = hipGetDevice(&device);
  if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device);
  if (e != hipSuccess) return e;
  auto launch = [&](void (*kernel)(Q8Args)) {
    if ((e = allow_lds((const void*)kernel, P::kLds)) != hipSuccess) return;
    const uint32_t grid = (uint32_t)std::min<uint64_t>(tiles, std::max(8, cus / 8 * 8));
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(P::NT), P::kLds, s, a);
  };
  const uint64_t row = a.n * sizeof(T);
  if (a.rows * row >= kManyBytes && row % 128 == 0 && (uintptr_t)a.out % 128 == 0) launch(k_q8_stay<P, T, kGelu, kPastCaches>);
  else if (row % 16 == 0) launch(k_q8_stay<P, T, kGelu, kWholeChunks>);
  else launch(k_q8_stay<P, T, kGelu, kAnyRow>);
  if (e != hipSuccess) return e;
  return hipGetLastError();
}

template <typename P, typename T, bool kGelu>
hipError_t launch_tile(Q8Args a, hipStream_t s) {
  a.col_tiles = (a.n + P::BN - 1) / P::BN;
  const uint64_t blocks = a.offsets ? std::min<uint64_t>(a.rows, a.rows / P::BM + a.E) : ((uint64_t)a.rows + P::BM - 1) / P::BM;
  const uint32_t grid = (uint32_t)std::min<uint64_t>(blocks * a.col_tiles, kMaxGrid);
  const hipError_t e = allow_lds((const void*)k_q8_tile<P, T, kGelu>, P::kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_q8_tile<P, T, kGelu>), dim3(grid), dim3(P::NT * P::KS), P::kLds, s, a);
  return hipGetLastError();
}

// ---- a few rows: the weights pass through registers ----------------------------

// Each wave multiplies 16 columns of its expert's matrix, over one of KS parts of
// their length, with up to 16 rows: all 16 KiB of the matrix that it can hold
// are on their way at once, and no other wave reads them. The parts' sums (whole
// numbers: exact in any order) meet in LDS. Every workgroup makes the codes of its
// rows itself, while the matrix is on its way. Against codes in a launch of their
// own and tiles: one row 4096 -> 1024 in 7.1 us instead of 15.3, one token's 8 experts 4096 ->
// 1024 in 10.1 instead of 18.1, 1024 -> 4096 in 11.4 instead of 12.2 (33.8 MB: 4.8 us at the rate of a
// large read; what is left is the launch, the codes and the ramp of the loads). With more rows codes are
// made over and over, and no tile shares what it loads (tiles / so, weights not in the caches): 2
// tokens of 8 1024 -> 4096 19.1 and 19.9, 4096 -> 1024 18.1 and 19.2, 3 25.8 and 26.2, 26.0 and 24.8; of one
// expert 9 rows 9.4 and 9.7, 12.8 and 11.3, 16 rows 9.5 and 11.4, 13.0 and 14.2.
constexpr int kHeld = 16;              // 64-byte steps of 16 columns in registers
constexpr uint32_t kCodeWidth = 4096;  // of the rows that a workgroup codes: 8 chunks a lane
constexpr uint32_t kFewRows = 8;       // of a call

template <typename T, bool kGelu, int KS>
__global__ __launch_bounds__(kThreads) void k_q8_few(Q8Args a) {
  constexpr int kGroups = 4 / KS;  // of 16 columns
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int32_t s_sum[KS > 1 ? KS : 1][16][20];  // [part][row][column]
  __shared__ float s_scale[kFewRows];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  // every row's id at once with the segments: nothing else stands before the rows
  const int32_t ids = a.src_index ? a.src_index[min((uint32_t)lane, a.rows - 1)] : 0;
  auto row_at = [&](uint32_t i) { return row_from(a, i, __shfl(ids, (int)i)); };  // by whole waves
  const Piece g = piece_of<16, 16 * kGroups>(a, blockIdx.x);
  if (g.rows == 0) return;
  const int part = w % KS, group = w / KS;
  const uint32_t nk = a.stride / 64, each = (nk + KS - 1) / KS, k0 = min(part * each, nk), k1 = min(k0 + each, nk);
  const uint32_t chunk = lane / 16 * 16, pitch = a.stride + 16;  // (of the codes in LDS: rows in different banks)

  // the rows to be coded come first: nothing waits for the matrix before it has to
  constexpr int kEach = kCodeWidth / 512;
  typename Eight<T>::Vec v[kEach];
  auto load_row = [&](uint32_t r) {
    const T* x = static_cast<const T*>(a.x) + (uint64_t)row_at(g.row0 + r).in * a.d;
#pragma unroll
    for (int c = 0; c < kEach; ++c) v[c] = eight_of<T>(x, c * 64 + lane, a.d);
  };
  load_row(min((uint32_t)w, g.rows - 1));
  const uint32_t col0 = g.col0 + group * 16;
  const int8_t* pw = a.w + ((uint64_t)g.e * a.n + min(col0 + lane % 16, a.n - 1)) * a.stride + chunk;
  i32x4 b[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) b[i] = *reinterpret_cast<const i32x4*>(pw + min(k0 + i, nk - 1) * 64);
#pragma unroll 1
  for (uint32_t r = w; r < g.rows; r += 4) {
    if (r >= 4) load_row(r);
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kEach; ++c) top = max(top, Eight<T>::top(v[c]));
#pragma unroll
    for (int m = 1; m < 64; m *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    const CodeScale s = code_scale(top);
#pragma unroll
    for (int c = 0; c < kEach; ++c)
      if (512 * c + 8 * lane < a.stride) *reinterpret_cast<u32x2*>(lds + r * pitch + 512 * c + 8 * lane) = codes_of<T>(v[c], s);
    if (lane == 0) s_scale[r] = s.scale;
  }
  __syncthreads();

  i32x4 acc = {};
  const unsigned char* from = lds + min((uint32_t)lane % 16, g.rows - 1) * pitch + chunk;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int keep = k0 + i < k1 ? ~0 : 0;  // the steps behind the part's last are zeros
    const i32x4 x = *reinterpret_cast<const i32x4*>(from + min(k0 + i, nk - 1) * 64) & keep;
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[i], x, acc, 0, 0, 0);
  }

  // the lane holds 4 columns from 4 (lane / 16) on of row lane % 16
  const float* ws = a.w_scale + (uint64_t)g.e * a.n;
  T* out = static_cast<T*>(a.out);
  if constexpr (KS == 1) {
    const uint32_t r = lane % 16;
    const RowOf to = row_at(g.row0 + min(r, g.rows - 1));
    if (r < g.rows && to.out >= 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t c = col0 + lane / 16 * 4 + e;
        if (c < a.n) out[(uint64_t)to.out * a.n + c] = (T)finish<T, kGelu>(acc[e], row_scale(s_scale[r]), ws[c]);
      }
    }
  } else {
    // one group of columns after the other: its parts' sums, then a thread for each result
    const uint32_t r = threadIdx.x / 16;
    const RowOf to = row_at(g.row0 + min(r, g.rows - 1));
    for (int t = 0; t < kGroups; ++t) {
      __syncthreads();
      if (group == t) *reinterpret_cast<i32x4*>(&s_sum[part][lane % 16][lane / 16 * 4]) = acc;
      __syncthreads();
      const uint32_t c = g.col0 + 16 * t + threadIdx.x % 16;
      if (r < g.rows && c < a.n && to.out >= 0) {
        int sum = 0;
#pragma unroll
        for (int p = 0; p < KS; ++p) sum += s_sum[p][r][threadIdx.x % 16];
        out[(uint64_t)to.out * a.n + c] = (T)finish<T, kGelu>(sum, row_scale(s_scale[r]), ws[c]);
      }
    }
  }
}

template <typename T, bool kGelu, int KS>
hipError_t launch_few(Q8Args a, hipStream_t s) {
  constexpr uint32_t N = 16 * (4 / KS);
  a.col_tiles = (a.n + N - 1) / N;
  const uint32_t blocks = a.offsets ? a.rows : 1, lds = kFewRows * (a.stride + 16);
  hipLaunchKernelGGL((k_q8_few<T, kGelu, KS>), dim3(blocks * a.col_tiles), dim3(kThreads), lds, s, a);
  return hipGetLastError();
}

// Whether a product makes the codes of x itself, in one launch.
bool codes_inside(uint32_t rows, uint32_t stride) { return rows <= kFewRows && stride <= kCodeWidth; }

template <typename T, bool kGelu>
hipError_t launch_product(const Q8Args& a, hipStream_t s) {
  typedef Shape<256, 256, 2, 4, 128, 2> Large;
  typedef Shape<128, 256, 2, 2, 64, 3> Middle;
  typedef Shape<128, 128, 2, 2, 64, 4> Square;
  typedef Shape<64, 128, 2, 2, 128, 3> Long;
  typedef Shape<64, 64, 2, 2, 64, 4> Small;
  typedef Shape<64, 64, 2, 2, 64, 4, 4, 4> Parted;
  typedef Shape<32, 64, 1, 2, 128, 5> Flat;
  if (a.x) {
    // as many parts of a row as waves need to hold it in their registers
    constexpr uint32_t kPart = kHeld * 64;
    static_assert(kCodeWidth <= 4 * kPart, "four parts hold the longest row");
    if (a.stride > 2 * kPart) return launch_few<T, kGelu, 4>(a, s);
    return a.stride > kPart ? launch_few<T, kGelu, 2>(a, s) : launch_few<T, kGelu, 1>(a, s);
  }
  // tiles of a height and width that there will be about, half of each expert's last one empty
  auto tiles = [&](uint32_t m, uint32_t n) {
    const uint64_t blocks = a.E > 1 ? std::min<uint64_t>(a.rows, a.rows / m + a.E / 2) : ((uint64_t)a.rows + m - 1) / m;
    return blocks * ((a.n + n - 1) / n);
  };
  // Times in us with the codes given, where no other case is named for 64 experts and two of
  // them a token ("dense": one expert); rows are counted on the host as a call's most, so an
  // expert's are a guess.
  //  Large, stays: tiles enough for every CU. Dense 1024 -> 4096, 65536 rows: Large 396,
  //    Middle 448, Square 546, Small 732; 4096 rows 31, 32, 34, 46; 16384 tokens (512 rows an
  //    expert) 287, 291, 347, 478, but 8192 tokens 194, 166, 200, 273. Few codes a row and one expert leave
  //    mostly the finishing of results, which two workgroups a CU share (65536 rows with GELU
  //    64 -> 1792: 109 and 86, 512 -> 1792: 138 and 131, in fp32 242 and 232; 128 -> 1792 without 61 and 56, but 512
  //    97 and 100, and fp32 103 and 129). 19 experts, 150396 rows -> 1792, without GELU 143 and 182 at 46 codes,
  //    228 and 291 at 512, fp32 215 and 278, 305 and 444; with GELU 263 and 233, 323 and 344, fp32 516 and 415,
  //    559 and 555: there the shortest rows would gain by Middle too.
  //  Middle: three tiles for two CUs at least. 2048 tokens 1024 -> 4096: Middle 88, Square 93,
  //    Small 102; 256 tokens (8 rows an expert) 69, 76, 63. Dense, 2048 rows: 20.2, 18.8, 24.5.
  //  Long: 128-byte stages are whole lines and half as many waits, where rows are long. Dense 4096 -> 1024,
  //    2048 rows 15.6 (Square 20.6, Small 18.4), 4096 rows 23.8 (22.7, 35.3); 2048 -> 1024, 2048 rows 10.9 (Square
  //    11.8), 3000 rows 14.8 (16.9). Shorter rows: 1984 codes 11.4 (Small 12.8) and 16.0 (17.3) but 18.1 (16.5)
  //    for 4096 rows; 1024 codes 8.2 (8.3), 10.9 (10.9), 11.3 (11.6); 512 codes 6.8 (6.7), 9.0 (7.9), 8.9 (9.5); with
  //    fewer than 256 tiles it loses (1000 rows 2048 -> 1024 10.7 and 9.1, 1024 -> 1024 8.1 and 6.8).
  //  Square: dense 1024 -> 4096, 2048 rows 18.8 (Middle 20.2, Small 24.5); dense 4096 -> 1024,
  //    8192 rows 43.3 (Middle 39.7, Small 69.5).
  //  Flat: few rows an expert and long rows, so the weights come from memory: tiles of whole lines
  //    and a deep ring. Weights not in the caches, 16, 48, 128, 200 tokens of 8 (Flat / Small),
  //    codes made in the call: 4096 -> 1024 60 / 62, 65 / 67, 77 / 78, 80 / 83; 4096 -> 2048 99 / 98,
  //    112 / 116, 121 / 133, 137 / 147; 2560 -> 1024 38 / 39, 41 / 44, 51 / 52, 55 / 57; but 2048 -> 1024
  //    33 / 31, 36 / 34, 44 / 40, 47 / 45 and 1024 -> 4096 (codes given) 69 / 56, 78 / 63, 88 / 71.
  //  Parted: fewer tiles than CUs and long rows: four groups of waves share a tile's length.
  //    Dense 4096 -> 1024, 16 to 256 rows: 13.2 to 14.2 (Small 16.4); 2048 -> 1024 7.8 to 8.4 (8.9 to 9.1), 512 rows
  //    8.9 (9.2); 1984 codes 7.9 to 8.9 (8.9 to 9.1), 1024 codes 5.5 to 6.6 (5.8 to 6.5), 512 codes 5.0 to 5.5 (4.5
  //    to 5.2); 512 tiles 11.6 (8.3, 1024 codes).
  const uint64_t each = a.rows / a.E, large = tiles(256, 256);
  const bool finishing = a.E == 1 && a.stride <= 512 && (sizeof(T) == 2 || kGelu);
  if (each >= 512 && !finishing && large >= 256 && large <= 0x3fffffff) return launch_stay<Large, T, kGelu>(a, s);
  if (each >= 32 && tiles(128, 256) >= 384) return launch_tile<Middle, T, kGelu>(a, s);
  if (each >= 32 && a.stride >= 2048 && tiles(64, 128) >= 256) return launch_tile<Long, T, kGelu>(a, s);
  if (each >= 32 && tiles(128, 128) >= 256) return launch_tile<Square, T, kGelu>(a, s);
  if (a.E > 1 && a.stride > 2048 && each < 32 && tiles(32, 64) >= 512) return launch_tile<Flat, T, kGelu>(a, s);
  if (tiles(64, 64) <= 256 && a.stride >= 2048) return launch_tile<Parted, T, kGelu>(a, s);
  return launch_tile<Small, T, kGelu>(a, s);
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
  if (io->x && codes_inside(a.rows, a.stride)) {
    a.x = io->x;
    a.d = d->d;
  } else if (io->x) {
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
