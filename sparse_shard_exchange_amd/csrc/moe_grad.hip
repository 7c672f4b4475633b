// Gradients of a mixture-of-experts step's combine, dispatch and router.
//
// The step (moe.hip): row slot(t, s) of the dispatched rows holds token t for
// its s-th expert (s = 0, 1; slot -1: dropped by the capacity);
//   out_t = sum_s g_ts y[slot(t, s)],   xd[slot(t, s)] = x_t,   l_t = x_t W
// Its gradients, with the experts' own products in between left to the
// caller (from dy to dxd):
//   dy[slot(t, s)] = g_ts dout_t        dg_ts = dout_t . y[slot(t, s)]
//   dx_t = sum_s dxd[slot(t, s)] + dl_t W^T      dW = x^T dl
#include "ops.h"

#include <algorithm>

namespace pw {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

struct CombineGradArgs {
  const __bf16* dout;
  const __bf16* y;
  const float* gates;
  const int32_t* src_index;
  const int64_t* offsets;
  const uint8_t* valid;
  __bf16* dy;
  float* dgates;
  int32_t* slot_of;
  uint64_t rows;
  uint32_t tokens, d, E;
};

struct DispatchGradArgs {
  const __bf16* dxd;
  const float* dlogits;
  const __bf16* w;
  const __bf16* x;
  const int32_t* slot_of;
  const uint8_t* valid;
  __bf16* dx;
  float* dw;
  float* part;         // [splits][d / 256][Ep][256] partial sums of dw
  uint64_t rows;
  uint32_t tokens, d, E;
  uint32_t splits;     // token ranges of dw
  uint32_t split_tokens;
  uint32_t col_groups; // workgroups that share the columns of dx
  bool whole_w;        // rows of w are whole aligned chunks of 8 experts
};

// Row loads bypass the caches (kStream) where the call's rows are twice the
// last-level cache (256 MiB) or more, so that none can still be there: combine,
// 131072 tokens x 1024, 260 us against 267 with plain loads, dispatch 228
// against 237; below, rows that the caches hold are read from them (16384 tokens:
// combine 36.3 us against 37.7, dispatch 51.3 against 54.2). Rows are always stored
// nontemporally: written plainly, they are written back during later reads
// (131072 tokens: combine 273 us, dispatch 239; 16384: 41.5 and 52.0). All are
// times of the whole call.
constexpr uint64_t kStreamBytes = 512ull << 20;

template <bool kStream, typename V>
__device__ __forceinline__ V load_row(const V* p) {
  if constexpr (kStream) return __builtin_nontemporal_load(p);
  return *p;
}

// Eight logit gradients as three bf16 terms each, of 8 of their 24 bits in turn:
// cut off, not rounded, so that the largest finite value does not become infinite
// and the last term holds what is left exactly. (The third term of a value below
// 2^-110 may fall under bf16's range; an infinite value leaves a NaN behind.)
__device__ __forceinline__ void split_terms(const float (&v)[8], bf16x8 (&terms)[3]) {
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = v[j];
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    u32x4 p;
#pragma unroll
    for (int j = 0; j < 4; ++j)  // the upper halves of two values
      p[j] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, r[2 * j + 1]), __builtin_bit_cast(uint32_t, r[2 * j]), 0x07060302u);
    terms[m] = __builtin_bit_cast(bf16x8, p);
    if (m == 2) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] -= __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r[j]) & 0xffff0000u);
  }
}

// ---- slot_of: the inverse of src_index ---------------------------------------

// Up to kSlotsInside tuples the combine's kernel inverts the index itself: each
// workgroup reads all of it and keeps, in LDS, the slots of its own tokens (on
// the GPU 300 tokens x 512: 3.6 us against 6.8 with two launches of its own,
// 4096 x 1024: 12.2 against 11.9, 8192 x 1024: 24 against 19).
constexpr uint32_t kSlotsInside = 8192;

__device__ __forceinline__ uint64_t kept_rows(const CombineGradArgs& a) {
  const int64_t n = a.offsets[a.E];
  return n < 0 ? 0 : min((uint64_t)n, a.rows);
}

__global__ __launch_bounds__(256) void k_slots_clear(CombineGradArgs a) {
  const uint32_t t = blockIdx.x * 256 + threadIdx.x;
  if (t < a.tokens) reinterpret_cast<int2*>(a.slot_of)[t] = int2{-1, -1};
}
__global__ __launch_bounds__(256) void k_slots_put(CombineGradArgs a) {
  const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= kept_rows(a)) return;
  const uint32_t g = (uint32_t)a.src_index[i];
  if (g < 2 * a.tokens) a.slot_of[g] = (int32_t)i;
}

// ---- gradient of the combine ---------------------------------------------------
// One wave handles kTokens tokens: their slots and gates in one round of loads,
// then every chunk of dout and of both y rows in flight before any is used (a
// dropped tuple reads row 0 and is masked). A workgroup takes its 8 tokens and
// ends: 131072 tokens x 1024, 254 us, 5.3 TB/s on random rows of 2 KiB, against
// 264 us with 2048 workgroups that walk the tokens. Bound by HBM.
constexpr int kTokens = 2;

template <bool kInside, bool kStream>  // kInside: the slots of the workgroup's 4 kTokens tokens are found here
__global__ __launch_bounds__(256) void k_combine_grad(CombineGradArgs a) {
  __shared__ int own[kInside ? 8 * kTokens : 1];
  if (kInside) {
    const uint32_t g0 = blockIdx.x * 8 * kTokens;  // the workgroup's first tuple
    if (threadIdx.x < 8 * kTokens) own[threadIdx.x] = -1;
    __syncthreads();
    const uint32_t n = (uint32_t)kept_rows(a);
    for (uint32_t i = threadIdx.x; i < n; i += 256) {
      const uint32_t g = (uint32_t)a.src_index[i] - g0;
      if (g < 8 * kTokens) own[g] = (int)i;
    }
    __syncthreads();
    if (threadIdx.x < 8 * kTokens && g0 + threadIdx.x < 2 * a.tokens) a.slot_of[g0 + threadIdx.x] = own[threadIdx.x];
  }
  const int lane = threadIdx.x & 63;
  const uint32_t nch = a.d / 8;  // 16-byte chunks of a row
  const u32x4* y = reinterpret_cast<const u32x4*>(a.y);
  const u32x4* dout = reinterpret_cast<const u32x4*>(a.dout);
  u32x4* dy = reinterpret_cast<u32x4*>(a.dy);
  for (uint32_t t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * kTokens; t0 < a.tokens; t0 += gridDim.x * 4 * kTokens) {
    int slot[kTokens][2];
    float gate[kTokens][2], dot[kTokens][2] = {};
    bool ok[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const uint32_t t = min(t0 + k, a.tokens - 1);
      int2 s;
      if (kInside) s = int2{own[(threadIdx.x >> 6) * 2 * kTokens + 2 * k], own[(threadIdx.x >> 6) * 2 * kTokens + 2 * k + 1]};
      else s = *reinterpret_cast<const int2*>(a.slot_of + (uint64_t)t * 2);
      const float2 g = *reinterpret_cast<const float2*>(a.gates + (uint64_t)t * 2);
      const int s0 = __builtin_amdgcn_readfirstlane(s.x), s1 = __builtin_amdgcn_readfirstlane(s.y);
      const bool here = t0 + k < a.tokens;
      ok[k] = !a.valid || a.valid[t];
      slot[k][0] = here ? s0 : -1;
      slot[k][1] = here ? s1 : -1;
      gate[k][0] = g.x;
      gate[k][1] = g.y;
    }
    for (uint32_t c0 = 0; c0 < nch; c0 += 128) {
      u32x4 vo[kTokens][2], vy[kTokens][2][2];  // [token][chunk], [token][tuple][chunk]
#pragma unroll
      for (int k = 0; k < kTokens; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t ch = min(c0 + lane + 64 * c, nch - 1);
          vo[k][c] = load_row<kStream>(dout + (uint64_t)min(t0 + k, a.tokens - 1) * nch + ch);
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (a.rows) vy[k][s][c] = load_row<kStream>(y + (uint64_t)max(slot[k][s], 0) * nch + ch);
        }
#pragma unroll
      for (int k = 0; k < kTokens; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t ch = c0 + lane + 64 * c;
          const bool in = ch < nch;
          const bf16x8 o = __builtin_bit_cast(bf16x8, vo[k][c]);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (slot[k][s] < 0) continue;  // wave-uniform
            const bf16x8 v = __builtin_bit_cast(bf16x8, vy[k][s][c]);
            bf16x8 r;
            float p = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              p = fmaf((float)o[j], (float)v[j], p);
              r[j] = ok[k] ? (__bf16)(gate[k][s] * (float)o[j]) : (__bf16)0.f;
            }
            if (in) {
              dot[k][s] += p;
              __builtin_nontemporal_store(__builtin_bit_cast(u32x4, r), dy + (uint64_t)slot[k][s] * nch + ch);
            }
          }
        }
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      dot[k][0] = lanes_sum<64>(dot[k][0]);
      dot[k][1] = lanes_sum<64>(dot[k][1]);
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k)
      if (lane == 0 && t0 + k < a.tokens) {
        const float2 r = {ok[k] && slot[k][0] >= 0 ? dot[k][0] : 0.f, ok[k] && slot[k][1] >= 0 ? dot[k][1] : 0.f};
        *reinterpret_cast<float2*>(a.dgates + (uint64_t)(t0 + k) * 2) = r;
      }
  }
}

// ---- gradient of dispatch and router, to the tokens ------------------------------
// A wave walks tiles of 16 tokens: dl W^T by v_mfma_f32_16x16x32_bf16 with the
// tokens as the first operand's rows, 128 columns of dx at a time. W lies in
// LDS in the order its operands are read (64 lanes of 16 bytes each). Column
// block b of the second operand holds every eighth column (8 n + b for lane
// n), so a lane's eight accumulators are 8 consecutive columns of its 4
// tokens, and rows of dxd and dx are read and written 16 bytes a lane, 256
// contiguous bytes a row. dl is split into three bf16 terms, which hold all 24
// bits of it: every product is exact and the sums are fp32 (with two terms 2^-16 of
// dl was lost, which shows where the terms of dx cancel; the whole call: 131072 x
// 1024 as long, 3000 x 1024 20.5 us against 21.0). 131072 tokens x 1024, 64 experts:
// 155 us, 5.4 TB/s, the rate of a large copy; bound by HBM. (W in registers,
// 128 columns a wave, 8 waves per CU: 223 us; one token a lane, 64 bytes of
// its row: 306 us.)
constexpr uint32_t kDxThreads = 1024;
constexpr uint32_t kDxWaves = kDxThreads / 64;
constexpr uint32_t kDxTokens = 16;
constexpr uint32_t kDxCols = 128;
constexpr uint32_t kDxGrid = 256;  // workgroups: one per CU

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4), aligned(4))) float f32x4_at4;  // loads of 16 bytes need 4-byte alignment

// Where the four inner positions from e on begin: experts past the last are
// reached by moving back (positions already covered get zeros of W), so that a
// row of dl is read in whole 16-byte loads, however many experts there are.
__device__ __forceinline__ uint32_t four_from(uint32_t e, uint32_t E) { return min(e, E - 4); }

// W[c] at the inner positions e0 .. e0 + 7, zero where there is no expert or
// an earlier position holds it.
template <bool kFour>
__device__ __forceinline__ bf16x8 load_w(const DispatchGradArgs& a, uint32_t c, uint32_t e0) {
  const __bf16* row = a.w + (uint64_t)c * a.E;
  bf16x8 v = {};
  if (a.whole_w) {  // uniform
    if (e0 < a.E) v = *reinterpret_cast<const bf16x8*>(row + e0);
    return v;
  }
  uint32_t at[8];
#pragma unroll
  for (uint32_t j = 0; j < 8; ++j) {
    const uint32_t e = e0 + (j & ~3u);
    at[j] = kFour ? four_from(e, a.E) + (j & 3) : min(e0 + j, a.E - 1);
    v[j] = row[at[j]];
  }
#pragma unroll
  for (uint32_t j = 0; j < 8; ++j)
    if (kFour ? at[j] < e0 + (j & ~3u) : e0 + j >= a.E) v[j] = (__bf16)0.f;
  return v;
}

template <int KS, bool kFour, bool kStream>  // steps of 32 experts; at least 4 experts
__global__ __launch_bounds__(kDxThreads) void k_dispatch_grad(DispatchGradArgs a) {
  extern __shared__ __attribute__((aligned(16))) bf16x8 lds_w[];  // [column block][b][s][64 lanes]
  const uint32_t lane = threadIdx.x & 63, i = lane & 15, h = lane >> 4;
  const uint32_t tiles = (a.tokens + kDxTokens - 1) / kDxTokens;
  const uint32_t blocks = a.d / kDxCols / a.col_groups, block0 = blockIdx.x % a.col_groups * blocks;
  const uint32_t streams = gridDim.x / a.col_groups * kDxWaves;
  for (uint32_t o = threadIdx.x; o < blocks * 8 * KS * 64; o += kDxThreads) {
    const uint32_t l = o & 63, f = o >> 6, s = f % KS, b = f / KS % 8, cb = block0 + f / (KS * 8);
    lds_w[o] = load_w<kFour>(a, cb * kDxCols + 8 * (l & 15) + b, 32 * s + 8 * (l >> 4));
  }
  __syncthreads();
  for (uint32_t tile = blockIdx.x / a.col_groups * kDxWaves + (threadIdx.x >> 6); tile < tiles; tile += streams) {
    // token i's logit gradients, experts 32 s + 8 h .. + 7, and its rows of dxd
    const uint32_t ti = min(tile * kDxTokens + i, a.tokens - 1);
    const int2 sl = *reinterpret_cast<const int2*>(a.slot_of + (uint64_t)ti * 2);
    const float* row = a.dlogits + (uint64_t)ti * a.E;
    bf16x8 dt[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t e0 = 32 * s + 8 * h;  // past the last expert: repeated values, against zeros of W
      float v[8];
      if (kFour) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f32x4 x = *reinterpret_cast<const f32x4_at4*>(row + four_from(e0 + 4 * q, a.E));
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * q + j] = x[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = row[min(e0 + j, a.E - 1)];
      }
      split_terms(v, dt[s]);
    }
    const bool pad = a.valid && !a.valid[ti];
    // of the lane's own 4 tokens (4 h + r): row, whether there is one, padding
    uint32_t src[2][4];
    uint32_t have = 0;  // bit 4 s + r; bit 8 + r: padding
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int v = __shfl(s ? sl.y : sl.x, 4 * h + r);
        const bool in = v >= 0 && (uint64_t)v < a.rows;
        have |= (in ? 1u : 0u) << (4 * s + r);
        src[s][r] = in ? (uint32_t)v : 0u;
      }
      have |= (__shfl((int)pad, 4 * h + r) ? 1u : 0u) << (8 + r);
    }
    const __bf16* dxd = a.dxd + block0 * kDxCols + 8 * i;
    __bf16* out = a.dx + ((uint64_t)tile * kDxTokens + 4 * h) * a.d + block0 * kDxCols + 8 * i;
    for (uint32_t cb = 0; cb < blocks; ++cb) {
      bf16x8 g[2][4];
      if (a.rows)  // uniform; a dropped tuple reads row 0, and does not use it
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            asm volatile("" : "+v"(src[s][r]));  // keeps the address out of registers between the column blocks
            g[s][r] = load_row<kStream>(reinterpret_cast<const bf16x8*>(dxd + (uint64_t)src[s][r] * a.d + cb * kDxCols));
          }
      f32x4 acc[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        acc[b] = f32x4{};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const bf16x8 w = lds_w[((cb * 8 + b) * KS + s) * 64 + lane];
#pragma unroll
          for (int m = 0; m < 3; ++m) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dt[s][m], w, acc[b], 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool have0 = have >> r & 1, have1 = have >> (4 + r) & 1, padding = have >> (8 + r) & 1;
        bf16x8 o;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          float f = acc[b][r];
          f += have0 ? (float)g[0][r][b] : 0.f;
          f += have1 ? (float)g[1][r][b] : 0.f;
          o[b] = (__bf16)(padding ? 0.f : f);
        }
        if (tile * kDxTokens + 4 * h + r < a.tokens)
          __builtin_nontemporal_store(o, reinterpret_cast<bf16x8*>(out + (uint64_t)r * a.d + cb * kDxCols));
      }
    }
  }
}

// ---- gradient of the router's weights --------------------------------------------
// dW = x^T dl over a range of tokens, by v_mfma_f32_32x32x16_bf16 with the
// tokens as the inner index. A lane needs 8 tokens of one column: it loads 4
// columns (8 bytes) of each of its 8 tokens and pairs the tokens with byte
// permutes, so operand q holds columns 4 i + q. dl is split into three bf16
// terms, which hold all 24 bits of it: every product is exact and the sums
// are fp32 (an infinite dl gives NaN). A workgroup covers 256 columns (2 waves
// of 128) with 4 waves of tokens each, joined through LDS in a fixed order.
// 131072 tokens x 1024, 64 experts: 57 to 72 us from one run to another (4.2-5.3
// TB/s), reading x and dl once from HBM; what makes the difference is not known.
// (Sharing the split terms between the waves through LDS, and requesting x two
// steps ahead, measured no faster.)
constexpr uint32_t kDwThreads = 512;
constexpr uint32_t kDwCols = 256;
constexpr int kNontemporal = 2;  // nt in the cache-policy operand of buffer instructions
// Tokens of a range at most: 768 additions to an accumulator, three for each 64
// tokens, so that the sums are as good for any batch (2^26 equal tokens x 256 in
// ranges of 2^18: off by 2.0e-4). A range's rows of x and dl are buffers below 2^31 bytes.
constexpr uint32_t kDwMaxTokens = 1u << 14;
constexpr uint32_t kDistant = 1u << 30;      // past the end of any range's dl, and below 2^32 with all that is added

template <int NC, bool kStream, bool kMasked>  // expert blocks of 32; kMasked: there is a mask
__global__ __launch_bounds__(kDwThreads) void k_router_dw(DispatchGradArgs a) {
  extern __shared__ __attribute__((aligned(16))) float lds[];  // [2][32 NC][kDwCols]
  constexpr uint32_t Ep = 32 * NC;
  const uint32_t lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = lane & 31, h = lane >> 5;
  const uint32_t groups = a.d / kDwCols;
  // the column groups of one token range run on one XCD (workgroup b runs on
  // XCD b mod 8) and share its L2 for dl
  const uint32_t k = blockIdx.x / 8, cg = k % groups, split = (k / groups) * 8 + blockIdx.x % 8;
  if (split >= a.splits) return;  // whole workgroups
  const uint32_t cw = w & 1, tw = w >> 1;
  const uint32_t first = split * a.split_tokens, last = min(first + a.split_tokens, a.tokens);
  f32x16 acc[4][NC];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[q][c] = f32x16{};
  struct Step {
    u32x2 v[8];        // 4 columns of 8 tokens
    float dl[NC][8];
    uint32_t valid[8];
  };
  // The range's rows of x and dl as buffers: past its end, and for experts
  // that are none (a distant offset), a load returns zero.
  const uint32_t n = last - first, xrow = a.d * 2, drow = a.E * 4;
  const auto xb = raw_buffer(a.x + (uint64_t)first * a.d, n * xrow);
  const auto db = raw_buffer(a.dlogits + (uint64_t)first * a.E, n * drow);
  const uint32_t xoff = (16 * tw + 8 * h) * xrow + (cg * kDwCols + cw * 128 + 4 * i) * 2;
  uint32_t doff[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) doff[c] = (16 * tw + 8 * h) * drow + (32 * c + i < a.E ? (32 * c + i) * 4 : kDistant);
  const auto vb = raw_buffer(kMasked ? a.valid + first : nullptr, kMasked ? n : 0);
  auto fetch = [&](Step& s, uint32_t t) {  // tokens t + 16 tw + 8 h + j of the range
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s.v[j] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(xb, xoff + (t + j) * xrow, 0, kStream ? kNontemporal : 0));
#pragma unroll
      for (int c = 0; c < NC; ++c)
        s.dl[c][j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(db, doff[c] + (t + j) * drow, 0, 0));
    }
    if (kMasked)  // a step ahead too (131072 tokens x 1024, the call: 221-224 us, looked up when needed 232-235)
#pragma unroll
      for (int j = 0; j < 8; ++j) s.valid[j] = __builtin_amdgcn_raw_buffer_load_b8(vb, t + 16 * tw + 8 * h + j, 0, 0);
  };
  // A step's operands are made from its loads, the next step's loads requested
  // into the same registers, and then its products run.
  Step s;
  fetch(s, 0);
  for (uint32_t t = 0; t < n; t += 64) {
    if (kMasked)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!s.valid[j]) {
          s.v[j] = u32x2{0, 0};
#pragma unroll
          for (int c = 0; c < NC; ++c) s.dl[c][j] = 0.f;
        }
    bf16x8 xa[4], dt[NC][3];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      u32x4 p;
#pragma unroll
      for (int j = 0; j < 4; ++j)  // halves q & 1 of tokens 2 j and 2 j + 1
        p[j] = __builtin_amdgcn_perm(s.v[2 * j + 1][q >> 1], s.v[2 * j][q >> 1], q & 1 ? 0x07060302u : 0x05040100u);
      xa[q] = __builtin_bit_cast(bf16x8, p);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) split_terms(s.dl[c], dt[c]);
    __builtin_amdgcn_sched_barrier(0);
    fetch(s, t + 64);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < 3; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[q][c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xa[q], dt[c][m], acc[q][c], 0, 0, 0);
  }
  // The token waves add up in two tables in LDS, [expert][256 columns]: 0 and 2
  // in one, 1 and 3 in the other. A lane's four operands of one register are 4
  // consecutive columns: 16-byte accesses, their chunks permuted by expert so
  // that 16 lanes meet 64 banks.
  auto chunk = [&](uint32_t table, uint32_t e, uint32_t c) {
    return reinterpret_cast<f32x4*>(lds + (table * Ep + e) * kDwCols + 4 * (c ^ (e & 15)));
  };
  for (uint32_t turn = 0; turn < 2; ++turn) {
    if (tw >> 1 == turn)
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          f32x4* p = chunk(tw & 1, 32 * c + i, cw * 32 + 8 * (r >> 2) + 4 * h + (r & 3));
          const f32x4 v = {acc[0][c][r], acc[1][c][r], acc[2][c][r], acc[3][c][r]};
          *p = turn ? *p + v : v;
        }
    __syncthreads();
  }
  if (a.splits == 1) {  // dw itself, an expert per lane
    for (uint32_t o = threadIdx.x; o < Ep * kDwCols; o += kDwThreads) {
      const uint32_t e = o % Ep, c = o / Ep;
      if (e >= a.E) continue;
      const float* p0 = reinterpret_cast<const float*>(chunk(0, e, c / 4)) + c % 4;
      const float* p1 = reinterpret_cast<const float*>(chunk(1, e, c / 4)) + c % 4;
      a.dw[(uint64_t)(cg * kDwCols + c) * a.E + e] = *p0 + *p1;
    }
    return;
  }
  float* part = a.part + ((uint64_t)split * groups + cg) * Ep * kDwCols;
  for (uint32_t o = threadIdx.x; o < Ep * kDwCols / 4; o += kDwThreads)
    *reinterpret_cast<f32x4*>(part + 4 * o) = *chunk(0, o / (kDwCols / 4), o % (kDwCols / 4)) +
                                              *chunk(1, o / (kDwCols / 4), o % (kDwCols / 4));
}

// Adds the partial sums of the token ranges: 64 columns of one expert per
// workgroup, 4 slices of the ranges, in a fixed order: up to 64 ranges of a slice
// in fp32, and these sums, whose number is not bounded, in double.
constexpr uint32_t kDwJoinRun = 64 * 4;

template <int NC>
__global__ __launch_bounds__(256) void k_router_dw_join(DispatchGradArgs a) {
  __shared__ float s[4][64];
  constexpr uint32_t Ep = 32 * NC;
  const uint32_t lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
  const uint32_t o = blockIdx.x * 64 + lane, e = o / kDwCols % Ep, col = o / (kDwCols * Ep) * kDwCols + o % kDwCols;
  if (e >= a.E) return;  // whole workgroups
  const uint64_t n = (uint64_t)a.d * Ep;
  double runs = 0.0;
  for (uint32_t i0 = 0; i0 < a.splits; i0 += kDwJoinRun) {
    const uint32_t end = min(i0 + kDwJoinRun, a.splits);
    float v = 0.f;
#pragma unroll 16
    for (uint32_t i = i0 + slice; i < end; i += 4) v += a.part[i * n + o];
    runs += (double)v;
  }
  s[slice][lane] = (float)runs;
  __syncthreads();
  if (slice == 0) a.dw[(uint64_t)col * a.E + e] = s[0][lane] + s[1][lane] + s[2][lane] + s[3][lane];
}

// Zeroes dw (a call without tokens).
__global__ __launch_bounds__(256) void k_router_dw_zero(DispatchGradArgs a) {
  const uint32_t o = blockIdx.x * 256 + threadIdx.x;
  if (o < a.d * a.E) a.dw[o] = 0.f;
}

constexpr size_t kDefaultLds = 64 << 10;  // what a kernel may use without asking
constexpr uint32_t kMaxD = 1280;          // width of a row at most

template <int KS, bool kFour, bool kStream>
hipError_t launch_dx_steps(const DispatchGradArgs& a, uint32_t grid, hipStream_t s) {
  const size_t lds = (size_t)a.d / a.col_groups * KS * 64;
  static_assert(kMaxD * 2 * 64 <= 160 << 10, "all of W in the LDS of a CU");
  if (lds > kDefaultLds) {
    const hipError_t e = hipFuncSetAttribute((const void*)k_dispatch_grad<KS, kFour, kStream>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_dispatch_grad<KS, kFour, kStream>), dim3(grid), dim3(kDxThreads), lds, s, a);
  return hipGetLastError();
}

template <int KS, bool kFour>
hipError_t launch_dx_loads(const DispatchGradArgs& a, uint32_t grid, bool stream, hipStream_t s) {
  return stream ? launch_dx_steps<KS, kFour, true>(a, grid, s) : launch_dx_steps<KS, kFour, false>(a, grid, s);
}

hipError_t launch_dx(DispatchGradArgs& a, bool stream, hipStream_t s) {
  const uint32_t tiles = (a.tokens + kDxTokens - 1) / kDxTokens, blocks = a.d / kDxCols;
  // With a tile for every wave of the GPU a workgroup keeps all of W and a wave
  // takes whole rows; below that the column blocks go to different workgroups.
  a.col_groups = tiles >= kDxGrid * kDxWaves ? 1 : blocks;
  const uint32_t most = kDxGrid * (a.col_groups > 1 ? 2 : 1) / a.col_groups;
  const uint32_t grid = std::min(most, (tiles + kDxWaves - 1) / kDxWaves) * a.col_groups;
  a.whole_w = a.E % 8 == 0 && !misaligned({a.w}, 16);
  if (a.E < 4) return launch_dx_loads<1, false>(a, grid, stream, s);
  return a.E <= 32 ? launch_dx_loads<1, true>(a, grid, stream, s) : launch_dx_loads<2, true>(a, grid, stream, s);
}

template <int NC, bool kStream, bool kMasked>
hipError_t launch_dw_loads(const DispatchGradArgs& a, uint32_t grid, hipStream_t s) {
  constexpr size_t lds = (size_t)2 * kDwCols * 32 * NC * 4;
  if (lds > kDefaultLds) {
    const hipError_t e = hipFuncSetAttribute((const void*)k_router_dw<NC, kStream, kMasked>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_router_dw<NC, kStream, kMasked>), dim3(grid), dim3(kDwThreads), lds, s, a);
  return hipGetLastError();
}

template <int NC, bool kMasked>
hipError_t launch_dw(const DispatchGradArgs& a, uint32_t grid, bool stream, hipStream_t s) {
  return stream ? launch_dw_loads<NC, true, kMasked>(a, grid, s) : launch_dw_loads<NC, false, kMasked>(a, grid, s);
}

struct DwLayout {
  uint32_t splits = 1, split_tokens = 64;
  size_t total = 0;
};

// Token ranges of dw: one workgroup per CU for long batches, two, three and so on
// for those whose ranges would pass kDwMaxTokens; short ones are cut into 16
// ranges of up to 256 tokens, as a range costs a partial sum of 64 KiB (3000 x
// 1024: 22.2 us the whole call against 25.2 with ranges of 64 tokens).
constexpr uint32_t kDwGrid = 256;
constexpr uint64_t kDwShort = 256;

DwLayout dw_layout(const pw_moe_grad_desc& d) {
  DwLayout l;
  const uint32_t groups = d.d / kDwCols;
  uint64_t want = std::max<uint64_t>(1, kDwGrid / groups);
  want *= std::max<uint64_t>(1, (d.tokens + want * kDwMaxTokens - 1) / (want * kDwMaxTokens));
  const uint64_t per = std::max((d.tokens + want - 1) / want, std::min(kDwShort, (d.tokens + 15) / 16));
  l.split_tokens = (uint32_t)std::max<uint64_t>(64, (per + 63) / 64 * 64);  // at most kDwMaxTokens
  l.splits = (uint32_t)std::max<uint64_t>(1, (d.tokens + l.split_tokens - 1) / l.split_tokens);
  if (l.splits > 1) l.total = up256((size_t)l.splits * d.d * (d.num_experts > 32 ? 64 : 32) * 4);
  return l;
}

int validate(const pw_moe_grad_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->tokens > (1ull << 28)) return fail(PW_ERR_INVALID, "tokens must be at most 2^28");
  if (d->rows > 2 * d->tokens) return fail(PW_ERR_INVALID, "rows must be at most 2 tokens");
  if (d->d == 0 || d->d % 256 || d->d > kMaxD)
    return fail(PW_ERR_INVALID, "d must be a positive multiple of 256, <= %u", kMaxD);
  if (d->num_experts < 2 || d->num_experts > 64) return fail(PW_ERR_INVALID, "num_experts must be in [2, 64]");
  if (d->top_k != 2) return fail(PW_ERR_UNSUPPORTED, "only top-2 routing is built");
  if (d->dtype != PW_BF16) return fail(PW_ERR_INVALID, "rows and weights are bf16");
  return PW_OK;
}

}  // namespace

}  // namespace pw

using namespace pw;

extern "C" int pw_moe_combine_grad(const pw_moe_grad_desc* d, const pw_combine_grad_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->tokens == 0) return PW_OK;
  if (!io->dout || !io->gates || !io->offsets || !io->dgates || !io->slot_of)
    return fail(PW_ERR_INVALID, "dout, gates, offsets, dgates and slot_of are required");
  if (d->rows && (!io->y || !io->src_index || !io->dy)) return fail(PW_ERR_INVALID, "y, src_index and dy are required");
  if (misaligned({io->dout, io->y, io->dy}, 16)) return fail(PW_ERR_INVALID, "row buffers must be 16-byte aligned");
  if (misaligned({io->gates, io->dgates, io->slot_of, io->offsets}, 8) || misaligned({io->src_index}, 4))
    return fail(PW_ERR_INVALID, "gates, dgates, slot_of and offsets must be 8-byte aligned, src_index 4-byte");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  CombineGradArgs a{};
  a.dout = static_cast<const __bf16*>(io->dout);
  a.y = static_cast<const __bf16*>(io->y);
  a.gates = io->gates;
  a.src_index = io->src_index;
  a.offsets = io->offsets;
  a.valid = io->valid;
  a.dy = static_cast<__bf16*>(io->dy);
  a.dgates = io->dgates;
  a.slot_of = io->slot_of;
  a.rows = d->rows;
  a.tokens = (uint32_t)d->tokens;
  a.d = d->d;
  a.E = d->num_experts;
  hipError_t e;
  const uint32_t per = 4 * kTokens;
  if (2 * a.tokens <= kSlotsInside) {
    hipLaunchKernelGGL((k_combine_grad<true, false>), dim3((a.tokens + per - 1) / per), dim3(256), 0, s, a);
    e = hipGetLastError();
    return e == hipSuccess ? PW_OK : hip_fail(e, "launch combine_grad");
  }
  hipLaunchKernelGGL(k_slots_clear, dim3((a.tokens + 255) / 256), dim3(256), 0, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "launch slots_clear");
  if (a.rows) {
    hipLaunchKernelGGL(k_slots_put, dim3((uint32_t)((a.rows + 255) / 256)), dim3(256), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "launch slots_put");
  }
  const dim3 grid(std::min((a.tokens + per - 1) / per, kMaxGrid));
  if (((uint64_t)a.tokens + 2 * a.rows) * a.d * 2 >= kStreamBytes)
    hipLaunchKernelGGL((k_combine_grad<false, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_combine_grad<false, false>), grid, dim3(256), 0, s, a);
  e = hipGetLastError();
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch combine_grad");
}

extern "C" int pw_moe_dispatch_grad_workspace(const pw_moe_grad_desc* d, size_t* bytes) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!bytes) return fail(PW_ERR_INVALID, "bytes is NULL");
  *bytes = dw_layout(*d).total;
  return PW_OK;
}

extern "C" int pw_moe_dispatch_grad(const pw_moe_grad_desc* d, const pw_dispatch_grad_io* io, void* ws, size_t ws_bytes,
                                    void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (d->tokens && (!io->dlogits || !io->w_router || !io->slot_of || !io->dx))
    return fail(PW_ERR_INVALID, "dlogits, w_router, slot_of and dx are required");
  if (d->rows && !io->dxd) return fail(PW_ERR_INVALID, "dxd is required");
  if (d->tokens && io->dw_router && !io->x) return fail(PW_ERR_INVALID, "dw_router needs x");
  if (misaligned({io->dxd, io->x, io->dx}, 16)) return fail(PW_ERR_INVALID, "row buffers must be 16-byte aligned");
  if (misaligned({io->slot_of}, 8) || misaligned({io->dlogits, io->dw_router}, 4) || misaligned({io->w_router}, 2))
    return fail(PW_ERR_INVALID, "slot_of must be 8-byte aligned, dlogits and dw_router 4-byte, w_router 2-byte");
  const DwLayout l = dw_layout(*d);
  if (io->dw_router && (st = check_workspace(ws, ws_bytes, l.total))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  DispatchGradArgs a{};
  a.dxd = static_cast<const __bf16*>(io->dxd);
  a.dlogits = io->dlogits;
  a.w = static_cast<const __bf16*>(io->w_router);
  a.x = static_cast<const __bf16*>(io->x);
  a.slot_of = io->slot_of;
  a.valid = io->valid;
  a.dx = static_cast<__bf16*>(io->dx);
  a.dw = io->dw_router;
  a.part = static_cast<float*>(ws);
  a.rows = d->rows;
  a.tokens = (uint32_t)d->tokens;
  a.d = d->d;
  a.E = d->num_experts;
  a.splits = l.splits;
  a.split_tokens = l.split_tokens;
  const bool stream_rows = ((uint64_t)a.tokens * (a.dw ? 2 : 1) + a.rows) * a.d * 2 >= kStreamBytes;
  hipError_t e;
  if (a.tokens == 0) {
    if (!a.dw) return PW_OK;
    hipLaunchKernelGGL(k_router_dw_zero, dim3((a.d * a.E + 255) / 256), dim3(256), 0, s, a);
    e = hipGetLastError();
    return e == hipSuccess ? PW_OK : hip_fail(e, "launch router_dw_zero");
  }
  if ((e = launch_dx(a, stream_rows, s)) != hipSuccess) return hip_fail(e, "launch dispatch_grad");
  if (!a.dw) return PW_OK;
  const bool two = a.E > 32;
  const uint32_t grid = 8 * (a.d / kDwCols) * ((a.splits + 7) / 8);
  if (two) e = a.valid ? launch_dw<2, true>(a, grid, stream_rows, s) : launch_dw<2, false>(a, grid, stream_rows, s);
  else e = a.valid ? launch_dw<1, true>(a, grid, stream_rows, s) : launch_dw<1, false>(a, grid, stream_rows, s);
  if (e != hipSuccess) return hip_fail(e, "launch router_dw");
  if (a.splits > 1) {
    const uint32_t jb = a.d * (two ? 64 : 32) / 64;
    if (two) hipLaunchKernelGGL(k_router_dw_join<2>, dim3(jb), dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_router_dw_join<1>, dim3(jb), dim3(256), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "launch router_dw_join");
  }
  return PW_OK;
}
