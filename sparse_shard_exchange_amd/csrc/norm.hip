// Norms around a block, fused with its gate and residual scale, forward and
// backward. One pass closes a block (norm of its output, gate, residual) and
// opens the next (norm of the new residual stream):
//
//   N(v; w) = v s(v) w,  s(v) = 1 / sqrt(mean(v^2) + eps)
//   r = ax x + ay gate N(y; wy)          h = N(r; wr)
//
// and back, with G = dh wr, s = s(r), t = s(y):
//
//   D  = dr + s (G - r s^2 mean(G r))    dx = ax D
//   q  = ay D gate wy                    dy = t (q - y t^2 mean(q y))
//   Q_g = sum over g's rows of D y t     dgate_g = ay wy Q_g
//   dwy = ay sum_g gate_g Q_g            dwr = sum dh r s
//
// A row lives in the registers of its team (16 lanes up to 128 elements, up to
// 16 waves for the widest) from its only read to its only write, so the passes
// move 4 and 6 row tensors and nothing else; the bound is HBM. 131072 x 1024
// bf16, all parts: forward 178 us (6.0 TB/s), backward 307 + 11.6 us (5.2 TB/s in
// the first); a large copy reaches 5.2. Rows are stored nontemporally: written
// plainly, they are written back during the next operator's reads (forward and
// backward in turn, 131072 rows 493 us against 508, 32768 rows 142 against 146,
// 16384 rows 86.8 against 87.7). They are loaded plainly: nontemporal loads take
// 4% less in the gradient from 65536 rows on (131072: 306 us against 318), as long
// or up to 17% more below (forward 16384 rows 25.4 against 21.7, gradient 4096 rows
// 21.6 against 19.4).
#include "ops.h"

#include <algorithm>

namespace pw {

namespace {

constexpr int kThreads = 256;  // of a workgroup, or a wider team's
constexpr uint32_t kMaxWidth = 8192;
constexpr int threads_of(int team) { return team > kThreads ? team : kThreads; }

struct NormArgs {
  const void* x;
  const void* y;
  const void* w_y;
  const void* gate;
  const void* w_r;
  const void* r_in;
  void* r;
  void* h;
  const void* dr;
  const void* dh;
  const uint8_t* valid;
  void* dx;
  void* dy;
  float* dw_y;
  float* dgate;
  float* dw_r;
  float* part_w;   // [grid][d] partial sums of dw_r
  float* part_p;   // [grid][d] partial sums of dw_y / ay
  float* part_q;   // [segments][d] sums of D y t of each segment
  uint32_t rows, d, gates;
  uint32_t group;      // rows that share a gate row (rows if there is one gate or none)
  uint32_t segs;       // segments of a group: every segs-th turn of its rows
  uint32_t num_segs;   // groups x segs
  uint32_t grid;       // workgroups of k_norm_grad
  uint32_t joins;      // results k_norm_join looks at: dw_r, dw_y, then gates
  float x_scale, y_scale, eps, inv_d;
};

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// One chunk of a row: 16 bytes, or one element where a row is shorter. Kept as
// loaded until it is used. At: the chunk in memory, aligned to its elements.
template <typename T, int V>
struct Chunk;
template <>
struct Chunk<__bf16, 8> {
  typedef __attribute__((ext_vector_type(8), aligned(2))) __bf16 At;
  bf16x8 q;
};
template <>
struct Chunk<float, 4> {
  typedef __attribute__((ext_vector_type(4), aligned(4))) float At;
  f32x4 q;
};
template <typename T>
struct Chunk<T, 1> {
  typedef T At;
  T q;
};

template <typename T, int V, bool kWhole>
__device__ __forceinline__ Chunk<T, V> load(const void* base, uint64_t off) {
  const T* p = static_cast<const T*>(base) + off;
  if constexpr (kWhole) return *reinterpret_cast<const Chunk<T, V>*>(p);
  return {*reinterpret_cast<const typename Chunk<T, V>::At*>(p)};
}
template <typename T, int V>
__device__ __forceinline__ float at(const Chunk<T, V>& c, int v) {
  if constexpr (V == 1) return (float)c.q;
  else return (float)c.q[v];
}
template <typename T, int V>
__device__ __forceinline__ void put(Chunk<T, V>& c, int v, float f) {
  if constexpr (V == 1) c.q = (T)f;
  else c.q[v] = (T)f;
}

// A row's chunks. Rows that are whole aligned chunks (kWhole) have no rest; in
// others the last chunk is moved back to end with the row, and its first `over`
// elements are those of the chunk before it (131072 x 1023 bf16, all parts, in
// 16-byte accesses at any alignment: forward 182 us, backward 338, by single
// elements 270 and 471). No sum sees them twice. Chunks of 8 write them twice (kTwice), with
// the same bits; chunks of 4, two or four of them a thread and fewer registers
// left, zero them after the load and store their own elements one by one
// (backward, this way against the other: 131072 x 1023 bf16 341 us against 370,
// 4000 x 3001 fp32 65 against 100).
template <typename T, int V, bool kWhole>
struct Row {
  static constexpr bool kTwice = !kWhole && V == 8;
  uint32_t d, nch, over;
  __device__ __forceinline__ explicit Row(uint32_t d) : d(d), nch(kWhole ? d / V : (d + V - 1) / V), over(nch * V - d) {}
  __device__ __forceinline__ uint32_t start(uint32_t ch) const { return kWhole ? ch * V : min(ch * V, d - V); }
  __device__ __forceinline__ Chunk<T, V> load_chunk(const void* base, uint64_t row, uint32_t ch) const {
    return load<T, V, kWhole>(base, row + start(min(ch, nch - 1)));
  }
  // Element v of chunk ch, d where it is none.
  __device__ __forceinline__ uint32_t column(uint32_t ch, uint32_t v) const {
    const uint32_t c = start(ch) + v;
    return kWhole || c >= ch * V ? c : d;
  }
  __device__ __forceinline__ bool again(uint32_t ch, uint32_t v) const { return !kWhole && ch + 1 == nch && v < over; }
  // After the load of a chunk whose values are summed.
  __device__ __forceinline__ void clip(Chunk<T, V>& c, uint32_t ch) const {
    if constexpr (!kWhole && !kTwice) {
      if (ch + 1 != nch) return;
#pragma unroll
      for (uint32_t v = 0; v < V; ++v)
        if (v < over) put<T, V>(c, v, 0.f);
    }
  }
  // Element v of chunk ch as sums take it.
  __device__ __forceinline__ float own(float f, uint32_t ch, uint32_t v) const { return kTwice && again(ch, v) ? 0.f : f; }
  __device__ __forceinline__ void store_chunk(void* base, uint64_t row, uint32_t ch, const Chunk<T, V>& c) const {
    T* p = static_cast<T*>(base) + row + start(ch);
    if constexpr (V == 1) {
      *p = c.q;
    } else if constexpr (kWhole) {
      __builtin_nontemporal_store(c.q, reinterpret_cast<decltype(Chunk<T, V>::q)*>(p));
    } else if (kTwice || ch + 1 != nch || over == 0) {
      const typename Chunk<T, V>::At q = c.q;
      __builtin_nontemporal_store(q, reinterpret_cast<typename Chunk<T, V>::At*>(p));
    } else {
#pragma unroll
      for (uint32_t v = 0; v < V; ++v)
        if (!again(ch, v)) p[v] = c.q[v];
    }
  }
};

// A chunk of a row vector that every row uses (a weight or a gate). Chunks of
// bf16 the compiler may keep in registers for all rows; wider elements are
// loaded again for each row, from the caches (the empty asm statement hides
// that the address is the same): as many more registers would halve the waves.
template <typename T, int V, bool kWhole>
__device__ __forceinline__ Chunk<T, V> load_shared(const Row<T, V, kWhole>& R, const void* p, uint64_t row, uint32_t ch) {
  if constexpr (V < 8) asm volatile("" : "+s"(p));
  return R.load_chunk(p, row, ch);
}

// The waves' sums of one exchange, by wave. A workgroup alternates between two
// of them, so one barrier an exchange is enough: whoever writes one again has
// passed the barrier of the other, which every wave reaches after it has read
// the first.
template <int TEAM>
struct Exchange {
  float sums[2][threads_of(TEAM) / 64][3];
};

// Sums N values over the team; every thread of the team gets them.
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], Exchange<TEAM>& x, uint32_t& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum<(TEAM < 64 ? TEAM : 64)>(v[i]);
  if constexpr (TEAM > 64) {
    constexpr int W = TEAM / 64;
    auto& sums = x.sums[turn];
    turn ^= 1;
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sums[threadIdx.x / 64][i] = v[i];
    __syncthreads();
    const int w = threadIdx.x / TEAM * W + threadIdx.x % W;  // each lane a wave's sums, then across W lanes
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<W>(sums[w][i]);
  }
}

// C chunks of V elements per thread of a team of TEAM threads; a workgroup takes
// one row per team and ends (131072 x 1024 bf16: 178 us; walking the rows with
// 4096 workgroups 200, with 1024 224: rows that run at the same time are
// neighbours, and the next workgroup's loads overlap this one's stores).
template <typename T, int V, bool kWhole, int C, int TEAM, bool kY, bool kH>
__global__ __launch_bounds__(threads_of(TEAM)) void k_norm(NormArgs a) {
  __shared__ Exchange<TEAM> ex;
  uint32_t turn = 0;
  const Row<T, V, kWhole> R(a.d);
  const uint32_t lane = threadIdx.x % TEAM, nch = R.nch;
  constexpr uint32_t kTeams = threads_of(TEAM) / TEAM;
  const bool norm_y = kY && a.w_y, gated = kY && a.gate;
  for (uint32_t row0 = blockIdx.x * kTeams; row0 < a.rows; row0 += gridDim.x * kTeams) {  // (one turn: see kMaxGrid)
    const uint32_t row = row0 + threadIdx.x / TEAM;
    const bool live = row < a.rows;  // every thread stays: barriers inside
    const uint64_t base = (uint64_t)min(row, a.rows - 1) * a.d;
    const uint64_t gbase = gated ? (uint64_t)(min(row, a.rows - 1) / a.group) * a.d : 0;
    Chunk<T, V> x[C], y[C], wy[C], g[C], wr[C];  // all requested before any is used
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t ch = lane + c * TEAM;
      x[c] = R.load_chunk(a.x, base, ch);
      if (kY) y[c] = R.load_chunk(a.y, base, ch);
      if (norm_y) wy[c] = R.load_chunk(a.w_y, 0, ch);
      if (gated) g[c] = R.load_chunk(a.gate, gbase, ch);
      if (kH) wr[c] = R.load_chunk(a.w_r, 0, ch);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      R.clip(x[c], lane + c * TEAM);
      if (kY) R.clip(y[c], lane + c * TEAM);
    }
    float ty = a.y_scale;
    if (norm_y) {
      float ss[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane + c * TEAM < nch)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float yv = R.own(at<T, V>(y[c], v), lane + c * TEAM, v);
            ss[0] = fmaf(yv, yv, ss[0]);
          }
      team_sum(ss, ex, turn);
      ty = a.y_scale * rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
    }
    float r[C][V], ss[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f = a.x_scale * at<T, V>(x[c], v);
        if (kY) {
          float n = ty * at<T, V>(y[c], v);
          if (norm_y) n *= at<T, V>(wy[c], v);
          f = gated ? fmaf(n, at<T, V>(g[c], v), f) : f + n;
        }
        r[c][v] = f;
        if (kH && lane + c * TEAM < nch) {
          const float rv = R.own(f, lane + c * TEAM, v);
          ss[0] = fmaf(rv, rv, ss[0]);
        }
      }
    }
    float s = 0.f;
    if (kH) {
      team_sum(ss, ex, turn);
      s = rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
    }
    if (R.kTwice && TEAM > 64 && !kH && !norm_y) __syncthreads();  // uniform; see k_norm_grad
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t ch = lane + c * TEAM;
      if (!live || ch >= nch) continue;
      Chunk<T, V> o;
      if (a.r) {
#pragma unroll
        for (int v = 0; v < V; ++v) put<T, V>(o, v, r[c][v]);
        R.store_chunk(a.r, base, ch, o);
      }
      if (kH) {
#pragma unroll
        for (int v = 0; v < V; ++v) put<T, V>(o, v, r[c][v] * s * at<T, V>(wr[c], v));
        R.store_chunk(a.h, base, ch, o);
      }
    }
  }
}

// Backward. The rows of a gate group are dealt to its segments in turn (a row
// for each team, segment after segment), so that workgroups running at the same
// time read neighbouring rows. A workgroup walks segments and keeps in
// registers, for its columns, the running sums of D y t (Q, until the end of
// the segment) and dh r s (W, until its own end). At a segment's end Q goes,
// summed over the teams, to dgate where the segment is the whole group, else to
// part_q; and gate Q to the running sum P of dw_y. W and P end in one partial
// row per workgroup; k_norm_join adds the rows.
template <typename T, int V, bool kWhole, int C, int TEAM, bool kY, bool kH>
__global__ __launch_bounds__(threads_of(TEAM), C * V > 8 ? 2 : 4) void k_norm_grad(NormArgs a) {
  constexpr int NT = threads_of(TEAM);
  extern __shared__ float lds[];  // several teams: [teams][d] their sums
  __shared__ Exchange<TEAM> ex;
  uint32_t turn = 0;
  const Row<T, V, kWhole> R(a.d);
  const uint32_t lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM, nch = R.nch;
  constexpr uint32_t kTeams = NT / TEAM;
  constexpr int kOwn = C * V < (int)kTeams ? 1 : C * V / (int)kTeams;  // columns of a thread at the end of a segment
  const bool norm_y = kY && a.w_y, gated = kY && a.gate, sums_y = norm_y || gated;
  float Q[C][V], W[C][V], P[kOwn];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int v = 0; v < V; ++v) W[c][v] = 0.f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) P[i] = 0.f;

  // Column i of this thread at a segment's end, and its sum over the teams.
  auto column = [&](int i) -> uint32_t {
    if constexpr (kTeams == 1) return R.column(lane + (i / V) * TEAM, i % V);
    return threadIdx.x + i * NT;
  };
  auto gather = [&](const float (&s)[C][V], float (&out)[kOwn]) {
    if constexpr (kTeams == 1) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) out[i] = s[i / V][i % V];
    } else {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane + c * TEAM < nch)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const uint32_t col = R.column(lane + c * TEAM, v);
            if (kWhole || col < a.d) lds[team * a.d + col] = s[c][v];
          }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        out[i] = 0.f;
        if (column(i) < a.d)
          for (uint32_t t = 0; t < kTeams; ++t) out[i] += lds[t * a.d + column(i)];
      }
    }
  };

  for (uint32_t sg = blockIdx.x; sg < a.num_segs; sg += gridDim.x) {
    const uint32_t g = sg / a.segs, k = sg % a.segs;
    const uint64_t gbase = (uint64_t)g * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int v = 0; v < V; ++v) Q[c][v] = 0.f;
    for (uint32_t i0 = k * kTeams; i0 < a.group; i0 += a.segs * kTeams) {
      const bool live = i0 + team < a.group;
      const uint64_t row = (uint64_t)g * a.group + min(i0 + team, a.group - 1), base = row * a.d;
      const bool ok = live && (!a.valid || a.valid[row]);
      Chunk<T, V> dr[C], dh[C], r[C], y[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t ch = lane + c * TEAM;
        if (a.dr) dr[c] = R.load_chunk(a.dr, base, ch);
        if (kH) {
          dh[c] = R.load_chunk(a.dh, base, ch);
          r[c] = R.load_chunk(a.r_in, base, ch);
        }
        if (kY) y[c] = R.load_chunk(a.y, base, ch);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (kH) R.clip(r[c], lane + c * TEAM);
        if (kY) R.clip(y[c], lane + c * TEAM);
      }
      float D[C][V];
      float sum[3] = {0.f, 0.f, 0.f};  // r^2, G r, y^2
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool in = lane + c * TEAM < nch;
        Chunk<T, V> w;
        if (kH) w = load_shared(R, a.w_r, 0, lane + c * TEAM);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (kH) {
            D[c][v] = at<T, V>(dh[c], v) * at<T, V>(w, v);
            if (in) {
              const float rv = R.own(at<T, V>(r[c], v), lane + c * TEAM, v);
              sum[0] = fmaf(rv, rv, sum[0]);
              sum[1] = fmaf(D[c][v], rv, sum[1]);
            }
          }
          if (norm_y && in) {
            const float yv = R.own(at<T, V>(y[c], v), lane + c * TEAM, v);
            sum[2] = fmaf(yv, yv, sum[2]);
          }
        }
      }
      float s = 0.f, m = 0.f, t = 1.f;
      // An element that two waves hold (kTwice) is written in place when both
      // have read it: the sums' barrier, or this one.
      if (kH || norm_y) team_sum(sum, ex, turn);  // uniform
      else if (R.kTwice && TEAM > 64) __syncthreads();
      if (kH) {
        s = rsqrtf(fmaf(sum[0], a.inv_d, a.eps));
        m = s * sum[1] * (s * a.inv_d);  // (s may be too large for its square)
      }
      if (norm_y) t = rsqrtf(fmaf(sum[2], a.inv_d, a.eps));
      float qy[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t ch = lane + c * TEAM;
        const bool in = ok && ch < nch;
        Chunk<T, V> o, wy, gt;
        if (norm_y) wy = load_shared(R, a.w_y, 0, ch);
        if (gated) gt = load_shared(R, a.gate, gbase, ch);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f = a.dr ? at<T, V>(dr[c], v) : 0.f;
          if (kH) {
            const float rv = at<T, V>(r[c], v);
            f = fmaf(s, D[c][v] - rv * m, f);
            if (in) W[c][v] = fmaf(at<T, V>(dh[c], v), rv * s, W[c][v]);
          }
          put<T, V>(o, v, ok ? a.x_scale * f : 0.f);
          if (kY) {
            const float yv = at<T, V>(y[c], v);
            if (sums_y && in) Q[c][v] = fmaf(f, yv * t, Q[c][v]);
            f *= a.y_scale;
            if (gated) f *= at<T, V>(gt, v);
            if (norm_y) {
              f *= at<T, V>(wy, v);
              if (ch < nch) qy[0] = fmaf(f, R.own(yv, ch, v), qy[0]);
            }
          }
          D[c][v] = f;
        }
        if (live && ch < nch) R.store_chunk(a.dx, base, ch, o);
      }
      if (kY) {
        float m2 = 0.f;
        if (norm_y) {
          team_sum(qy, ex, turn);
          m2 = t * qy[0] * (t * a.inv_d);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t ch = lane + c * TEAM;
          if (!live || ch >= nch) continue;
          Chunk<T, V> o;
#pragma unroll
          for (int v = 0; v < V; ++v)
            put<T, V>(o, v, !ok ? 0.f : norm_y ? t * (D[c][v] - at<T, V>(y[c], v) * m2) : D[c][v]);
          R.store_chunk(a.dy, base, ch, o);
        }
      }
    }
    if (sums_y) {
      float q[kOwn];
      gather(Q, q);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const uint32_t col = column(i);
        if (col >= a.d) continue;
        if (norm_y) P[i] += gated ? q[i] * (float)static_cast<const T*>(a.gate)[gbase + col] : q[i];
        if (gated) {
          if (a.segs == 1)
            a.dgate[gbase + col] = q[i] * a.y_scale * (norm_y ? (float)static_cast<const T*>(a.w_y)[col] : 1.f);
          else
            a.part_q[(uint64_t)sg * a.d + col] = q[i];
        }
      }
    }
  }
  float w[kOwn];
  if (kH) gather(W, w);
  const bool whole = gridDim.x == 1;  // nothing to join
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const uint32_t col = column(i);
    if (col >= a.d) continue;
    const uint64_t o = whole ? col : (uint64_t)blockIdx.x * a.d + col;
    if (kH) (whole ? a.dw_r : a.part_w)[o] = w[i];
    if (norm_y) (whole ? a.dw_y : a.part_p)[o] = whole ? P[i] * a.y_scale : P[i];
  }
}

// Adds the partial rows: 0: dw_r, 1: dw_y, 2 + g: dgate of group g. 32 columns
// per workgroup, 32 slices of rows, added in a fixed order: up to 64 rows of a
// slice in fp32, and these sums, whose number is not bounded, in double.
constexpr uint32_t kJoinCols = 32, kJoinSlices = 1024 / kJoinCols, kJoinRun = 64 * kJoinSlices;
constexpr uint32_t kMaxGridY = 65535;

template <typename T>
__global__ __launch_bounds__(1024) void k_norm_join(NormArgs a) {
  __shared__ float s[kJoinSlices][kJoinCols];
  const uint32_t c = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols, col = blockIdx.x * kJoinCols + c;
  const uint32_t what = blockIdx.z * gridDim.y + blockIdx.y;
  if (what >= a.joins || (what == 0 && !a.dw_r) || (what == 1 && !a.dw_y)) return;  // whole workgroups
  const float* part = what == 0 ? a.part_w : what == 1 ? a.part_p : a.part_q + (uint64_t)(what - 2) * a.segs * a.d;
  const uint32_t n = what < 2 ? a.grid : a.segs;
  double runs = 0.0;
  if (col < a.d)
    for (uint32_t i0 = 0; i0 < n; i0 += kJoinRun) {
      const uint32_t end = min(i0 + kJoinRun, n);
      float v = 0.f;
#pragma unroll 16
      for (uint32_t i = i0 + slice; i < end; i += kJoinSlices) v += part[(uint64_t)i * a.d + col];
      runs += (double)v;
    }
  s[slice][c] = (float)runs;
  __syncthreads();
  if (slice != 0 || col >= a.d) return;
  float v = 0.f;
#pragma unroll
  for (uint32_t i = 0; i < kJoinSlices; ++i) v += s[i][c];
  if (what == 0) a.dw_r[col] = v;
  else if (what == 1) a.dw_y[col] = v * a.y_scale;
  else
    a.dgate[(uint64_t)(what - 2) * a.d + col] =
        v * a.y_scale * (a.w_y ? (float)static_cast<const T*>(a.w_y)[col] : 1.f);
}

// Zeroes the parameter gradients of a call without rows.
__global__ __launch_bounds__(kThreads) void k_norm_zero(NormArgs a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.d) return;
  if (a.dw_r) a.dw_r[i] = 0.f;
  if (a.dw_y) a.dw_y[i] = 0.f;
  if (a.dgate)
    for (uint32_t g = 0; g < a.gates; ++g) a.dgate[(uint64_t)g * a.d + i] = 0.f;
}

// The kernel variant of a row: elements per chunk, chunks per thread, threads
// per row. At most 8 elements a thread, so that the gradient's registers (rows,
// sums, weights) leave room for 4 waves per SIMD (2047 x 1001 fp32 by 256
// threads with room for 8 elements each, half of it unused: 42 us against 16).
// Narrow rows share a wave, 4 or 2 at a time (300000 x 128 bf16, all parts: forward
// 53.5 us, backward 95; with a wave for each row 109 and 202).
// Above 4096 elements fp32 rows take 16 elements by 512 threads: 1024 threads of
// 8 spill (backward, 8192 x 8192: 570 us against 405; for bf16, whose chunks are
// half as wide in registers, it is the other way round, 477 against 505; both
// before the rows were dealt in turn). Rows shorter than a chunk go by single
// elements.
struct Shape {
  int V, C, team;
};

Shape shape_of(uint32_t d, bool f32) {
  const int V = f32 ? 4 : 8;
  if (d < (uint32_t)V) return {1, 1, 16};
  if (d > 4096) return V == 8 ? Shape{8, 1, 1024} : Shape{V, 16 / V, 512};
  if (d > 2048) return {V, 8 / V, 512};
  if (d > 1024) return {V, 8 / V, 256};
  if (d > 512) return {V, 8 / V, 128};
  if (d > 256) return {V, 8 / V, 64};
  if (d > 128) return {V, 8 / V, 32};
  return {V, 8 / V, 16};
}

// Rows a workgroup takes at a time.
uint32_t teams_of(uint32_t d) {
  const uint32_t team = shape_of(d, false).team;  // (fp32: as many teams)
  return threads_of(team) / team;
}

struct Segments {
  uint32_t group, segs, num_segs, grid;
};

// Segments wanted: 8 workgroups per CU for long batches (131072 x 1024 bf16 back:
// 318 us with the join, with 1024 segments 338: the second half of the
// workgroups starts as the first ends, and evens out their ends), 4 where a
// workgroup takes one row at a time (16384 x 8192: 422 and 373 us); for short
// batches up to 512 of up to 8 rows, since a segment's partial sums (two or three fp32 rows
// written and read back) weigh against its rows, and a row's turn is a few
// memory latencies (backward, bf16: 64 x 1024 8.2 us with 4 rows a segment, 7.1
// with 2; 4096 x 1024 20.2 with 4, 18.3 with 8; 64 x 8192 25.8 and 20.0 with 4
// and 2).
// However many rows there are, a workgroup takes kTurns turns of its teams or little
// more (twice as many where the groups divide badly), so that no fp32 chain of the
// weights' sums gets longer: 2^29 equal rows of 8 elements, 16384 turns, left dw_y
// off by 9e-5.
constexpr uint32_t kSegments = 2048;
constexpr uint32_t kTurns = 512;
constexpr uint32_t kShortSegments = 512;
constexpr uint32_t kShortRows = 8;

Segments segments(uint32_t rows, uint32_t gates, uint32_t d) {
  Segments s;
  const uint32_t groups = std::max(1u, gates);
  s.group = rows / groups;
  const uint32_t teams = teams_of(d);
  const uint64_t turns = (uint64_t)groups * ((s.group + teams - 1) / teams);
  const uint32_t most = std::max(teams > 1 ? kSegments : kSegments / 2,
                                 (uint32_t)std::min<uint64_t>((turns + kTurns - 1) / kTurns, kMaxGrid));
  const uint32_t want = std::max(1u, most / groups);
  uint32_t short_rows = teams;  // a power of two: whole turns of the teams
  while (short_rows < kShortRows && (uint64_t)short_rows * kShortSegments < rows) short_rows *= 2;
  const uint32_t seg_rows = std::max((s.group + want - 1) / want, std::min(s.group, short_rows));
  s.segs = (s.group + seg_rows - 1) / seg_rows;
  s.num_segs = s.segs * groups;
  s.grid = std::min(s.num_segs, most);
  return s;
}

struct GradLayout {
  size_t w = 0, p = 0, q = 0, total = 0;
};

GradLayout grad_layout(const pw_norm_desc& d) {
  GradLayout l;
  if (d.rows == 0) return l;
  const Segments s = segments((uint32_t)d.rows, d.gates, d.d);
  const size_t row = (size_t)d.d * 4;
  if (s.grid > 1) {
    l.p = up256(s.grid * row);
    l.q = 2 * l.p;
    l.total = l.q;
  }
  if (d.gates && s.segs > 1) l.total = l.q + up256((size_t)s.num_segs * row);
  return l;
}

int validate(const pw_norm_desc* d) {
  if (!d) return fail(PW_ERR_INVALID, "descriptor is NULL");
  if (d->rows > 0x7fffffffull) return fail(PW_ERR_INVALID, "rows must be at most 2^31 - 1");
  if (d->d < 1 || d->d > kMaxWidth) return fail(PW_ERR_INVALID, "d must be in [1, %u]", kMaxWidth);
  if (d->dtype != PW_F32 && d->dtype != PW_BF16) return fail(PW_ERR_INVALID, "unknown dtype %u", d->dtype);
  if (d->gates && d->rows % d->gates) return fail(PW_ERR_INVALID, "rows must be a multiple of gates");
  if (d->gates > 0x7fffffffu) return fail(PW_ERR_INVALID, "gates must be at most 2^31 - 1");
  if (!isfinite(d->x_scale) || !isfinite(d->y_scale)) return fail(PW_ERR_INVALID, "the scales must be finite");
  if (!isfinite(d->eps) || d->eps <= 0.f) return fail(PW_ERR_INVALID, "eps must be finite and above zero");
  return PW_OK;
}

int validate_parts(const pw_norm_desc& d, const pw_norm_io* io) {
  if (!io) return fail(PW_ERR_INVALID, "io is NULL");
  if (!io->y && (io->w_y || io->gate)) return fail(PW_ERR_INVALID, "w_y and gate need y");
  if (!io->gate != !d.gates) return fail(PW_ERR_INVALID, "gate is given if and only if gates is above zero");
  if (!io->y && !io->w_r) return fail(PW_ERR_INVALID, "nothing to do: neither y nor w_r is given");
  if (misaligned({io->x, io->y, io->w_y, io->gate, io->w_r, io->r, io->h, io->dr, io->dh, io->dx, io->dy},
                 d.dtype == PW_F32 ? 4 : 2) || misaligned({io->dw_y, io->dgate, io->dw_r}, 4))
    return fail(PW_ERR_INVALID, "a buffer is not aligned to its elements");
  return PW_OK;
}

NormArgs args(const pw_norm_desc& d, const pw_norm_io& io) {
  NormArgs a{};
  a.x = io.x;
  a.y = io.y;
  a.w_y = io.w_y;
  a.gate = io.gate;
  a.w_r = io.w_r;
  a.r_in = io.r;
  a.r = io.r;
  a.h = io.h;
  a.dr = io.dr;
  a.dh = io.dh;
  a.valid = io.valid;
  a.dx = io.dx;
  a.dy = io.dy;
  a.dw_y = io.w_y ? io.dw_y : nullptr;
  a.dgate = io.gate ? io.dgate : nullptr;
  a.dw_r = io.w_r ? io.dw_r : nullptr;
  a.rows = (uint32_t)d.rows;
  a.d = d.d;
  a.gates = d.gates;
  a.x_scale = d.x_scale;
  a.y_scale = d.y_scale;
  a.eps = d.eps;
  a.inv_d = 1.0f / (float)d.d;
  a.group = std::max(1u, a.rows / std::max(1u, d.gates));
  return a;
}

template <typename T, int V, bool kWhole, int C, int TEAM, bool kY, bool kH>
void launch(const NormArgs& a, bool grad, hipStream_t s) {
  constexpr uint32_t NT = threads_of(TEAM), teams = NT / TEAM;
  if (grad) {
    const size_t lds = teams > 1 ? (size_t)teams * a.d * 4 : 0;
    hipLaunchKernelGGL((k_norm_grad<T, V, kWhole, C, TEAM, kY, kH>), dim3(a.grid), dim3(NT), lds, s, a);
  } else {
    const uint32_t blocks = std::min((a.rows + teams - 1) / teams, kMaxGrid);
    hipLaunchKernelGGL((k_norm<T, V, kWhole, C, TEAM, kY, kH>), dim3(blocks), dim3(NT), 0, s, a);
  }
}

template <typename T, int V, bool kWhole, int C, int TEAM>
void launch_parts(const NormArgs& a, bool grad, hipStream_t s) {
  if (!a.y) launch<T, V, kWhole, C, TEAM, false, true>(a, grad, s);
  else if (!a.w_r) launch<T, V, kWhole, C, TEAM, true, false>(a, grad, s);
  else launch<T, V, kWhole, C, TEAM, true, true>(a, grad, s);
}

template <typename T, int V, bool kWhole>
void launch_shape(const NormArgs& a, const Shape& sh, bool grad, hipStream_t s) {
  switch (sh.team) {
    case 1024:
      if constexpr (V == 8) return launch_parts<T, 8, kWhole, 1, 1024>(a, grad, s);
    case 512:
      if constexpr (V < 8)
        if (sh.C * V == 16) return launch_parts<T, V, kWhole, 16 / V, 512>(a, grad, s);
      return launch_parts<T, V, kWhole, 8 / V, 512>(a, grad, s);
    case 256: return launch_parts<T, V, kWhole, 8 / V, 256>(a, grad, s);
    case 128: return launch_parts<T, V, kWhole, 8 / V, 128>(a, grad, s);
    case 64: return launch_parts<T, V, kWhole, 8 / V, 64>(a, grad, s);
    case 32: return launch_parts<T, V, kWhole, 8 / V, 32>(a, grad, s);
  }
  launch_parts<T, V, kWhole, 8 / V, 16>(a, grad, s);
}

template <typename T, int V>
void launch_type(const NormArgs& a, const Shape& sh, bool aligned, bool grad, hipStream_t s) {
  if (sh.V == 1) launch_parts<T, 1, true, 1, 16>(a, grad, s);
  else if (aligned && a.d % V == 0) launch_shape<T, V, true>(a, sh, grad, s);
  else launch_shape<T, V, false>(a, sh, grad, s);
}

hipError_t launch_any(const NormArgs& a, const pw_norm_desc& d, bool aligned, bool grad, hipStream_t s) {
  const bool f32 = d.dtype == PW_F32;
  const Shape sh = shape_of(d.d, f32);
  if (f32) launch_type<float, 4>(a, sh, aligned, grad, s);
  else launch_type<__bf16, 8>(a, sh, aligned, grad, s);
  return hipGetLastError();
}

}  // namespace

}  // namespace pw

using namespace pw;

extern "C" int pw_block_norm(const pw_norm_desc* d, const pw_norm_io* io, void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if ((st = validate_parts(*d, io))) return st;
  if (!io->r && !io->w_r) return fail(PW_ERR_INVALID, "nothing to write: neither r nor w_r is given");
  if (!io->w_r != !io->h) return fail(PW_ERR_INVALID, "h and w_r are given together or not at all");
  if (d->rows == 0) return PW_OK;
  if (!io->x) return fail(PW_ERR_INVALID, "x is required");
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  const NormArgs a = args(*d, *io);
  const hipError_t e = launch_any(a, *d, !misaligned({a.x, a.y, a.w_y, a.gate, a.w_r, a.r, a.h}, 16), false, s);
  return e == hipSuccess ? PW_OK : hip_fail(e, "launch norm");
}

extern "C" int pw_block_norm_grad_workspace(const pw_norm_desc* d, size_t* bytes) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if (!bytes) return fail(PW_ERR_INVALID, "bytes is NULL");
  *bytes = grad_layout(*d).total;
  return PW_OK;
}

extern "C" int pw_block_norm_grad(const pw_norm_desc* d, const pw_norm_io* io, void* ws, size_t ws_bytes,
                                  void* stream) {
  clear_error();
  int st = validate(d);
  if (st) return st;
  if ((st = validate_parts(*d, io))) return st;
  if (io->w_y && !io->dw_y) return fail(PW_ERR_INVALID, "w_y needs dw_y");
  if (io->gate && !io->dgate) return fail(PW_ERR_INVALID, "gate needs dgate");
  if (io->w_r && !io->dw_r) return fail(PW_ERR_INVALID, "w_r needs dw_r");
  if (d->rows && io->w_r && (!io->dh || !io->r)) return fail(PW_ERR_INVALID, "w_r needs dh and r");
  if (d->rows && !io->w_r && !io->dr) return fail(PW_ERR_INVALID, "without w_r, dr is required");
  if (d->rows && !io->dx) return fail(PW_ERR_INVALID, "dx is required");
  if (d->rows && io->y && !io->dy) return fail(PW_ERR_INVALID, "y needs dy");
  const GradLayout l = grad_layout(*d);
  if ((st = check_workspace(ws, ws_bytes, l.total))) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = check_stream(s))) return st;
  NormArgs a = args(*d, *io);
  hipError_t e;
  if (a.rows == 0) {
    hipLaunchKernelGGL(k_norm_zero, dim3((a.d + kThreads - 1) / kThreads), dim3(kThreads), 0, s, a);
    e = hipGetLastError();
    return e == hipSuccess ? PW_OK : hip_fail(e, "launch norm_zero");
  }
  const Segments sg = segments(a.rows, a.gates, a.d);
  a.group = sg.group;
  a.segs = sg.segs;
  a.num_segs = sg.num_segs;
  a.grid = sg.grid;
  unsigned char* base = static_cast<unsigned char*>(ws);
  if (l.total) {
    a.part_w = reinterpret_cast<float*>(base + l.w);
    a.part_p = reinterpret_cast<float*>(base + l.p);
    a.part_q = reinterpret_cast<float*>(base + l.q);
  }
  // without a next norm the gradient of h plays no part
  const bool aligned = !misaligned({a.y, a.w_y, a.gate, a.w_r, a.w_r ? a.r_in : nullptr, a.dr,
                                    a.w_r ? a.dh : nullptr, a.dx, a.dy}, 16);
  e = launch_any(a, *d, aligned, true, s);
  if (e != hipSuccess) return hip_fail(e, "launch norm_grad");
  const bool gates = a.gate && a.segs > 1;
  if ((a.grid > 1 && (a.dw_r || a.dw_y)) || gates) {
    a.joins = 2 + (gates ? a.gates : 0);
    const dim3 grid((a.d + kJoinCols - 1) / kJoinCols, std::min(a.joins, kMaxGridY), (a.joins + kMaxGridY - 1) / kMaxGridY);
    if (d->dtype == PW_F32) hipLaunchKernelGGL(k_norm_join<float>, grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL(k_norm_join<__bf16>, grid, dim3(1024), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "launch norm_join");
  }
  return PW_OK;
}
