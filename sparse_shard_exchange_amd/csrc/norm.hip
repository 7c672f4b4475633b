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
// A row lives in the registers of its team (one wave for narrow rows, the
// whole workgroup for wide ones) from its only read to its only write, so the
// passes move 4 and 6 row tensors and nothing else; the bound is HBM.
#include "ops.h"

#include <algorithm>

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxWidth = 8192;

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
  uint32_t seg_rows;   // rows of a segment; segments do not cross groups
  uint32_t segs;       // segments of a group
  uint32_t num_segs;   // groups x segs
  uint32_t grid;       // workgroups of k_norm_grad
  float x_scale, y_scale, eps, inv_d;
};

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

// One chunk of a row: 16 bytes, or one element where rows are not 16-byte
// aligned. Kept as loaded until it is used.
template <typename T, int V>
struct Chunk;
template <>
struct Chunk<__bf16, 8> { bf16x8 q; };
template <>
struct Chunk<float, 4> { f32x4 q; };
template <typename T>
struct Chunk<T, 1> { T q; };

template <typename T, int V>
__device__ __forceinline__ Chunk<T, V> load(const void* base, uint64_t off) {
  return *reinterpret_cast<const Chunk<T, V>*>(static_cast<const T*>(base) + off);
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
template <typename T, int V>
__device__ __forceinline__ void store(void* base, uint64_t off, const Chunk<T, V>& c) {
  *reinterpret_cast<Chunk<T, V>*>(static_cast<T*>(base) + off) = c;
}

// Sums a and b over the team; every thread of the team gets both. Teams of a
// workgroup exchange through LDS (two barriers: before the first write the
// previous sums have been read).
template <int TEAM>
__device__ __forceinline__ void team_sum(float& a, float& b, float (*red)[2]) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    a += __shfl_xor(a, m);
    b += __shfl_xor(b, m);
  }
  if constexpr (TEAM > 64) {
    __syncthreads();
    if (threadIdx.x % 64 == 0) {
      red[threadIdx.x / 64][0] = a;
      red[threadIdx.x / 64][1] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < TEAM / 64; ++w) {
      a += red[w][0];
      b += red[w][1];
    }
  }
}

// C chunks of V elements per thread of a team of TEAM threads.
template <typename T, int V, int C, int TEAM, bool kY, bool kH>
__global__ __launch_bounds__(kThreads) void k_norm(NormArgs a) {
  __shared__ float red[kThreads / 64][2];
  const uint32_t lane = threadIdx.x % TEAM, nch = a.d / V;
  constexpr uint32_t kTeams = kThreads / TEAM;
  const bool norm_y = kY && a.w_y, gated = kY && a.gate;
  // the trip count is the same for all threads of a workgroup (barriers inside)
  for (uint32_t row0 = blockIdx.x * kTeams; row0 < a.rows; row0 += gridDim.x * kTeams) {
    const uint32_t row = row0 + threadIdx.x / TEAM;
    const bool live = row < a.rows;
    const uint64_t base = (uint64_t)(live ? row : a.rows - 1) * a.d;
    Chunk<T, V> x[C], y[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t ch = min(lane + c * TEAM, nch - 1);
      x[c] = load<T, V>(a.x, base + (uint64_t)ch * V);
      if (kY) y[c] = load<T, V>(a.y, base + (uint64_t)ch * V);
    }
    float ty = a.y_scale;
    if (norm_y) {
      float ss = 0.f, none = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane + c * TEAM < nch)
#pragma unroll
          for (int v = 0; v < V; ++v) ss = fmaf(at<T, V>(y[c], v), at<T, V>(y[c], v), ss);
      team_sum<TEAM>(ss, none, red);
      ty = a.y_scale * rsqrtf(fmaf(ss, a.inv_d, a.eps));
    }
    const uint64_t gbase = gated ? (uint64_t)((live ? row : a.rows - 1) / a.group) * a.d : 0;
    float r[C][V], ss = 0.f, none = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t ch = min(lane + c * TEAM, nch - 1);
      Chunk<T, V> wy, g;
      if (norm_y) wy = load<T, V>(a.w_y, (uint64_t)ch * V);
      if (gated) g = load<T, V>(a.gate, gbase + (uint64_t)ch * V);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f = a.x_scale * at<T, V>(x[c], v);
        if (kY) {
          float n = ty * at<T, V>(y[c], v);
          if (norm_y) n *= at<T, V>(wy, v);
          f = gated ? fmaf(n, at<T, V>(g, v), f) : f + n;
        }
        r[c][v] = f;
        if (kH && lane + c * TEAM < nch) ss = fmaf(f, f, ss);
      }
    }
    float s = 0.f;
    if (kH) {
      team_sum<TEAM>(ss, none, red);
      s = rsqrtf(fmaf(ss, a.inv_d, a.eps));
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t ch = lane + c * TEAM;
      if (!live || ch >= nch) continue;
      Chunk<T, V> o;
      if (a.r) {
#pragma unroll
        for (int v = 0; v < V; ++v) put<T, V>(o, v, r[c][v]);
        store<T, V>(a.r, base + (uint64_t)ch * V, o);
      }
      if (kH) {
        const Chunk<T, V> w = load<T, V>(a.w_r, (uint64_t)ch * V);
#pragma unroll
        for (int v = 0; v < V; ++v) put<T, V>(o, v, r[c][v] * s * at<T, V>(w, v));
        store<T, V>(a.h, base + (uint64_t)ch * V, o);
      }
    }
  }
}

// Backward. The rows are cut into segments of consecutive rows of one gate
// group; a workgroup walks segments, its teams taking the segment's rows in
// turn, and keeps in registers, for its columns, the running sums of D y t
// (Q, until the end of the segment) and dh r s (W, until its own end). At a
// segment's end Q goes, summed over the teams, to dgate where the segment is
// the whole group, else to part_q; and gate Q to the running sum P of dw_y.
// W and P end in one partial row per workgroup; k_norm_join adds the rows.
template <typename T, int V, int C, int TEAM, bool kY, bool kH>
__global__ __launch_bounds__(kThreads) void k_norm_grad(NormArgs a) {
  extern __shared__ float lds[];  // TEAM 64: [teams][d] sums of the teams
  __shared__ float red[kThreads / 64][2];
  const uint32_t lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM, nch = a.d / V;
  constexpr uint32_t kTeams = kThreads / TEAM;
  constexpr int kOwn = (C * V * TEAM + kThreads - 1) / kThreads;  // columns of a thread at the end of a segment
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
    if constexpr (TEAM == kThreads) return (lane + (i / V) * TEAM) * V + i % V;
    return threadIdx.x + i * kThreads;
  };
  auto gather = [&](const float (&s)[C][V], float (&out)[kOwn]) {
    if constexpr (TEAM == kThreads) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) out[i] = s[i / V][i % V];
    } else {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane + c * TEAM < nch)
#pragma unroll
          for (int v = 0; v < V; ++v) lds[team * a.d + (lane + c * TEAM) * V + v] = s[c][v];
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
    const uint32_t lo = k * a.seg_rows, hi = min(lo + a.seg_rows, a.group);  // rows of the group
    const uint64_t gbase = (uint64_t)g * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int v = 0; v < V; ++v) Q[c][v] = 0.f;
    for (uint32_t i0 = lo; i0 < hi; i0 += kTeams) {
      const bool live = i0 + team < hi;
      const uint64_t row = (uint64_t)g * a.group + (live ? i0 + team : hi - 1), base = row * a.d;
      const bool ok = live && (!a.valid || a.valid[row]);
      Chunk<T, V> dr[C], dh[C], r[C], y[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint64_t o = base + (uint64_t)min(lane + c * TEAM, nch - 1) * V;
        if (a.dr) dr[c] = load<T, V>(a.dr, o);
        if (kH) {
          dh[c] = load<T, V>(a.dh, o);
          r[c] = load<T, V>(a.r_in, o);
        }
        if (kY) y[c] = load<T, V>(a.y, o);
      }
      float D[C][V];
      float rr = 0.f, gr = 0.f, yy = 0.f, none = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool in = lane + c * TEAM < nch;
        Chunk<T, V> w;
        if (kH) w = load<T, V>(a.w_r, (uint64_t)min(lane + c * TEAM, nch - 1) * V);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (kH) {
            D[c][v] = at<T, V>(dh[c], v) * at<T, V>(w, v);
            if (in) {
              rr = fmaf(at<T, V>(r[c], v), at<T, V>(r[c], v), rr);
              gr = fmaf(D[c][v], at<T, V>(r[c], v), gr);
            }
          }
          if (norm_y && in) yy = fmaf(at<T, V>(y[c], v), at<T, V>(y[c], v), yy);
        }
      }
      float s = 0.f, m = 0.f, t = 1.f;
      if (kH) {
        team_sum<TEAM>(rr, gr, red);
        s = rsqrtf(fmaf(rr, a.inv_d, a.eps));
        m = s * s * gr * a.inv_d;
      }
      if (norm_y) {
        team_sum<TEAM>(yy, none, red);
        t = rsqrtf(fmaf(yy, a.inv_d, a.eps));
      }
      float qy = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t ch = lane + c * TEAM;
        const bool in = ok && ch < nch;
        Chunk<T, V> o, wy, gt;
        if (norm_y) wy = load<T, V>(a.w_y, (uint64_t)min(ch, nch - 1) * V);
        if (gated) gt = load<T, V>(a.gate, gbase + (uint64_t)min(ch, nch - 1) * V);
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
              if (ch < nch) qy = fmaf(f, yv, qy);
            }
          }
          D[c][v] = f;
        }
        if (live && ch < nch) store<T, V>(a.dx, base + (uint64_t)ch * V, o);
      }
      if (kY) {
        float m2 = 0.f;
        if (norm_y) {
          team_sum<TEAM>(qy, none, red);
          m2 = t * t * qy * a.inv_d;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t ch = lane + c * TEAM;
          if (!live || ch >= nch) continue;
          Chunk<T, V> o;
#pragma unroll
          for (int v = 0; v < V; ++v)
            put<T, V>(o, v, !ok ? 0.f : norm_y ? t * (D[c][v] - at<T, V>(y[c], v) * m2) : D[c][v]);
          store<T, V>(a.dy, base + (uint64_t)ch * V, o);
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

// Adds the partial rows: blockIdx.y 0: dw_r, 1: dw_y, 2 + g: dgate of group
// g. 64 columns per workgroup, 16 slices of rows, added in a fixed order.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_join(NormArgs a) {
  __shared__ float s[16][64];
  const uint32_t c = threadIdx.x % 64, slice = threadIdx.x / 64, col = blockIdx.x * 64 + c;
  const uint32_t what = blockIdx.y;
  const float* part = what == 0 ? a.part_w : what == 1 ? a.part_p : a.part_q + (uint64_t)(what - 2) * a.segs * a.d;
  const uint32_t n = what < 2 ? a.grid : a.segs;
  if ((what == 0 && !a.dw_r) || (what == 1 && !a.dw_y)) return;
  float v = 0.f;
  if (col < a.d)
    for (uint32_t i = slice; i < n; i += 16) v += part[(uint64_t)i * a.d + col];
  s[slice][c] = v;
  __syncthreads();
  if (slice != 0 || col >= a.d) return;
  v = 0.f;
  for (int i = 0; i < 16; ++i) v += s[i][c];
  if (what == 0) a.dw_r[col] = v;
  else if (what == 1) a.dw_y[col] = v * a.y_scale;
  else a.dgate[(uint64_t)(what - 2) * a.d + col] = v * a.y_scale * (a.w_y ? (float)static_cast<const T*>(a.w_y)[col] : 1.f);
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
// per row. One wave per row while the row fits 4 chunks a lane (no barrier in
// the row sums), else the workgroup. Rows that are not whole aligned 16-byte
// chunks go by single elements.
struct Shape {
  int V, C, team;
};

Shape shape_of(uint32_t d, bool f32, bool aligned) {
  const int V = aligned ? (f32 ? 4 : 8) : 1;
  const uint32_t nch = d / V;
  if (V > 1) {
    if (nch <= 64) return {V, 1, 64};
    if (nch <= 128) return {V, 2, 64};
    if (nch <= 256) return {V, 4, 64};
    if (nch <= 512) return {V, 2, 256};
    if (nch <= 1024) return {V, 4, 256};
    return {V, 8, 256};
  }
  if (nch <= 256) return {1, 4, 64};
  if (nch <= 2048) return {1, 8, 256};
  return {1, 32, 256};
}

struct Segments {
  uint32_t group, segs, seg_rows, num_segs, grid;
};

constexpr uint32_t kSegments = 1024;  // segments wanted: 4 workgroups per CU

// Enough segments to fill the GPU, none below 16 rows where a group has more.
Segments segments(uint32_t rows, uint32_t gates) {
  Segments s;
  const uint32_t groups = std::max(1u, gates);
  s.group = rows / groups;
  const uint32_t want = std::max(1u, kSegments / groups);
  s.seg_rows = std::max((s.group + want - 1) / want, std::min(s.group, 16u));
  s.segs = (s.group + s.seg_rows - 1) / s.seg_rows;
  s.num_segs = s.segs * groups;
  s.grid = std::min(s.num_segs, kSegments);
  return s;
}

struct GradLayout {
  size_t w = 0, p = 0, q = 0, total = 0;
};

GradLayout grad_layout(const pw_norm_desc& d) {
  GradLayout l;
  if (d.rows == 0) return l;
  const Segments s = segments((uint32_t)d.rows, d.gates);
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
  return PW_OK;
}

bool aligned16(std::initializer_list<const void*> ps) {
  uintptr_t v = 0;
  for (const void* p : ps) v |= (uintptr_t)p;
  return v % 16 == 0;
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

constexpr uint32_t kForwardGrid = 256 * 16;  // workgroups of k_norm at most

template <typename T, int V, int C, int TEAM, bool kY, bool kH>
void launch(const NormArgs& a, bool grad, hipStream_t s) {
  if (grad) {
    const size_t lds = TEAM < kThreads ? (size_t)(kThreads / TEAM) * a.d * 4 : 0;
    hipLaunchKernelGGL((k_norm_grad<T, V, C, TEAM, kY, kH>), dim3(a.grid), dim3(kThreads), lds, s, a);
  } else {
    const uint32_t teams = kThreads / TEAM;
    const uint32_t blocks = (uint32_t)std::min<uint64_t>(((uint64_t)a.rows + teams - 1) / teams, kForwardGrid);
    hipLaunchKernelGGL((k_norm<T, V, C, TEAM, kY, kH>), dim3(blocks), dim3(kThreads), 0, s, a);
  }
}

template <typename T, int V, int C, int TEAM>
void launch_parts(const NormArgs& a, bool grad, hipStream_t s) {
  if (!a.y) launch<T, V, C, TEAM, false, true>(a, grad, s);
  else if (!a.w_r) launch<T, V, C, TEAM, true, false>(a, grad, s);
  else launch<T, V, C, TEAM, true, true>(a, grad, s);
}

template <typename T, int V>
void launch_shape(const NormArgs& a, const Shape& sh, bool grad, hipStream_t s) {
  if constexpr (V > 1) {
    if (sh.team == 64) {
      if (sh.C == 1) launch_parts<T, V, 1, 64>(a, grad, s);
      else if (sh.C == 2) launch_parts<T, V, 2, 64>(a, grad, s);
      else launch_parts<T, V, 4, 64>(a, grad, s);
    } else {
      if (sh.C == 2) launch_parts<T, V, 2, 256>(a, grad, s);
      else if (sh.C == 4) launch_parts<T, V, 4, 256>(a, grad, s);
      else if constexpr (V == 4) launch_parts<T, V, 8, 256>(a, grad, s);  // 8192 fp32; bf16 ends at 4
    }
  } else {
    if (sh.team == 64) launch_parts<T, 1, 4, 64>(a, grad, s);
    else if (sh.C == 8) launch_parts<T, 1, 8, 256>(a, grad, s);
    else launch_parts<T, 1, 32, 256>(a, grad, s);
  }
}

hipError_t launch_any(const NormArgs& a, const pw_norm_desc& d, bool aligned, bool grad, hipStream_t s) {
  const bool f32 = d.dtype == PW_F32;
  const Shape sh = shape_of(d.d, f32, aligned && (uint64_t)d.d * (f32 ? 4 : 2) % 16 == 0);
  if (f32) sh.V > 1 ? launch_shape<float, 4>(a, sh, grad, s) : launch_shape<float, 1>(a, sh, grad, s);
  else sh.V > 1 ? launch_shape<__bf16, 8>(a, sh, grad, s) : launch_shape<__bf16, 1>(a, sh, grad, s);
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
  const hipError_t e = launch_any(a, *d, aligned16({a.x, a.y, a.w_y, a.gate, a.w_r, a.r, a.h}), false, s);
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
  const Segments sg = segments(a.rows, a.gates);
  a.group = sg.group;
  a.segs = sg.segs;
  a.seg_rows = sg.seg_rows;
  a.num_segs = sg.num_segs;
  a.grid = sg.grid;
  unsigned char* base = static_cast<unsigned char*>(ws);
  if (l.total) {
    a.part_w = reinterpret_cast<float*>(base + l.w);
    a.part_p = reinterpret_cast<float*>(base + l.p);
    a.part_q = reinterpret_cast<float*>(base + l.q);
  }
  // without a next norm the gradient of h plays no part
  e = launch_any(a, *d, aligned16({a.y, a.w_y, a.gate, a.w_r, a.w_r ? a.r_in : nullptr, a.dr, a.w_r ? a.dh : nullptr,
                                   a.dx, a.dy}), true, s);
  if (e != hipSuccess) return hip_fail(e, "launch norm_grad");
  const bool gates = a.gate && a.segs > 1;
  if ((a.grid > 1 && (a.dw_r || a.dw_y)) || gates) {
    const dim3 grid((a.d + 63) / 64, 2 + (gates ? a.gates : 0));
    if (d->dtype == PW_F32) hipLaunchKernelGGL(k_norm_join<float>, grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL(k_norm_join<__bf16>, grid, dim3(1024), 0, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return hip_fail(e, "launch norm_join");
  }
  return PW_OK;
}
