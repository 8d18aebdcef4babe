// gdr_linear_scan.hip -- gated linear recurrence of one decay per channel and
// token: prompts, gradient, single tokens.
//
//   e = sigmoid(r),  a = exp(A e),  m = sqrt(1 - a^2),  b = m sigmoid(i) x
//   h_t = a_t h_{t-1} + b_t,  y_t = h_t
//
// The token axis is cut into tiles of TOK tokens.  Over any run of tokens the
// state changes by h -> P h + S (P the product of the run's decays, S its end
// state from zero), and two runs one behind the other by P = P2 P1, S = P2 S1
// + S2: waves take TT tokens each, meet in LDS, and tiles meet in memory.  A
// run that starts or ends a sequence does not depend on what is before it:
// its P is kFresh, and S stands alone (a product with zero would carry a NaN
// of another sequence over).
#include "gdr_layer.h"

namespace gdr {

constexpr float kFresh = -1.f;   // in the place of a product of decays: the end does not depend on the start
constexpr int kLinVec = 4;       // channels a lane
constexpr int kLinCh = 64 * kLinVec;

// sqrt(1 - a^2) with a = exp(s), s = s2 ln 2: 1 - a^2 = -expm1(2 s).  Near zero
// the difference would lose all bits: below 2 |s| = 1/4 the Taylor series up to
// z^6 / 720 (the next term is 4.8e-8 of the first); above it 1 - a^2 >= 0.22.
// A positive s gives a NaN.
__device__ __forceinline__ float lin_factor(float s2, float a) {
  const float z = s2 * 1.3862943611198906f;
  float q = fmaf(z, 1.f / 720.f, 1.f / 120.f);
  q = fmaf(q, z, 1.f / 24.f);
  q = fmaf(q, z, 1.f / 6.f);
  q = fmaf(q, z, 0.5f);
  q = fmaf(q, z, 1.f);
  return __builtin_amdgcn_sqrtf(z > -0.25f ? -z * q : fmaf(-a, a, 1.f));
}
// a and b of one value; A2 = A log2(e)
__device__ __forceinline__ void lin_gates(float x, float r, float i, float A2, float& a, float& b) {
  const float s2 = A2 * sigmoid_f(r);
  a = __builtin_amdgcn_exp2f(s2);
  b = lin_factor(s2, a) * sigmoid_f(i) * x;
}
// sigmoid(x) and 1 - sigmoid(x), both to a few ulps on either side of zero
__device__ __forceinline__ void sigmoid_both(float x, float& e, float& ne) {
  const float t = exp_f(-fabsf(x)), big = __builtin_amdgcn_rcpf(1.f + t), small = t * big;
  e = x >= 0.f ? big : small;
  ne = x >= 0.f ? small : big;
}

// The runs of a wave's TT tokens, in scalar registers.
template <int TT>
__device__ __forceinline__ TokenRuns lin_runs(const SeqFinder& sf, int t0) {
  TokenRuns m = token_runs(sf, t0, TT);
  m.first = __builtin_amdgcn_readfirstlane(m.first);
  m.last = __builtin_amdgcn_readfirstlane(m.last);
  m.gap = __builtin_amdgcn_readfirstlane(m.gap);
  return m;
}
__device__ __forceinline__ int lin_seq_at(const SeqFinder& sf, int t) {
  int start, end;
  return __builtin_amdgcn_readfirstlane(sf.find(t, start, end));
}

// TT tokens of a strided operand from token t0 on, four channels a lane; rows
// behind the last are the last one.
template <typename T, int TT>
__device__ __forceinline__ void lin_load(const void* base, long stride, int t0, int Ttot, int d, int nd, bool full,
                                         typename VecIO<T, kLinVec>::raw (&out)[TT]) {
  const T* p = static_cast<const T*>(base) + d;
  if (full) {
#pragma unroll
    for (int k = 0; k < TT; ++k)
      out[k] = *reinterpret_cast<const typename VecIO<T, kLinVec>::raw*>(p + (long)min(t0 + k, Ttot - 1) * stride);
  } else {
#pragma unroll
    for (int k = 0; k < TT; ++k) out[k] = vec_raw<T, kLinVec>(p + (long)min(t0 + k, Ttot - 1) * stride, max(0, nd));
  }
}

// Sequences without a token: their final state is their initial state (the
// gradient of that one the gradient of the final state).  Each tile of tokens
// takes its share of the sequences.
__device__ __forceinline__ void lin_empty(const SeqFinder& sf, const float* from, float* to, int tile, int tiles, int d, int D) {
  for (int n = tile; n < sf.N; n += tiles)
    if (sf.at(n + 1) <= sf.at(n) && d < D) to[(long)n * D + d] = from ? from[(long)n * D + d] : 0.f;
}

struct LinAgg { f32x4 p[8][64], s[8][64]; };

// OUT false: what each tile does to the state (P, S).  OUT true: the states
// from the tiles' entry states, and the outputs.
template <typename T, int NW, int TT, bool OUT>
__global__ __launch_bounds__(64 * NW) void k_lin_fwd(LinParams p) {
  constexpr int TOK = NW * TT;
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ LinAgg agg;
  const int tile = blockIdx.x / p.cols, col = blockIdx.x - tile * p.cols;
  const int w = wave_id(), l = lane_id(), t0 = tile * TOK + w * TT;
  const int d = col * kLinCh + l * kLinVec, nd = min(kLinVec, p.D - d);
  const bool full = (col + 1) * kLinCh <= p.D;
  typename VecIO<T, kLinVec>::raw xr[TT], rr[TT], ir[TT];
  if (t0 < p.s.Ttot) {
    lin_load<T, TT>(p.r, p.r_stride, t0, p.s.Ttot, d, nd, full, rr);
    lin_load<T, TT>(p.i, p.i_stride, t0, p.s.Ttot, d, nd, full, ir);
    lin_load<T, TT>(p.x, p.x_stride, t0, p.s.Ttot, d, nd, full, xr);
  }
  float A2[kLinVec], h[kLinVec];
  vec_load<float, kLinVec>(p.A + d, max(0, nd), A2);
  if (OUT && tile > 0) vec_load<float, kLinVec>(p.S + (long)(tile - 1) * p.D + d, max(0, nd), h);
  else
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = 0.f;
#pragma unroll
  for (int c = 0; c < kLinVec; ++c) A2[c] *= 1.4426950408889634f;
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  const TokenRuns run = lin_runs<TT>(sf, t0);
  float a[TT][kLinVec], b[TT][kLinVec];
  f32x4 P = f32x4{1.f, 1.f, 1.f, 1.f}, S = zero4();
  if (t0 < p.s.Ttot) {
#pragma unroll
    for (int k = 0; k < TT; ++k) {
      float x[kLinVec], r[kLinVec], i[kLinVec];
      VecIO<T, kLinVec>::up(rr[k], r);
      VecIO<T, kLinVec>::up(ir[k], i);
      VecIO<T, kLinVec>::up(xr[k], x);
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) lin_gates(x[c], r[c], i[c], A2[c], a[k][c], b[k][c]);
      if (run.first >> k & 1) {   // h_t = a h_0 + b
        if (p.h0) {
          float h0[kLinVec];
          vec_load<float, kLinVec>(p.h0 + (long)lin_seq_at(sf, t0 + k) * p.D + d, max(0, nd), h0);
#pragma unroll
          for (int c = 0; c < kLinVec; ++c) b[k][c] = fmaf(a[k][c], h0[c], b[k][c]);
        }
      }
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) {
        P[c] *= a[k][c];
        S[c] = run.gap >> k & 1 ? 0.f : run.first >> k & 1 ? b[k][c] : fmaf(a[k][c], S[c], b[k][c]);
      }
    }
  }
  if (run.first | run.gap) P = f32x4{kFresh, kFresh, kFresh, kFresh};
  agg.p[w][l] = P;
  agg.s[w][l] = S;
  __syncthreads();
  if constexpr (!OUT) {
    for (int c = threadIdx.x; c < kLinCh; c += 64 * NW) {
      if (col * kLinCh + c >= p.D) break;
      float q = 1.f, s = 0.f;
#pragma unroll
      for (int u = 0; u < NW; ++u) {
        const float pu = agg.p[u][c / 4][c % 4], su = agg.s[u][c / 4][c % 4];
        s = pu == kFresh ? su : fmaf(pu, s, su);
        q = pu == kFresh || q == kFresh ? kFresh : q * pu;
      }
      p.P[(long)tile * p.D + col * kLinCh + c] = q;
      p.S[(long)tile * p.D + col * kLinCh + c] = s;
    }
    return;
  }
  for (int u = 0; u < w; ++u) {
    const f32x4 pu = agg.p[u][l], su = agg.s[u][l];
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = pu[c] == kFresh ? su[c] : fmaf(pu[c], h[c], su[c]);
  }
  T* y = static_cast<T*>(p.y) + d;
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    if (t0 + k >= p.s.Ttot) break;
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = run.gap >> k & 1 ? 0.f : run.first >> k & 1 ? b[k][c] : fmaf(a[k][c], h[c], b[k][c]);
    if (nd > 0) vec_store<T, kLinVec>(y + (long)(t0 + k) * p.D, nd, h);
    if (p.ht && (run.last >> k & 1)) {
      const int n = lin_seq_at(sf, t0 + k);
      if (nd > 0) vec_store<float, kLinVec>(p.ht + (long)n * p.D + d, nd, h);
    }
  }
  if (p.ht) {
    for (int c = threadIdx.x; c < kLinCh; c += 64 * NW) lin_empty(sf, p.h0, p.ht, tile, p.tiles, col * kLinCh + c, p.D);
  }
}

// The tiles' (P, S) turned into the states at their ends, and, for the
// gradient, Q (what a tile hands on to the tile before it of the gradient of
// the state, from zero) into what it hands on: 64 channels by 16 strands of
// consecutive tiles a workgroup.
template <bool BWD>
__global__ __launch_bounds__(1024) void k_lin_join(LinParams p) {
  __shared__ float lp[16][64], ls[16][64], lq[16][64];
  const int c = threadIdx.x & 63, u = threadIdx.x >> 6, d = blockIdx.x * 64 + c;
  const int per = (p.tiles + 15) / 16, j0 = min(u * per, p.tiles), j1 = min(j0 + per, p.tiles);
  const bool live = d < p.D;
  const float* P = p.P + d;
  float* S = p.S + d;
  float* Q = BWD ? p.Q + d : nullptr;
  float q = 1.f, s = 0.f, g = 0.f;
  if (live) {
#pragma unroll 8
    for (int j = j0; j < j1; ++j) {
      const float pj = P[(long)j * p.D], sj = S[(long)j * p.D];
      s = pj == kFresh ? sj : fmaf(pj, s, sj);
      q = pj == kFresh || q == kFresh ? kFresh : q * pj;
    }
    if (BWD)
#pragma unroll 8
      for (int j = j1 - 1; j >= j0; --j) {
        const float pj = P[(long)j * p.D], qj = Q[(long)j * p.D];
        g = pj == kFresh ? qj : fmaf(pj, g, qj);
      }
  }
  lp[u][c] = q;
  ls[u][c] = s;
  lq[u][c] = g;
  __syncthreads();
  if (!live) return;
  float h = 0.f;
  for (int v = 0; v < u; ++v) h = lp[v][c] == kFresh ? ls[v][c] : fmaf(lp[v][c], h, ls[v][c]);
#pragma unroll 8
  for (int j = j0; j < j1; ++j) {
    const float pj = P[(long)j * p.D], sj = S[(long)j * p.D];
    h = pj == kFresh ? sj : fmaf(pj, h, sj);
    S[(long)j * p.D] = h;
  }
  if (BWD) {
    g = 0.f;
    for (int v = 15; v > u; --v) g = lp[v][c] == kFresh ? lq[v][c] : fmaf(lp[v][c], g, lq[v][c]);
#pragma unroll 8
    for (int j = j1 - 1; j >= j0; --j) {
      const float pj = P[(long)j * p.D], qj = Q[(long)j * p.D];
      g = pj == kFresh ? qj : fmaf(pj, g, qj);
      Q[(long)j * p.D] = g;
    }
  }
}

// Gradient.  With g_t the gradient of h_t from everything behind it,
//   g_t = dy_t + a_{t+1} g_{t+1}  (+ dht at a sequence's last token)
//   dx = g m sigmoid(i),  di = g b (1 - sigmoid(i))
//   ds = g (a h_{t-1} - a^2 / m sigmoid(i) x),  dr = ds A e (1 - e),  dA = sum of ds e
// (s = A e; where m is zero its term is left out).  A lane walks its TT tokens
// three times: for the run's P, S and Q, forwards for the states before each
// token, which take the place of b, and backwards for the gradients.
template <typename T, int NW, int TT, bool OUT>
__global__ __launch_bounds__(64 * NW) void k_lin_bwd(LinParams p) {
  constexpr int TOK = NW * TT;
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ LinAgg agg;
  __shared__ f32x4 back[NW][64];
  const int tile = blockIdx.x / p.cols, col = blockIdx.x - tile * p.cols;
  const int w = wave_id(), l = lane_id(), t0 = tile * TOK + w * TT;
  const int d = col * kLinCh + l * kLinVec, nd = min(kLinVec, p.D - d);
  const bool full = (col + 1) * kLinCh <= p.D;
  typename VecIO<T, kLinVec>::raw xr[TT], rr[TT], ir[TT], gr[TT];
  if (t0 < p.s.Ttot) {
    lin_load<T, TT>(p.r, p.r_stride, t0, p.s.Ttot, d, nd, full, rr);
    lin_load<T, TT>(p.i, p.i_stride, t0, p.s.Ttot, d, nd, full, ir);
    lin_load<T, TT>(p.x, p.x_stride, t0, p.s.Ttot, d, nd, full, xr);
    lin_load<T, TT>(p.dy, p.D, t0, p.s.Ttot, d, nd, full, gr);
  }
  float A[kLinVec], h[kLinVec], g[kLinVec];
  vec_load<float, kLinVec>(p.A + d, max(0, nd), A);
#pragma unroll
  for (int c = 0; c < kLinVec; ++c) h[c] = g[c] = 0.f;
  if (OUT && tile > 0) vec_load<float, kLinVec>(p.S + (long)(tile - 1) * p.D + d, max(0, nd), h);
  if (OUT && tile + 1 < p.tiles) vec_load<float, kLinVec>(p.Q + (long)(tile + 1) * p.D + d, max(0, nd), g);
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  const TokenRuns run = lin_runs<TT>(sf, t0);
  float a[TT][kLinVec], b[TT][kLinVec];
  f32x4 P = f32x4{1.f, 1.f, 1.f, 1.f}, S = zero4(), Q = zero4();
  auto dy_at = [&](int k, float (&f)[kLinVec]) __attribute__((always_inline)) {
    VecIO<T, kLinVec>::up(gr[k], f);
    if (p.dht && (run.last >> k & 1)) {
      float e[kLinVec];
      vec_load<float, kLinVec>(p.dht + (long)lin_seq_at(sf, t0 + k) * p.D + d, max(0, nd), e);
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) f[c] += e[c];
    }
  };
  auto h0_at = [&](int k, float (&f)[kLinVec]) __attribute__((always_inline)) {
    if (p.h0) vec_load<float, kLinVec>(p.h0 + (long)lin_seq_at(sf, t0 + k) * p.D + d, max(0, nd), f);
    else
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) f[c] = 0.f;
  };
  if (t0 < p.s.Ttot) {
#pragma unroll
    for (int k = 0; k < TT; ++k) {
      float x[kLinVec], r[kLinVec], i[kLinVec];
      VecIO<T, kLinVec>::up(rr[k], r);
      VecIO<T, kLinVec>::up(ir[k], i);
      VecIO<T, kLinVec>::up(xr[k], x);
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) lin_gates(x[c], r[c], i[c], A[c] * 1.4426950408889634f, a[k][c], b[k][c]);
      if (run.first >> k & 1) {
        float h0[kLinVec];
        h0_at(k, h0);
#pragma unroll
        for (int c = 0; c < kLinVec; ++c) S[c] = fmaf(a[k][c], h0[c], b[k][c]);
      } else {
#pragma unroll
        for (int c = 0; c < kLinVec; ++c) S[c] = run.gap >> k & 1 ? 0.f : fmaf(a[k][c], S[c], b[k][c]);
      }
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) P[c] *= a[k][c];
    }
#pragma unroll
    for (int k = TT - 1; k >= 0; --k) {
      float f[kLinVec];
      dy_at(k, f);
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) Q[c] = (run.first | run.gap) >> k & 1 ? 0.f : a[k][c] * (f[c] + Q[c]);
    }
  }
  if (run.first | run.gap) P = f32x4{kFresh, kFresh, kFresh, kFresh};
  agg.p[w][l] = P;
  agg.s[w][l] = S;
  back[w][l] = Q;
  __syncthreads();
  if constexpr (!OUT) {
    for (int c = threadIdx.x; c < kLinCh; c += 64 * NW) {
      if (col * kLinCh + c >= p.D) break;
      float q = 1.f, s = 0.f, b = 0.f;
#pragma unroll
      for (int u = 0; u < NW; ++u) {
        const float pu = agg.p[u][c / 4][c % 4], su = agg.s[u][c / 4][c % 4];
        s = pu == kFresh ? su : fmaf(pu, s, su);
        q = pu == kFresh || q == kFresh ? kFresh : q * pu;
      }
#pragma unroll
      for (int u = NW - 1; u >= 0; --u) {
        const float pu = agg.p[u][c / 4][c % 4], qu = back[u][c / 4][c % 4];
        b = pu == kFresh ? qu : fmaf(pu, b, qu);
      }
      p.P[(long)tile * p.D + col * kLinCh + c] = q;
      p.S[(long)tile * p.D + col * kLinCh + c] = s;
      p.Q[(long)tile * p.D + col * kLinCh + c] = b;
    }
    return;
  }
  for (int u = 0; u < w; ++u) {
    const f32x4 pu = agg.p[u][l], su = agg.s[u][l];
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = pu[c] == kFresh ? su[c] : fmaf(pu[c], h[c], su[c]);
  }
  for (int u = NW - 1; u > w; --u) {
    const f32x4 pu = agg.p[u][l], qu = back[u][l];
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) g[c] = pu[c] == kFresh ? qu[c] : fmaf(pu[c], g[c], qu[c]);
  }
  // forwards: the state before each token in the place of b
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    if (run.first >> k & 1) h0_at(k, h);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) {
      const float old = h[c];
      h[c] = run.gap >> k & 1 ? 0.f : fmaf(a[k][c], old, b[k][c]);
      b[k][c] = old;
    }
  }
  f32x4 dA = zero4();
  T *dx = static_cast<T*>(p.dx) + d, *dr = static_cast<T*>(p.dr) + d, *di = static_cast<T*>(p.di) + d;
#pragma unroll
  for (int k = TT - 1; k >= 0; --k) {
    const long at = (long)(t0 + k) * p.D;
    if (run.gap >> k & 1) {
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) g[c] = 0.f;
      if (t0 + k < p.s.Ttot && nd > 0) {
        vec_store<T, kLinVec>(dx + at, nd, g);
        vec_store<T, kLinVec>(dr + at, nd, g);
        vec_store<T, kLinVec>(di + at, nd, g);
      }
      continue;
    }
    float x[kLinVec], r[kLinVec], i[kLinVec], f[kLinVec], ox[kLinVec], orr[kLinVec], oi[kLinVec];
    dy_at(k, f);
    VecIO<T, kLinVec>::up(rr[k], r);
    VecIO<T, kLinVec>::up(ir[k], i);
    VecIO<T, kLinVec>::up(xr[k], x);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) {
      const float gt = f[c] + g[c], at = a[k][c];
      float e, ne, j, nj;
      sigmoid_both(r[c], e, ne);
      sigmoid_both(i[c], j, nj);
      const float m = lin_factor(A[c] * 1.4426950408889634f * e, at);
      const float jx = j * x[c];
      const float dm = m > 0.f ? at * at * __builtin_amdgcn_rcpf(m) : (m == 0.f ? 0.f : m);
      const float ds = gt * (at * b[k][c] - dm * jx);
      ox[c] = gt * m * j;
      oi[c] = gt * m * jx * nj;
      orr[c] = ds * A[c] * e * ne;
      dA[c] = fmaf(ds, e, dA[c]);
      g[c] = at * gt;
    }
    if (nd > 0) {
      vec_store<T, kLinVec>(dx + at, nd, ox);
      vec_store<T, kLinVec>(dr + at, nd, orr);
      vec_store<T, kLinVec>(di + at, nd, oi);
    }
    if (run.first >> k & 1) {
      if (p.dh0 && nd > 0) vec_store<float, kLinVec>(p.dh0 + (long)lin_seq_at(sf, t0 + k) * p.D + d, nd, g);
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) g[c] = 0.f;
    }
  }
  __syncthreads();   // every wave has read the others' runs
  back[w][l] = dA;
  __syncthreads();
  for (int c = threadIdx.x; c < kLinCh; c += 64 * NW) {
    if (p.dh0) lin_empty(sf, p.dht, p.dh0, tile, p.tiles, col * kLinCh + c, p.D);
    if (col * kLinCh + c >= p.D) continue;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < NW; ++u) s += back[u][c / 4][c % 4];
    p.part[(long)tile * p.D + col * kLinCh + c] = s;
  }
}

// One new token per row; a wave takes 256 channels of one row.
template <typename T>
__global__ __launch_bounds__(256) void k_lin_step(LinParams p) {
  const long unit = (long)blockIdx.x * (blockDim.x >> 6) + wave_id();
  const int row = (int)(unit / p.cols);
  if (row >= p.s.Ttot) return;   // wave-uniform
  const int d = (int)(unit - (long)row * p.cols) * kLinCh + lane_id() * kLinVec, nd = min(kLinVec, p.D - d);
  const int slot = step_slot(p.slots, row, p.num_slots);
  if (nd <= 0) return;
  T* y = static_cast<T*>(p.y) + (long)row * p.D + d;
  float h[kLinVec] = {0.f, 0.f, 0.f, 0.f};
  if (slot >= 0) {
    float x[kLinVec], r[kLinVec], i[kLinVec], A[kLinVec];
    float* state = p.ht + (long)slot * p.D + d;
    vec_load<float, kLinVec>(state, nd, h);
    vec_load<T, kLinVec>(static_cast<const T*>(p.r) + (long)row * p.r_stride + d, nd, r);
    vec_load<T, kLinVec>(static_cast<const T*>(p.i) + (long)row * p.i_stride + d, nd, i);
    vec_load<T, kLinVec>(static_cast<const T*>(p.x) + (long)row * p.x_stride + d, nd, x);
    vec_load<float, kLinVec>(p.A + d, nd, A);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) {
      float a, b;
      lin_gates(x[c], r[c], i[c], A[c] * 1.4426950408889634f, a, b);
      h[c] = fmaf(a, h[c], b);
    }
    vec_store<float, kLinVec>(state, nd, h);
  }
  vec_store<T, kLinVec>(y, nd, h);
}

constexpr int kLinWaves = 8, kLinTok = 8;   // waves a tile, tokens a wave
int lin_tiles(int tokens) {
  const int n = (tokens + kLinWaves * kLinTok - 1) / (kLinWaves * kLinTok);
  return n > 0 ? n : 1;
}
int lin_cols(int D) { return (D + kLinCh - 1) / kLinCh; }

template <typename K>
static hipError_t lin_launch(const char* name, K kernel, dim3 grid, dim3 block, const LinParams& p, hipStream_t st) {
  timing_before(name, st);
  hipLaunchKernelGGL(kernel, grid, block, 0, st, p);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}

template <typename T>
static hipError_t lin_fwd(const LinParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.cols)), block(64 * kLinWaves);
  if (p.tiles > 1) {
    if (hipError_t e = lin_launch("linear_scan_parts", k_lin_fwd<T, kLinWaves, kLinTok, false>, grid, block, p, st)) return e;
    if (hipError_t e = lin_launch("linear_scan_join", k_lin_join<false>, dim3((p.D + 63) / 64), dim3(1024), p, st)) return e;
  }
  return lin_launch("linear_scan_out", k_lin_fwd<T, kLinWaves, kLinTok, true>, grid, block, p, st);
}
hipError_t launch_lin_fwd(DType dt, const LinParams& p, hipStream_t st) {
  return dt == DType::BF16 ? lin_fwd<bf16>(p, st) : lin_fwd<float>(p, st);
}

template <typename T>
static hipError_t lin_bwd(const LinParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.cols)), block(64 * kLinWaves);
  if (p.tiles > 1) {
    if (hipError_t e = lin_launch("linear_scan_bwd_parts", k_lin_bwd<T, kLinWaves, kLinTok, false>, grid, block, p, st)) return e;
    if (hipError_t e = lin_launch("linear_scan_bwd_join", k_lin_join<true>, dim3((p.D + 63) / 64), dim3(1024), p, st)) return e;
  }
  if (hipError_t e = lin_launch("linear_scan_bwd", k_lin_bwd<T, kLinWaves, kLinTok, true>, grid, block, p, st)) return e;
  RowsSum s = {};
  s.part = p.part;
  s.rows = p.tiles;
  s.dim = p.D;
  s.out[0] = p.dA;
  return launch_rows_sum(DType::F32, 1, s, st);
}
hipError_t launch_lin_bwd(DType dt, const LinParams& p, hipStream_t st) {
  return dt == DType::BF16 ? lin_bwd<bf16>(p, st) : lin_bwd<float>(p, st);
}

hipError_t launch_lin_step(DType dt, const LinParams& p, hipStream_t st) {
  const long units = (long)p.s.Ttot * p.cols;
  const int waves = units >= 8L * kComputeUnits ? 4 : 1;
  const dim3 grid((unsigned)((units + waves - 1) / waves)), block(64 * waves);
  return dt == DType::BF16 ? lin_launch("linear_scan_step", k_lin_step<bf16>, grid, block, p, st)
                           : lin_launch("linear_scan_step", k_lin_step<float>, grid, block, p, st);
}

}  // namespace gdr
