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
// of another sequence over).  A product of positive decays stays positive: one
// that falls below fp32's smallest value, 2^-149, counts as that, so that an
// infinite state stays infinite across runs as it does token by token, and only a
// decay that is zero makes it NaN (a finite state adds 2^-149 of itself at most,
// as the rounding of a product next to that size does).
#include "gdr_layer.h"

namespace gdr {

constexpr float kFresh = -1.f;   // in the place of a product of decays: the end does not depend on the start
typedef float lin_v __attribute__((ext_vector_type(kLinVec)));
constexpr int kLinJoinCh = 16;

// 1 - a^2 with a = exp(s), s = s2 ln 2: -expm1(2 s).  Near zero the difference
// would lose all bits: below 2 |s| = 1/4 the Taylor series up to z^6 / 720 (the
// next term is 4.8e-8 of the first); above it 1 - a^2 >= 0.22.  A positive s
// gives a negative value, and a NaN as its root.
__device__ __forceinline__ float lin_factor2(float s2, float a) {
  const float z = s2 * 1.3862943611198906f;
  float q = fmaf(z, 1.f / 720.f, 1.f / 120.f);
  q = fmaf(q, z, 1.f / 24.f);
  q = fmaf(q, z, 1.f / 6.f);
  q = fmaf(q, z, 0.5f);
  q = fmaf(q, z, 1.f);
  return z > -0.25f ? -z * q : fmaf(-a, a, 1.f);
}
// a and b of one value; A2 = A log2(e)
__device__ __forceinline__ void lin_gates(float x, float r, float i, float A2, float& a, float& b) {
  const float s2 = A2 * sigmoid_f(r);
  a = __builtin_amdgcn_exp2f(s2);
  b = __builtin_amdgcn_sqrtf(lin_factor2(s2, a)) * sigmoid_f(i) * x;
}
// sigmoid(x) and 1 - sigmoid(x), both to a few ulps on either side of zero
// (below -16 the latter is one; e^-x overflows from -88 on, and 1 / (1 + it) is
// zero then).
__device__ __forceinline__ void sigmoid_both(float x, float& e, float& ne) {
  const float t = exp_f(-x);
  e = __builtin_amdgcn_rcpf(1.f + t);
  ne = x < -16.f ? 1.f : t * e;
}

// The runs of a wave's TT tokens, in scalar registers; seq: the wave's place in LDS.
template <int TT>
__device__ __forceinline__ TokenRuns lin_runs(const SeqFinder& sf, int t0, int* seq) {
  TokenRuns m = token_runs(sf, t0, TT, seq);
  m.first = __builtin_amdgcn_readfirstlane(m.first);
  m.last = __builtin_amdgcn_readfirstlane(m.last);
  m.gap = __builtin_amdgcn_readfirstlane(m.gap);
  return m;
}
__device__ __forceinline__ int lin_seq(const int* seq, int k) { return __builtin_amdgcn_readfirstlane(seq[k]); }
// The same pointer, to global memory, in scalar registers (it is equal across the wave).
#define GDR_GLOBAL __attribute__((address_space(1)))
__device__ __forceinline__ GDR_GLOBAL char* lin_uniform(const void* p) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a), hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return (GDR_GLOBAL char*)(uintptr_t)((uint64_t)hi << 32 | lo);
}

// A row's values of a lane's channels; NARROW: fewer than kLinVec are there.
template <bool NARROW, typename T>
__device__ __forceinline__ typename VecIO<T, kLinVec>::raw lin_read(const void* row, int d, int D) {
  GDR_GLOBAL char* at = lin_uniform(row) + (uint32_t)d * (uint32_t)sizeof(T);   // a scalar row address and one offset in a register
  if constexpr (NARROW) return vec_raw<T, kLinVec>((const T*)at, D);
  else return *(const GDR_GLOBAL typename VecIO<T, kLinVec>::raw*)at;
}
template <bool NARROW, typename T>
__device__ __forceinline__ void lin_write(void* row, int d, int D, const float (&f)[kLinVec]) {
  GDR_GLOBAL char* at = lin_uniform(row) + (uint32_t)d * (uint32_t)sizeof(T);
  if constexpr (NARROW) vec_store<T, kLinVec>((T*)at, D, f);
  else *(GDR_GLOBAL typename VecIO<T, kLinVec>::raw*)at = VecIO<T, kLinVec>::down(f);
}
template <bool NARROW>
__device__ __forceinline__ void lin_floats(const float* row, int d, int D, float (&f)[kLinVec]) {
  VecIO<float, kLinVec>::up(lin_read<NARROW, float>(row, d, D), f);
}

// TT tokens of an operand from token t0 on; tokens behind the last are the last one.
template <bool NARROW, typename T, int TT>
__device__ __forceinline__ void lin_load(const void* base, long stride, int t0, int Ttot, int d, int D,
                                         typename VecIO<T, kLinVec>::raw (&out)[TT]) {
#pragma unroll
  for (int k = 0; k < TT; ++k)
    out[k] = lin_read<NARROW, T>(static_cast<const char*>(base) + (long)min(t0 + k, Ttot - 1) * stride * (long)sizeof(T), d, D);
}

// Sequences without a token: their final state is their initial state (the
// gradient of that one the gradient of the final state).  Each wave of each tile
// of tokens takes its share of the sequences.
template <int NW>
__device__ __forceinline__ void lin_empty(const SeqFinder& sf, const float* from, float* to, int tile, int tiles, int col, int D) {
  if (!to) return;
  empty_sequences(sf, tile + (long)tiles * wave_id(), (long)tiles * NW, [&](long n) {
    for (int d = col * kLinCh + lane_id(); d < min(D, (col + 1) * kLinCh); d += 64) to[n * D + d] = from ? from[n * D + d] : 0.f;
  });
}

// What the waves of a tile do to the state.
struct LinAgg {
  lin_v p[8][64], s[8][64];
  int seq[8][32];   // of the waves' tokens that start or end a sequence
};

// a and b of a lane's tokens.
template <typename T, int TT>
__device__ __forceinline__ void lin_values(const float (&A2)[kLinVec], const typename VecIO<T, kLinVec>::raw (&xr)[TT],
                                           const typename VecIO<T, kLinVec>::raw (&rr)[TT], const typename VecIO<T, kLinVec>::raw (&ir)[TT],
                                           float (&a)[TT][kLinVec], float (&b)[TT][kLinVec]) {
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    float x[kLinVec], r[kLinVec], i[kLinVec];
    VecIO<T, kLinVec>::up(rr[k], r);
    VecIO<T, kLinVec>::up(ir[k], i);
    VecIO<T, kLinVec>::up(xr[k], x);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) lin_gates(x[c], r[c], i[c], A2[c], a[k][c], b[k][c]);
  }
}
// The initial state of the sequence that starts at the wave's token k.
template <bool NARROW>
__device__ __forceinline__ void lin_initial(const LinParams& p, const int* seq, int k, int d, float (&h)[kLinVec]) {
  if (p.h0) {
    lin_floats<NARROW>(p.h0 + (long)lin_seq(seq, k) * p.D, d, p.D, h);
  } else {
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = 0.f;
  }
}
// The state behind each token from the state h before them; then(k, h) takes it.
template <bool NARROW, int TT, typename F>
__device__ __forceinline__ void lin_states(const LinParams& p, const int* seq, const TokenRuns& run, int t0, int d,
                                           const float (&a)[TT][kLinVec], const float (&b)[TT][kLinVec], float (&h)[kLinVec], F then) {
  if ((run.first | run.gap | run.last) == 0) {
#pragma unroll
    for (int k = 0; k < TT; ++k) {
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) h[c] = fmaf(a[k][c], h[c], b[k][c]);
      then(k, h);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    if (run.first >> k & 1) lin_initial<NARROW>(p, seq, k, d, h);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = run.gap >> k & 1 ? 0.f : fmaf(a[k][c], h[c], b[k][c]);
    if (t0 + k < p.s.Ttot) then(k, h);
  }
}
// The product of decays, at least 2^-149 if none of them is zero; low: the
// least of that one's bits, which are 1, and theirs (numbers that are not
// negative are in order as their bits are).  No branch: one that looked at products
// of zero alone took 369 us where this takes 363 (65536 x 2560 in bf16; 361 with
// products that vanish).
__device__ __forceinline__ float lin_product(float P, int low) { return __builtin_bit_cast(float, max(low, __builtin_bit_cast(int, P))); }
// n <= N runs one behind another: at(k) gives (P, S) of the k-th.
struct LinRun { float P, S; };
template <int N, typename F> __device__ __forceinline__ LinRun lin_joined(int n, F at) {
  float P = 1.f, S = 0.f;
  int low = 1;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k < n) {
      const LinRun r = at(k);
      S = r.P == kFresh ? r.S : fmaf(r.P, S, r.S);
      P *= r.P;
      low = min(low, __builtin_bit_cast(int, r.P));
    }
  return {low < 0 ? kFresh : lin_product(P, low), S};   // below zero is kFresh alone, or a NaN with a sign, whose S is NaN and stands alone too
}
__device__ __forceinline__ float lin_after(float h, float P, float S) { return P == kFresh ? S : fmaf(P, h, S); }

// What the tokens do to the state: (P, S).
template <bool NARROW, int TT>
__device__ __forceinline__ void lin_effect(const LinParams& p, const int* seq, const TokenRuns& run, int t0, int d,
                                           const float (&a)[TT][kLinVec], const float (&b)[TT][kLinVec], lin_v& P, lin_v& S) {
  float h[kLinVec] = {};
  lin_states<NARROW, TT>(p, seq, run, t0, d, a, b, h, [](int, const float (&)[kLinVec]) {});
#pragma unroll
  for (int c = 0; c < kLinVec; ++c) {
    S[c] = h[c];
    float prod = 1.f;
    int low = 1;
#pragma unroll
    for (int k = 0; k < TT; ++k) {
      prod *= a[k][c];
      low = min(low, __builtin_bit_cast(int, a[k][c]));
    }
    P[c] = lin_product(prod, low);
    if (run.first | run.gap) P[c] = kFresh;
  }
}
// The outputs of a lane's tokens from the state h before them.
template <bool NARROW, typename T, int TT>
__device__ __forceinline__ void lin_leave(const LinParams& p, const int* seq, const TokenRuns& run, int t0, int d,
                                          const float (&a)[TT][kLinVec], const float (&b)[TT][kLinVec], float (&h)[kLinVec]) {
  lin_states<NARROW, TT>(p, seq, run, t0, d, a, b, h, [&](int k, const float (&h)[kLinVec]) {
    lin_write<NARROW, T>(static_cast<char*>(p.y) + (long)(t0 + k) * p.D * (long)sizeof(T), d, p.D, h);
    if (p.ht && (run.last >> k & 1)) lin_write<NARROW, float>(p.ht + (long)lin_seq(seq, k) * p.D, d, p.D, h);
  });
}
// What tiles leave for those behind them: a word of (P, S) for each tile and
// channel, and the state at the end of each group of kLinGroup tiles.  The
// words are written and read whole, past the caches that the XCDs do not
// share, so that a word that is there needs no flag and no order with others;
// kLinEmpty stands in those that are not there yet (never in one that is: a
// NaN is written as kLinNan).
constexpr int kLinGroup = 16;
constexpr int kLinLine = 32;   // between the counters of two columns, so that they share no cache line
constexpr uint32_t kLinEmpty = 0xffffffffu, kLinNan = 0x7fc00000u;
// How often a wait looks.  Every wait ends long before that, as the tiles are
// handed out in order and a tile leaves its own word before it waits for
// those before it.  Only if another call clears the words meanwhile (two
// calls that share a workspace) is it reached, once a wave: the state is NaN
// then.
constexpr int kLinLooks = 1 << 18;
__device__ __forceinline__ uint32_t lin_bits(float x) { return x != x ? kLinNan : __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ void lin_put(uint64_t* at, LinRun r) {
  __hip_atomic_store(at, (uint64_t)lin_bits(r.S) << 32 | lin_bits(r.P), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t lin_get(const char* row, uint32_t off) {
  return __hip_atomic_load((const GDR_GLOBAL uint64_t*)(lin_uniform(row) + off), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(256) void k_lin_clear(LinParams p) {
  const long n = (long)p.tiles * p.D, words = n * 2 + (long)(p.tiles / kLinGroup + 1) * p.D;   // of 32 bits
  uint32_t* w = reinterpret_cast<uint32_t*>(p.words);
  for (long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4; i < words; i += (long)gridDim.x * 1024) {
    if (i + 4 <= words) *reinterpret_cast<u32x4_u4*>(w + i) = u32x4_u4{kLinEmpty, kLinEmpty, kLinEmpty, kLinEmpty};
    else
      for (long j = i; j < words; ++j) w[j] = kLinEmpty;
  }
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.cols; i += 256) p.ticket[i * kLinLine] = 0;
}

// One pass: persistent workgroups take the tiles of a column of channels in
// order, and a tile's entry state comes from the words of the tiles of its
// group and the state at the end of the group before.  Every wait ends: a
// workgroup finishes its tiles in the order in which it took them, and of all
// tiles taken and not yet finished the one taken first waits for finished ones
// only (none is taken by a workgroup that does not run).
//
// 8192 x 4096 in bf16: 80 us (3.3 TB/s), 65536 x 2560 360 (3.7); without the
// waits 65 and 288.  Two passes (the tiles' words, a join, the outputs) took 111
// and 477, as the values are made twice; tiles of 64 tokens 88 and 447, which
// wait more often; one counter for all columns 93 and 383 (512 workgroups that
// draw their first tile from one word: 13 us); the next tile's loads ahead of
// the waits 95 and 425, as a word's load is not there before data asked for
// earlier.
template <typename T, int NW, int TT, bool NARROW>
__global__ __launch_bounds__(64 * NW, 4) void k_lin_one(LinParams p) {
  constexpr int TOK = NW * TT, SHARE = 64 * NW / kLinCh, EACH = kLinGroup / SHARE;   // lanes that look back for a channel, words for each
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ LinAgg aggs[2];
  __shared__ float half_p[SHARE][kLinCh], half_s[SHARE][kLinCh], entry[kLinCh], before[kLinCh];
  __shared__ int ticket;
  // a workgroup stays with its column of channels
  const int w = wave_id(), l = lane_id(), col = blockIdx.x % p.cols, d = lin_base(col * kLinCh + l * kLinVec, p.D);
  const int hf = w / (kLinCh / 64), c = 64 * (w - kLinCh / 64 * hf) + l;
  const uint32_t dc = lin_channel(col, c, p.D);
  const int cl = c / kLinVec, cv = lin_place(c, p.D);
  int* tickets = p.ticket + col * kLinLine;
  if (threadIdx.x == 0) ticket = atomicAdd(tickets, 1);
  float A2[kLinVec];
  lin_floats<NARROW>(p.A, d, p.D, A2);
#pragma unroll
  for (int e = 0; e < kLinVec; ++e) A2[e] *= 1.4426950408889634f;
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  __syncthreads();
  int tile = __builtin_amdgcn_readfirstlane(ticket), most = kLinLooks;
  for (int par = 0; tile < p.tiles; par ^= 1) {
    const int t0 = tile * TOK + w * TT;
    LinAgg& agg = aggs[par];
    typename VecIO<T, kLinVec>::raw xr[TT], rr[TT], ir[TT];
    lin_load<NARROW, T, TT>(p.r, p.r_stride, t0, p.s.Ttot, d, p.D, rr);
    lin_load<NARROW, T, TT>(p.i, p.i_stride, t0, p.s.Ttot, d, p.D, ir);
    lin_load<NARROW, T, TT>(p.x, p.x_stride, t0, p.s.Ttot, d, p.D, xr);
    int next = 0;
    if (threadIdx.x == 0) next = atomicAdd(tickets, 1);
    const TokenRuns run = lin_runs<TT>(sf, t0, agg.seq[w]);
    float a[TT][kLinVec], b[TT][kLinVec];
    lin_values<T, TT>(A2, xr, rr, ir, a, b);
    lin_v P, S;
    lin_effect<NARROW, TT>(p, agg.seq[w], run, t0, d, a, b, P, S);
    agg.p[w][l] = P;
    agg.s[w][l] = S;
    lds_barrier();
    LinRun whole = {1.f, 0.f};
    if (hf == 0) {
      whole = lin_joined<NW>(NW, [&](int u) { return LinRun{agg.p[u][cl][cv], agg.s[u][cl][cv]}; });
      lin_put(p.words + (long)tile * p.D + dc, whole);
    }
    const int grp = tile / kLinGroup, in = tile - grp * kLinGroup, n = max(0, min(EACH, in - EACH * hf));
    const bool reach = hf == SHARE - 1 && grp > 0;   // the state at the end of the group before
    const char* words = reinterpret_cast<const char*>(p.words + (long)(grp * kLinGroup + EACH * hf) * p.D);
    const char* end = reinterpret_cast<const char*>(p.ends + (long)(grp - 1) * p.D);
    LinRun back = {1.f, 0.f};
    uint32_t ve = 0;
    if (n > 0 || reach) {
      uint64_t v[EACH];
      for (int looks = 0;; ++looks) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) v[k] = k < n ? lin_get(words + (long)k * p.D * 8, 8 * dc) : 0;
        if (reach) ve = __hip_atomic_load((const GDR_GLOBAL uint32_t*)(lin_uniform(end) + 4 * dc), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        bool all = ve != kLinEmpty;
#pragma unroll
        for (int k = 0; k < EACH; ++k) all &= (uint32_t)v[k] != kLinEmpty;
        if (all) break;
        if (looks >= most) {   // never again as long
          most = 0;
          break;
        }
        __builtin_amdgcn_s_sleep(2);
      }
      back = lin_joined<EACH>(n, [&](int k) {
        return LinRun{__builtin_bit_cast(float, (uint32_t)v[k]), __builtin_bit_cast(float, (uint32_t)(v[k] >> 32))};
      });
    }
    half_p[hf][c] = back.P;
    half_s[hf][c] = back.S;
    if (hf == SHARE - 1) before[c] = __builtin_bit_cast(float, ve);
    if (threadIdx.x == 0) ticket = next;
    lds_barrier();
    if (hf == 0) {
      float h = before[c];
#pragma unroll
      for (int u = 0; u < SHARE; ++u) h = lin_after(h, half_p[u][c], half_s[u][c]);
      entry[c] = h;
      if (in == kLinGroup - 1)
        __hip_atomic_store(p.ends + (long)grp * p.D + dc, lin_bits(lin_after(h, whole.P, whole.S)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    lds_barrier();
    const int done = tile;
    tile = __builtin_amdgcn_readfirstlane(ticket);
    float h[kLinVec];
#pragma unroll
    for (int e = 0; e < kLinVec; ++e) h[e] = entry[l * kLinVec + e];
    for (int u = 0; u < w; ++u) {
      const lin_v pu = agg.p[u][l], su = agg.s[u][l];
#pragma unroll
      for (int e = 0; e < kLinVec; ++e) h[e] = lin_after(h[e], pu[e], su[e]);
    }
    lin_leave<NARROW, T, TT>(p, agg.seq[w], run, t0, d, a, b, h);
    lin_empty<NW>(sf, p.h0, p.ht, done, p.tiles, col, p.D);
  }
}

// Prompts of one tile: nothing to look back for, and nothing to clear.
template <typename T, int NW, int TT, bool NARROW>
__global__ __launch_bounds__(64 * NW, 4) void k_lin_tile(LinParams p) {
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ LinAgg agg;
  const int w = wave_id(), l = lane_id(), t0 = w * TT, col = blockIdx.x;
  const int d = lin_base(col * kLinCh + l * kLinVec, p.D);
  float a[TT][kLinVec], b[TT][kLinVec], h[kLinVec] = {};
  if (p.s.Ttot > 0) {
    typename VecIO<T, kLinVec>::raw xr[TT], rr[TT], ir[TT];
    lin_load<NARROW, T, TT>(p.r, p.r_stride, t0, p.s.Ttot, d, p.D, rr);
    lin_load<NARROW, T, TT>(p.i, p.i_stride, t0, p.s.Ttot, d, p.D, ir);
    lin_load<NARROW, T, TT>(p.x, p.x_stride, t0, p.s.Ttot, d, p.D, xr);
    float A2[kLinVec];
    lin_floats<NARROW>(p.A, d, p.D, A2);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) A2[c] *= 1.4426950408889634f;
    lin_values<T, TT>(A2, xr, rr, ir, a, b);
  }
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  const TokenRuns run = lin_runs<TT>(sf, t0, agg.seq[w]);
  lin_v P, S;
  lin_effect<NARROW, TT>(p, agg.seq[w], run, t0, d, a, b, P, S);
  agg.p[w][l] = P;
  agg.s[w][l] = S;
  lds_barrier();
  for (int u = 0; u < w; ++u) {
    const lin_v pu = agg.p[u][l], su = agg.s[u][l];
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = lin_after(h[c], pu[c], su[c]);
  }
  lin_leave<NARROW, T, TT>(p, agg.seq[w], run, t0, d, a, b, h);
  lin_empty<NW>(sf, p.h0, p.ht, 0, 1, col, p.D);
}

// The tiles' (P, S) turned into the states at their ends, and Q into what the
// tiles hand on: 16 channels by 64 strands of consecutive tiles a workgroup, and
// the two workgroups that share cache lines on one XCD (683 tiles of 4096
// channels: 21 us; on two XCDs 34, 32 channels by 32 strands 27, and with a
// strand's tiles kept in registers between its walks 36).
__global__ __launch_bounds__(1024) void k_lin_join(LinParams p) {
  constexpr int CH = kLinJoinCh, ST = 1024 / CH;
  __shared__ float lp[ST][CH], ls[ST][CH], lq[ST][CH];
  const int c = threadIdx.x % CH, u = threadIdx.x / CH;
  const int y = blockIdx.x >> 3, d = ((y >> 1) * 16 + (blockIdx.x & 7) * 2 + (y & 1)) * CH + c;
  const int per = (p.tiles + ST - 1) / ST, j0 = min(u * per, p.tiles), j1 = min(j0 + per, p.tiles);
  const bool live = d < p.D;
  const float* P = p.P + d;
  float *S = p.S + d, *Q = p.Q + d;
  float q = 1.f, s = 0.f, g = 0.f;
  if (live) {
#pragma unroll 4
    for (int j = j0; j < j1; ++j) {
      const float pj = P[(long)j * p.D], sj = S[(long)j * p.D], gj = Q[(long)j * p.D];
      // what a later run hands on goes through this one's decays (kFresh: not at all)
      g = q == kFresh ? g : fmaf(q, gj, g);
      const LinRun r = lin_joined<2>(2, [&](int k) { return k ? LinRun{pj, sj} : LinRun{q, s}; });
      q = r.P;
      s = r.S;
    }
  }
  lp[u][c] = q;
  ls[u][c] = s;
  lq[u][c] = g;
  __syncthreads();
  if (!live || j0 == j1) return;
  float h = 0.f;
#pragma unroll 4
  for (int v = 0; v < u; ++v) h = lin_after(h, lp[v][c], ls[v][c]);
#pragma unroll 4
  for (int j = j0; j < j1; ++j) {
    const float pj = P[(long)j * p.D], sj = S[(long)j * p.D];
    h = lin_after(h, pj, sj);
    S[(long)j * p.D] = h;
  }
  g = 0.f;
#pragma unroll 4
  for (int v = ST - 1; v > u; --v) g = lin_after(g, lp[v][c], lq[v][c]);
#pragma unroll 4
  for (int j = j1 - 1; j >= j0; --j) {
    const float pj = P[(long)j * p.D], gj = Q[(long)j * p.D];
    g = lin_after(g, pj, gj);
    Q[(long)j * p.D] = g;
  }
}

// Gradient.  With g_t the gradient of h_t from everything behind it,
//   g_t = dy_t + a_{t+1} g_{t+1}  (+ dht at a sequence's last token)
//   dx = g m sigmoid(i),  di = g b (1 - sigmoid(i))
//   ds = g (a h_{t-1} - a^2 / m sigmoid(i) x),  dr = ds A e (1 - e),  dA = sum of ds e
// (s = A e; where m is zero its term is left out).  What does not depend on h
// and g is made once (seven values), the states turn it into five factors of g
// forwards, and the gradients come backwards.
//
// OUT false: what each tile does to the state (P, S) and to its gradient (P, Q:
// what it hands on to the tile before it, from zero).  Both directions cannot
// be had in one pass, as tiles would wait for each other.  32768 x 4096 in bf16:
// 236 us (4.5 TB/s), the join 21 to 23, this pass 380 to 408 by the run (4.6 to 4.9
// TB/s), dA 9 to 11.  With eight
// tokens a wave one workgroup of 152 registers is resident and not two (475); in
// workgroups of four waves 355, and the shorter tiles' joins take that again.
// Values made again for the walk backwards instead of held took 643.
template <typename T, int NW, int TT, bool OUT, bool NARROW>
__global__ __launch_bounds__(64 * NW, OUT ? 4 : 6) void k_lin_bwd(LinParams p) {
  constexpr int TOK = NW * TT;
  __shared__ int32_t cu_lds[kCuLds];
  __shared__ LinAgg agg;
  __shared__ lin_v back[NW][64];
  // the second pass starts with what the first one read last
  const int id = OUT ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x, tile = id / p.cols, col = id - tile * p.cols;
  const int w = wave_id(), l = lane_id(), t0 = tile * TOK + w * TT;
  const int d = lin_base(col * kLinCh + l * kLinVec, p.D);
  float a[TT][kLinVec], b[TT][kLinVec], g0[TT][kLinVec], h[kLinVec] = {}, g[kLinVec] = {};
  float mj[TT][kLinVec], fi[TT][kLinVec], u[TT][kLinVec], e[TT][kLinVec], q[TT][kLinVec];   // OUT
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  const TokenRuns run = lin_runs<TT>(sf, t0, agg.seq[w]);
  if (p.s.Ttot > 0) {
    typename VecIO<T, kLinVec>::raw xr[TT], rr[TT], ir[TT], gr[TT];
    lin_load<NARROW, T, TT>(p.r, p.r_stride, t0, p.s.Ttot, d, p.D, rr);
    lin_load<NARROW, T, TT>(p.i, p.i_stride, t0, p.s.Ttot, d, p.D, ir);
    lin_load<NARROW, T, TT>(p.x, p.x_stride, t0, p.s.Ttot, d, p.D, xr);
    lin_load<NARROW, T, TT>(p.dy, p.D, t0, p.s.Ttot, d, p.D, gr);
    float A[kLinVec], A2[kLinVec];
    lin_floats<NARROW>(p.A, d, p.D, A);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) A2[c] = A[c] * 1.4426950408889634f;
    if (OUT && tile > 0) lin_floats<NARROW>(p.S + (long)(tile - 1) * p.D, d, p.D, h);
    if (OUT && tile + 1 < p.tiles) lin_floats<NARROW>(p.Q + (long)(tile + 1) * p.D, d, p.D, g);
    if constexpr (!OUT) {
      lin_values<T, TT>(A2, xr, rr, ir, a, b);
    } else {
#pragma unroll
      for (int k = 0; k < TT; ++k) {
        float x[kLinVec], r[kLinVec], i[kLinVec];
        VecIO<T, kLinVec>::up(rr[k], r);
        VecIO<T, kLinVec>::up(ir[k], i);
        VecIO<T, kLinVec>::up(xr[k], x);
#pragma unroll
        for (int c = 0; c < kLinVec; ++c) {
          float ne, j, nj;
          sigmoid_both(r[c], e[k][c], ne);
          sigmoid_both(i[c], j, nj);
          const float s2 = A2[c] * e[k][c], ak = __builtin_amdgcn_exp2f(s2), m2 = lin_factor2(s2, ak);
          // 1 / m; none where m is zero or its square below the normal numbers, which the instruction takes as zero
          const float rm = fabsf(m2) < 0x1p-126f ? 0.f : __builtin_amdgcn_rsqf(m2);
          a[k][c] = ak;
          mj[k][c] = m2 * rm * j;
          b[k][c] = mj[k][c] * x[c];
          fi[k][c] = b[k][c] * nj;
          u[k][c] = ak * rm * (ak * rm) * b[k][c];   // a^2 / m sigmoid(i) x
          q[k][c] = A[c] * ne;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < TT; ++k) VecIO<T, kLinVec>::up(gr[k], g0[k]);
  }
  if (p.dht && run.last) {
#pragma unroll
    for (int k = 0; k < TT; ++k)
      if (run.last >> k & 1) {
        float f[kLinVec];
        lin_floats<NARROW>(p.dht + (long)lin_seq(agg.seq[w], k) * p.D, d, p.D, f);
#pragma unroll
        for (int c = 0; c < kLinVec; ++c) g0[k][c] += f[c];
      }
  }
  // the gradient that token k hands on to the one before it
  const uint32_t cut = run.first | run.gap;
  lin_v P, S, Q;
  lin_effect<NARROW, TT>(p, agg.seq[w], run, t0, d, a, b, P, S);
#pragma unroll
  for (int c = 0; c < kLinVec; ++c) Q[c] = 0.f;
#pragma unroll
  for (int k = TT - 1; k >= 0; --k) {
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) Q[c] = a[k][c] * (g0[k][c] + Q[c]);
    if (cut >> k & 1)
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) Q[c] = 0.f;
  }
  agg.p[w][l] = P;
  agg.s[w][l] = S;
  back[w][l] = Q;
  lds_barrier();
  if constexpr (!OUT) {
    for (int c = threadIdx.x; c < kLinCh; c += 64 * NW) {
      const int dc = lin_channel(col, c, p.D), cl = c / kLinVec, cv = lin_place(c, p.D);
      const LinRun whole = lin_joined<NW>(NW, [&](int v) { return LinRun{agg.p[v][cl][cv], agg.s[v][cl][cv]}; });
      float tq = 0.f;
#pragma unroll
      for (int v = NW - 1; v >= 0; --v) tq = lin_after(tq, agg.p[v][cl][cv], back[v][cl][cv]);
      p.P[(long)tile * p.D + dc] = whole.P;
      p.S[(long)tile * p.D + dc] = whole.S;
      p.Q[(long)tile * p.D + dc] = tq;
    }
    return;
  }
  for (int v = 0; v < w; ++v) {
    const lin_v pv = agg.p[v][l], sv = agg.s[v][l];
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) h[c] = lin_after(h[c], pv[c], sv[c]);
  }
  for (int v = NW - 1; v > w; --v) {
    const lin_v pv = agg.p[v][l], qv = back[v][l];
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) g[c] = lin_after(g[c], pv[c], qv[c]);
  }
#pragma unroll
  for (int k = 0; k < TT; ++k) {
    if (run.first >> k & 1) lin_initial<NARROW>(p, agg.seq[w], k, d, h);
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) {
      const float f = fmaf(a[k][c], h[c], -u[k][c]) * e[k][c];   // ds e / g
      u[k][c] = f;
      q[k][c] *= f;
      h[c] = fmaf(a[k][c], h[c], b[k][c]);
    }
    if (run.gap >> k & 1)
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) a[k][c] = g0[k][c] = mj[k][c] = fi[k][c] = u[k][c] = q[k][c] = h[c] = 0.f;
  }
  lin_v dA;
#pragma unroll
  for (int c = 0; c < kLinVec; ++c) dA[c] = 0.f;
#pragma unroll
  for (int k = TT - 1; k >= 0; --k) {
    float ox[kLinVec], orr[kLinVec], oi[kLinVec];
    if (run.gap >> k & 1)
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) g[c] = 0.f;
#pragma unroll
    for (int c = 0; c < kLinVec; ++c) {
      const float gt = g0[k][c] + g[c];
      ox[c] = gt * mj[k][c];
      oi[c] = gt * fi[k][c];
      orr[c] = gt * q[k][c];
      dA[c] = fmaf(gt, u[k][c], dA[c]);
      g[c] = a[k][c] * gt;
    }
    if (t0 + k < p.s.Ttot) {
      const long row = (long)(t0 + k) * p.D * (long)sizeof(T);
      lin_write<NARROW, T>(static_cast<char*>(p.dx) + row, d, p.D, ox);
      lin_write<NARROW, T>(static_cast<char*>(p.dr) + row, d, p.D, orr);
      lin_write<NARROW, T>(static_cast<char*>(p.di) + row, d, p.D, oi);
    }
    if (run.first >> k & 1) {
      if (p.dh0) lin_write<NARROW, float>(p.dh0 + (long)lin_seq(agg.seq[w], k) * p.D, d, p.D, g);
#pragma unroll
      for (int c = 0; c < kLinVec; ++c) g[c] = 0.f;
    }
  }
  lds_barrier();   // every wave has read the others' runs
  back[w][l] = dA;
  lds_barrier();
  lin_empty<NW>(sf, p.dht, p.dh0, tile, p.tiles, col, p.D);
  for (int c = threadIdx.x; c < kLinCh; c += 64 * NW) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) s += back[v][c / kLinVec][lin_place(c, p.D)];
    p.part[(long)tile * p.D + lin_channel(col, c, p.D)] = s;
  }
}

// One new token per row; a wave takes 128 channels of one row.  Bound by the
// launch: 256 x 4096 in bf16 6.3 us (17 MB, 3.0 at the rate of such streams), one row 3 (7.8
// a call).
template <typename T>
__global__ __launch_bounds__(256) void k_lin_step(LinParams p) {
  const long unit = (long)blockIdx.x * (blockDim.x >> 6) + wave_id();
  const int row = (int)(unit / p.cols);
  if (row >= p.s.Ttot) return;   // wave-uniform
  const int d = (int)(unit - (long)row * p.cols) * kLinCh + lane_id() * kLinVec, nd = min(kLinVec, p.D - d);
  const int slot = step_slot(p.slots, row, p.num_slots);
  if (nd <= 0) return;
  T* y = static_cast<T*>(p.y) + (long)row * p.D + d;
  float h[kLinVec] = {};
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

// Waves a tile, and tokens a wave (by the size of the type: a lane holds them all).
constexpr int kLinWaves = 8, kLinTok16 = 16, kLinTok32 = 8;
constexpr int kLinBwdWaves = 8, kLinBwdTok = 6;   // waves a tile, tokens a wave
static int lin_tiles_of(int tokens, int tile) {
  const int n = (tokens + tile - 1) / tile;
  return n > 0 ? n : 1;
}
int lin_tiles(DType dt, int tokens) { return lin_tiles_of(tokens, kLinWaves * (dt == DType::BF16 ? kLinTok16 : kLinTok32)); }
int lin_bwd_tiles(int tokens) { return lin_tiles_of(tokens, kLinBwdWaves * kLinBwdTok); }
int lin_cols(int D) { return (D + kLinCh - 1) / kLinCh; }

template <typename K>
static hipError_t lin_launch(const char* name, K kernel, dim3 grid, dim3 block, const LinParams& p, hipStream_t st) {
  timing_before(name, st);
  hipLaunchKernelGGL(kernel, grid, block, 0, st, p);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}

// Bytes of the words, the groups' states and the ticket; 32-bit values.
static long lin_words(int tiles, int D) { return (long)tiles * D * 2 + (long)(tiles / kLinGroup + 1) * D + (long)lin_cols(D) * kLinLine; }
size_t lin_fwd_bytes(DType dt, int tokens, int D) { return (size_t)lin_words(lin_tiles(dt, tokens), D) * 4; }

template <typename T>
static hipError_t lin_fwd(LinParams p, void* workspace, hipStream_t st) {
  constexpr int TT = sizeof(T) == 2 ? kLinTok16 : kLinTok32;
  const dim3 block(64 * kLinWaves);
#define CALL(K) (p.D < kLinVec ? K<T, kLinWaves, TT, true> : K<T, kLinWaves, TT, false>)
  if (p.tiles == 1) return lin_launch("linear_scan", CALL(k_lin_tile), dim3(p.cols), block, p, st);
  p.words = static_cast<uint64_t*>(workspace);
  p.ends = reinterpret_cast<uint32_t*>(p.words + (long)p.tiles * p.D);
  p.ticket = reinterpret_cast<int*>(p.ends + (long)(p.tiles / kLinGroup + 1) * p.D);
  const long blocks = (lin_words(p.tiles, p.D) + 4095) / 4096;
  if (hipError_t e = lin_launch("linear_scan_clear", k_lin_clear, dim3(blocks < 4 * kComputeUnits ? blocks : 4 * kComputeUnits), dim3(256), p, st)) return e;
  // as many workgroups a column as are resident at once
  const int resident = 2 * kComputeUnits / p.cols;
  return lin_launch("linear_scan", CALL(k_lin_one), dim3(p.cols * (resident < 1 ? 1 : resident < p.tiles ? resident : p.tiles)), block, p, st);
#undef CALL
}
hipError_t launch_lin_fwd(DType dt, const LinParams& p, void* workspace, hipStream_t st) {
  return dt == DType::BF16 ? lin_fwd<bf16>(p, workspace, st) : lin_fwd<float>(p, workspace, st);
}

template <typename T>
static hipError_t lin_bwd(const LinParams& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.tiles * p.cols)), block(64 * kLinBwdWaves);
#define CALL(OUT) (p.D < kLinVec ? k_lin_bwd<T, kLinBwdWaves, kLinBwdTok, OUT, true> : k_lin_bwd<T, kLinBwdWaves, kLinBwdTok, OUT, false>)
  if (p.tiles > 1) {
    if (hipError_t e = lin_launch("linear_scan_bwd_parts", CALL(false), grid, block, p, st)) return e;
    if (hipError_t e = lin_launch("linear_scan_bwd_join", k_lin_join, dim3((p.D + 16 * kLinJoinCh - 1) / (16 * kLinJoinCh) * 16), dim3(1024), p, st)) return e;
  }
  if (hipError_t e = lin_launch("linear_scan_bwd", CALL(true), grid, block, p, st)) return e;
#undef CALL
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
