// gdr_ssm.hip -- selective state space scan of prompts.
//
//   S_t = e^{g_t} S_{t-1} + B_t (d_t x_t)^T,  y_t = S_t^T C_t + D x_t,  g_t = d_t A
//
// in chunks of 64 tokens (gam = cumsum of g inside the chunk, h = the chunk's
// entry state):
//   y_i  = e^{gam_i} h^T C_i + sum_{j <= i} (C_i . B_j) e^{gam_i - gam_j} d_j x_j + D x_i
//   h'   = e^{gam_n} h + sum_j B_j (e^{gam_n - gam_j} d_j x_j)^T
// Every decay is the exponential of a difference of gam, so that strong gates
// underflow to zero instead of dividing by it.
//
// A workgroup of 4 waves takes 128 channels (x columns of one group's heads)
// and one segment of the token axis; a wave owns 32 of them, within one head,
// with its [N, 32] block of the state in fp32 accumulators.  The scores C B^T
// of a chunk are the same for every head of the group: the waves share their
// computation and each applies its own head's decays.
//
// Long prompts are cut into segments that run side by side: a first pass
// computes what each segment adds to the state and its decay, k_ssm_join
// turns those into the states at the segment ends, and the output pass starts
// from them, all exact.  Segments are cut on the packed token axis, so that
// ragged batches balance by themselves.
#include "gdr_layer.h"

namespace gdr {

constexpr int SC = 64;        // chunk
constexpr int SCOLS = 128;    // channels of a workgroup

// A contraction block of 32: lane group q = lane / 16 holds the indices
// 16 (e / 4) + 4 q + e % 4, e < 8, on both operands -- the order in which two
// accumulator tiles, one above the other, hold their rows.
template <typename T> struct Blk;
template <> struct Blk<bf16> {
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // the contraction runs along an LDS row
  static __device__ __forceinline__ frag along(const bf16* row) { return ld_a2(row, 4 * (lane_id() >> 4)); }
  // the contraction runs down the rows r0.., operand index = column
  static __device__ __forceinline__ frag down(const bf16* m, int pitch, int r0, int c0) {
    const int r = r0 + 4 * (lane_id() >> 4);
    return cat4(tr4(m, pitch, r, c0), tr4(m, pitch, r + 16, c0));
  }
  static __device__ __forceinline__ frag acc(const f32x4& x, const f32x4& y) { return pack_b(x, y); }
  static __device__ __forceinline__ float get(const frag& f, int e) { return static_cast<float>(f[e]); }
};
template <> struct Blk<float> {
  struct frag { float v[8]; };
  static __device__ __forceinline__ f32x4 mma(const frag& a, const frag& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ frag along(const float* row) {
    const float* p = row + 4 * (lane_id() >> 4);
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 16);
    return frag{{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}};
  }
  static __device__ __forceinline__ frag down(const float* m, int pitch, int r0, int c0) {
    const float* p = m + (r0 + 4 * (lane_id() >> 4)) * pitch + c0 + (lane_id() & 15);
    frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = p[(16 * (e / 4) + e % 4) * pitch];
    return f;
  }
  static __device__ __forceinline__ frag acc(const f32x4& x, const f32x4& y) {
    return frag{{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
  }
  static __device__ __forceinline__ float get(const frag& f, int e) { return f.v[e]; }
};

// 64 rows of COLS elements, global -> registers -> LDS; rows from `rows` on
// and columns from `cols` on read as zero.
template <typename T, int COLS>
struct ChunkRegs {
  static constexpr int VEC = 16 / (int)sizeof(T), VPR = COLS / VEC, NV = SC * VPR / 256;
  static constexpr int PITCH = COLS + VEC;
  uint4 v[NV];
  __device__ __forceinline__ void load(const T* base, long stride, int rows, int cols) {
    const rsrc_t r = make_rsrc_u(base, ((long)(rows - 1) * stride + cols) * (long)sizeof(T));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int idx = (int)threadIdx.x + 256 * i, row = idx / VPR, c = (idx % VPR) * VEC;
      const uint32_t off = (uint32_t)(row * (int)stride + c) * (uint32_t)sizeof(T);
      v[i] = buf_load16(r, (row < rows && c < cols) ? off : 0x80000000u);
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int idx = (int)threadIdx.x + 256 * i;
      *reinterpret_cast<uint4*>(lds + (idx / VPR) * PITCH + (idx % VPR) * VEC) = v[i];
    }
  }
};

template <typename T, int ND, bool OUT>
struct SsmLds {
  static constexpr int PB = ChunkRegs<T, ND>::PITCH, PX = ChunkRegs<T, SCOLS>::PITCH;
  T b[SC * PB];
  T c[OUT ? SC * PB : 4];
  T x[SC * PX];
  f32x4 score[OUT ? 10 * 64 : 1];   // tiles (jt <= it) of B C^T, by lane
  // per wave, its head's tokens: gam as a float (and its remainder, fp32), d,
  // e^gam, and the weight of the token in the chunk's end state
  float gam[4][SC], rem[sizeof(T) == 4 ? 4 : 1][SC], d[4][SC], eg[4][SC], wt[4][SC];
  int32_t cu[kCuLds];
};

template <typename T, int ND, bool OUT>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void k_ssm(SsmParams p, int total) {
  typedef Blk<T> K;
  typedef typename K::frag frag;
  constexpr int NT = ND / 16, NK = ND / 32;
  __shared__ __align__(16) SsmLds<T, ND, OUT> lds;
  constexpr int PB = lds.PB, PX = lds.PX;
  // workgroups of one segment share B and C: keep them on one XCD
  const int id = xcd_remap(blockIdx.x, total);
  if (id >= total) return;
  const SeqFinder sf = seq_finder(p.s, lds.cu);
  const int hp = p.H / p.G * p.P;                       // channels of a group
  const int per_group = (hp + SCOLS - 1) / SCOLS;
  const int seg = id / p.wgs, wi = id - seg * p.wgs;
  const int g = wi / per_group, col0 = (wi - g * per_group) * SCOLS;
  const int cols = min(SCOLS, hp - col0);
  const int w = wave_id(), l = lane_id(), c = l & 15, q = l >> 4;
  const bool live = 32 * w < cols;                      // waves without channels still help with tiles and scores
  const int chan0 = g * hp + col0;                      // the workgroup's first channel
  const int chan = chan0 + (live ? 32 * w : 0);
  const int head = chan / p.P, pc = chan - head * p.P;
  const long sstride = (long)p.N * p.P;
  const T* x = static_cast<const T*>(p.x);
  const T* dt = static_cast<const T*>(p.dt);
  const T* Bp = static_cast<const T*>(p.B) + (long)g * ND;
  const T* Cp = static_cast<const T*>(p.C) + (long)g * ND;
  T* y = static_cast<T*>(p.y);
  const long HP = (long)p.H * p.P;
  const float A = p.A[head], bias = p.bias ? p.bias[head] : 0.f;
  const float skip = OUT && p.D ? p.D[head] : 0.f;

  f32x4 h[NT][2];
  auto state_at = [&](const float* s) { return s + (long)head * sstride + pc; };
  // accumulator element e of tile (nt, pt): state row 16 nt + 4 q + e, column 16 pt + c
  auto load_state = [&](const float* s) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int e = 0; e < 4; ++e) h[nt][pt][e] = s ? s[(long)(16 * nt + 4 * q + e) * p.P + 16 * pt + c] : 0.f;
  };
  auto store_state = [&](float* s) {
    if (!live) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[(long)(16 * nt + 4 * q + e) * p.P + 16 * pt + c] = h[nt][pt][e];
  };

  if (seg >= p.segs) {   // final states of empty sequences
    const int n = seg - p.segs;
    if (sf.at(n + 1) > sf.at(n)) return;
    load_state(p.h0 ? state_at(p.h0 + n * (long)p.H * sstride) : nullptr);
    store_state(const_cast<float*>(state_at(p.ht + n * (long)p.H * sstride)));
    return;
  }

  const int seg0 = seg * p.seg, seg1 = min(seg0 + p.seg, p.s.Ttot);
  float total_gam = 0.f;

  // One run of tokens [t0, t1) of a sequence, from the state in h.
  auto run = [&](int t0, int t1) {
    ChunkRegs<T, ND> rb, rc;
    ChunkRegs<T, SCOLS> rx;
    float rdt;
    auto fetch = [&](int t) {
      const int len = min(SC, t1 - t);
      rb.load(Bp + (long)t * p.b_stride, p.b_stride, len, ND);
      if constexpr (OUT) rc.load(Cp + (long)t * p.c_stride, p.c_stride, len, ND);
      rx.load(x + (long)t * p.x_stride + chan0, p.x_stride, len, cols);
      rdt = l < len ? to_f(dt[(long)(t + l) * p.dt_stride + head]) : 0.f;
    };
    fetch(t0);
    for (int t = t0; t < t1; t += SC) {
      const int len = min(SC, t1 - t);
      lds_barrier();   // the tiles of the chunk before are no longer read
      rb.store(lds.b);
      if constexpr (OUT) rc.store(lds.c);
      rx.store(lds.x);
      float d = rdt + bias;
      if (p.softplus) d = softplus_f(d);
      if (l >= len) d = 0.f;
      // gam in 64 bits: a difference of two far sums keeps fp32's accuracy
      double gam = (double)d * (double)A;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(gam, m);
        if (l >= m) gam += o;
      }
      const double gend = __shfl(gam, 63);   // tokens behind the last have d = 0
      lds.gam[w][l] = (float)gam;
      if constexpr (sizeof(T) == 4) lds.rem[w][l] = (float)(gam - (double)(float)gam);
      lds.d[w][l] = d;
      if constexpr (OUT) lds.eg[w][l] = exp_f((float)gam);
      lds.wt[w][l] = exp_f((float)(gend - gam)) * d;
      total_gam += (float)gend;
      lds_barrier();
      if (t + SC < t1) fetch(t + SC);

      frag xf[2][2];   // x^T: columns 16 pt.., tokens 32 jb..
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) xf[pt][jb] = K::down(lds.x, PX, 32 * jb, 32 * w + 16 * pt);
      if constexpr (OUT) {
        // scores, transposed: tile (jt, it) holds B_j . C_i, rows j, columns i
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const int idx = w + 4 * k;
          if (idx < 10) {
            const int it = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0, jt = idx - it * (it + 1) / 2;
            f32x4 s = zero4();
#pragma unroll
            for (int kb = 0; kb < NK; ++kb)
              s = K::mma(K::along(lds.b + (16 * jt + c) * PB + 32 * kb), K::along(lds.c + (16 * it + c) * PB + 32 * kb), s);
            lds.score[idx * 64 + l] = s;
          }
        }
        lds_barrier();
        frag hf[2][NK];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int kb = 0; kb < NK; ++kb) hf[pt][kb] = K::acc(h[2 * kb][pt], h[2 * kb + 1][pt]);
        // rolled: unrolled, the four tiles' operands do not fit the registers
#pragma unroll 1
        for (int it = 0; it < 4; ++it) {
          const int i = 16 * it + c;
          f32x4 acc[2] = {zero4(), zero4()};
#pragma unroll
          for (int kb = 0; kb < NK; ++kb) {
            const frag cf = K::along(lds.c + i * PB + 32 * kb);
            acc[0] = K::mma(hf[0][kb], cf, acc[0]);
            acc[1] = K::mma(hf[1][kb], cf, acc[1]);
          }
          const float gi = lds.gam[w][i], ei = lds.eg[w][i];
          const float ri = sizeof(T) == 4 ? lds.rem[sizeof(T) == 4 ? w : 0][i] : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[0][e] *= ei;
            acc[1][e] *= ei;
          }
#pragma unroll
          for (int jb = 0; jb < 2; ++jb) {
            if (2 * jb > it) break;
            f32x4 pt2[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int jt = 2 * jb + k;
              pt2[k] = zero4();
              if (jt <= it) {
                const f32x4 s = lds.score[(it * (it + 1) / 2 + jt) * 64 + l];
                const f32x4 gj = *reinterpret_cast<const f32x4*>(&lds.gam[w][16 * jt + 4 * q]);
                const f32x4 dj = *reinterpret_cast<const f32x4*>(&lds.d[w][16 * jt + 4 * q]);
                f32x4 df;
#pragma unroll
                for (int e = 0; e < 4; ++e) df[e] = gi - gj[e];
                if constexpr (sizeof(T) == 4) {
                  const f32x4 rj = *reinterpret_cast<const f32x4*>(&lds.rem[w][16 * jt + 4 * q]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) df[e] += ri - rj[e];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float v = s[e] * (exp_f(df[e]) * dj[e]);
                  pt2[k][e] = (jt < it || 4 * q + e <= c) ? v : 0.f;
                }
              }
            }
            const frag pf = K::acc(pt2[0], pt2[1]);
            acc[0] = K::mma(xf[0][jb], pf, acc[0]);
            acc[1] = K::mma(xf[1][jb], pf, acc[1]);
          }
          if (live && i < len) {
#pragma unroll
            for (int pt = 0; pt < 2; ++pt) {
              float xv[4], o[4];
              vec_load<T, 4>(lds.x + i * PX + 32 * w + 16 * pt + 4 * q, 4, xv);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = p.D ? fmaf(skip, xv[e], acc[pt][e]) : acc[pt][e];
              vec_store<T, 4>(y + (long)(t + i) * HP + chan + 16 * pt + 4 * q, 4, o);
            }
          }
        }
      }

      // h' = e^{gam_n} h + B^T (w x), w_j = e^{gam_n - gam_j} d_j.  The fp32
      // product w x is taken as three bf16 terms of 8 bits each, so that the
      // state is as exact as fp32 operands would make it (one term would leave
      // 2^-8, two 2^-16); B and x are bf16 as they are.
      const float en = exp_f((float)gend);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int e = 0; e < 4; ++e) h[nt][pt][e] *= en;
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&lds.wt[w][32 * jb + 4 * q]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&lds.wt[w][32 * jb + 16 + 4 * q]);
        constexpr int TERMS = sizeof(T) == 2 ? 3 : 1;
        frag wx[TERMS][2];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) {
          f32x4 u, v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u[e] = K::get(xf[pt][jb], e) * w0[e];
            v[e] = K::get(xf[pt][jb], 4 + e) * w1[e];
          }
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            wx[k][pt] = K::acc(u, v);
            if (k + 1 < TERMS)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                u[e] -= K::get(wx[k][pt], e);
                v[e] -= K::get(wx[k][pt], 4 + e);
              }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const frag bf = K::down(lds.b, PB, 32 * jb, 16 * nt);
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
#pragma unroll
            for (int k = 0; k < TERMS; ++k) h[nt][pt] = K::mma(bf, wx[k][pt], h[nt][pt]);
        }
      }
    }
  };

  if constexpr (!OUT) {
    int start, end;
    const int n = sf.find(seg1 - 1, start, end);
    float* decay = p.seg_decay + (long)seg * p.H + head;
    const bool through = n >= 0 && end > seg1;     // the sequence goes on behind the segment
    const bool began = start >= seg0;              // and began in it
    if (through) {
      load_state(began && p.h0 ? state_at(p.h0 + n * (long)p.H * sstride) : nullptr);
      run(max(start, seg0), seg1);
      store_state(const_cast<float*>(state_at(p.seg_state + seg * (long)p.H * sstride)));
    }
    if (live && pc == 0 && l == 0) *decay = through && !began ? total_gam : -__builtin_inff();
  } else {
    for (int t = seg0; t < seg1;) {
      int start, end;
      const int n = sf.find(t, start, end);
      const int stop = min(end, seg1);
      if (n < 0) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (long i = threadIdx.x; i < (long)(stop - t) * (cols / 4); i += 256) {
          const long r = i / (cols / 4);
          vec_store<T, 4>(y + (t + r) * HP + chan0 + 4 * (i - r * (cols / 4)), 4, zero);
        }
      } else {
        if (start == t) load_state(p.h0 ? state_at(p.h0 + n * (long)p.H * sstride) : nullptr);
        else load_state(state_at(p.seg_state + (seg - 1) * (long)p.H * sstride));
        run(t, stop);
        if (p.ht && stop == end) store_state(const_cast<float*>(state_at(p.ht + n * (long)p.H * sstride)));
      }
      t = stop;
    }
  }
}

// States at the segment ends, in place: end_s = b_s + e^{decay_s} end_{s-1}.
// One thread walks four values over the segments, their loads eight ahead.
__global__ __launch_bounds__(256) void k_ssm_join(SsmParams p) {
  const long per = (long)p.H * p.N * p.P;
  const long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= per) return;
  const int head = (int)(i / ((long)p.N * p.P));
  const int n = p.segs - 1;
  f32x4 cur = zero4();
  for (int s0 = 0; s0 < n; s0 += 8) {
    f32x4 b[8];
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = min(s0 + k, n - 1);
      b[k] = *reinterpret_cast<const f32x4*>(p.seg_state + s * per + i);
      g[k] = p.seg_decay[(long)s * p.H + head];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (s0 + k >= n) break;
      // -inf: the segment's end does not depend on its start (no product with
      // a start that may hold anything)
      const float e = expf(g[k]);
#pragma unroll
      for (int v = 0; v < 4; ++v) cur[v] = g[k] == -__builtin_inff() ? b[k][v] : fmaf(e, cur[v], b[k][v]);
      *reinterpret_cast<f32x4*>(p.seg_state + (s0 + k) * per + i) = cur;
    }
  }
}

// Segments: enough workgroups for two (bf16) or one (fp32, by its LDS) on
// every compute unit, but not under 256 tokens, where the two further
// launches cost more than they save.
void ssm_plan(DType dt, SsmParams& p) {
  const int hp = p.H / p.G * p.P;
  p.wgs = p.G * ((hp + SCOLS - 1) / SCOLS);
  const long want = (dt == DType::BF16 ? 2L : 1L) * kComputeUnits;
  const long most = (p.s.Ttot + 255) / 256;
  long segs = (want + p.wgs - 1) / p.wgs;
  segs = segs > most ? most : segs;
  segs = segs < 1 ? 1 : segs;
  const long tokens = (p.s.Ttot + segs - 1) / segs;
  p.seg = (int)((tokens + SC - 1) / SC * SC);
  if (p.seg < SC) p.seg = SC;
  p.segs = (p.s.Ttot + p.seg - 1) / p.seg;
}

template <typename T, int ND>
static hipError_t ssm_scan(const SsmParams& p, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (p.segs > 1) {
    const int total = (p.segs - 1) * p.wgs;
    timing_before("ssm_states", st);
    hipLaunchKernelGGL((k_ssm<T, ND, false>), dim3((unsigned)((total + 7) / 8 * 8)), dim3(256), 0, st, p, total);
    e = hipGetLastError();
    timing_after(st);
    if (e != hipSuccess) return e;
    const long quads = (long)p.H * p.N * p.P / 4;
    timing_before("ssm_join", st);
    hipLaunchKernelGGL(k_ssm_join, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, p);
    e = hipGetLastError();
    timing_after(st);
    if (e != hipSuccess) return e;
  }
  // sequences without tokens have no segment: their states are copied by
  // workgroups of their own
  const int extra = p.ht && (p.s.cu || p.s.T == 0) ? p.s.N : 0;
  const long total = (long)(p.segs + extra) * p.wgs;
  if (total == 0) return hipSuccess;
  timing_before("ssm_scan", st);
  hipLaunchKernelGGL((k_ssm<T, ND, true>), dim3((unsigned)((total + 7) / 8 * 8)), dim3(256), 0, st, p, (int)total);
  e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_ssm_scan(DType dt, const SsmParams& p, hipStream_t st) {
  if (dt == DType::BF16) {
    if (p.N == 32) return ssm_scan<bf16, 32>(p, st);
    return p.N == 64 ? ssm_scan<bf16, 64>(p, st) : ssm_scan<bf16, 128>(p, st);
  }
  if (p.N == 32) return ssm_scan<float, 32>(p, st);
  return p.N == 64 ? ssm_scan<float, 64>(p, st) : ssm_scan<float, 128>(p, st);
}

}  // namespace gdr
