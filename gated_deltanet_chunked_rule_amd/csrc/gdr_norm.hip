// gdr_norm.hip -- root-mean-square norm with the residual's addition, a gate
// and an 8-bit output with scales; and its gradient.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w silu(gate)
//
// Bound by memory: TPR lanes hold a whole row in registers (NV vectors of 8
// values each), so every operand is read once and the row's sum needs no
// second pass.  The sum is fp32 over the unrounded h.
#include "gdr_layer.h"

namespace gdr {

typedef uint32_t u32x2_u1 __attribute__((ext_vector_type(2), aligned(1)));

constexpr float kE4M3Max = 448.f;
constexpr float kQuantTiny = 0x1p-100f;   // an all-zero group gets the scale kQuantTiny / 448

// Sum over the TPR lanes of a row (a power of two, 16 to 1024), the same value
// on every lane; rows of more than a wave meet in LDS.  Two values at once.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*lds)[2]) {
  a = row16_sum(a);
  b = row16_sum(b);
#pragma unroll
  for (int m = 16; m < (TPR < 64 ? TPR : 64); m <<= 1) {
    a += __shfl_xor(a, m);
    b += __shfl_xor(b, m);
  }
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    if (lane_id() == 0) {
      lds[w][0] = a;
      lds[w][1] = b;
    }
    __syncthreads();
    const int first = (threadIdx.x / TPR) * (TPR / 64);
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) {
      a += lds[first + i][0];
      b += lds[first + i][1];
    }
  }
}

// A double from another lane of the row of 16 by a DPP control.
template <int C>
__device__ __forceinline__ double dpp_d(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, C, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), C, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// The larger one; a NaN is above everything.
__device__ __forceinline__ double max_nan(double a, double b) { return b <= a || a != a ? a : b; }
// Sum over the TPR lanes of a row in 64 bits, as row_sum2.
template <int TPR>
__device__ __forceinline__ double row_sum_d(double a, double* lds) {
  a += dpp_d<0xB1>(a);
  a += dpp_d<0x4E>(a);
  a += dpp_d<0x141>(a);
  a += dpp_d<0x140>(a);
#pragma unroll
  for (int m = 16; m < (TPR < 64 ? TPR : 64); m <<= 1) a += __shfl_xor(a, m);
  if constexpr (TPR > 64) {
    if (lane_id() == 0) lds[threadIdx.x >> 6] = a;
    __syncthreads();
    const int first = (threadIdx.x / TPR) * (TPR / 64);
    a = 0.0;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) a += lds[first + i];
  }
  return a;
}

__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {
#define GDR_MAX_STEP(C) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, C, 0xF, 0xF, true))
  GDR_MAX_STEP(0xB1);
  GDR_MAX_STEP(0x4E);
  GDR_MAX_STEP(0x141);
  GDR_MAX_STEP(0x140);
#undef GDR_MAX_STEP
  return v;
}

__device__ __forceinline__ long row_at(long row, int inner, long outer_stride, long inner_stride) {
  if (inner == 1) return row * outer_stride;
  const long o = row / inner;
  return o * outer_stride + (row - o * inner) * inner_stride;
}

// Short rows (a head's 64 to 512 values) go R to a lane group: one row has but
// two 16-byte loads per lane in flight.
template <typename T, int TPR, int NV, int R, bool QUANT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_fwd(NormParams p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  static_assert(R == 1 || TPR <= 64, "rows of several waves meet in LDS, one at a time");
  __shared__ float red[NT / 64][2];
  __shared__ double red_d[QUANT && TPR > 64 ? NT / 64 : 1];
  const int t = threadIdx.x & (TPR - 1);
  typename VecIO<T, 8>::raw raw_r[R][NV], rawr_r[R][NV], rawg_r[R][NV];
  float w[NV][8];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const long row = ((long)blockIdx.x * R + k) * RPB + threadIdx.x / TPR;
    const bool live = row < p.rows;   // rows behind the last read row 0 and write nothing
    const long rr = live ? row : 0;
    const T* x = static_cast<const T*>(p.x) + row_at(rr, p.inner, p.xo, p.xi);
    const T* res = p.residual ? static_cast<const T*>(p.residual) + row_at(rr, p.inner, p.ro, p.ri) : nullptr;
    const T* gate = p.gate ? static_cast<const T*>(p.gate) + row_at(rr, p.inner, p.go, p.gi) : nullptr;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8;
      raw_r[k][v] = vec_raw<T, 8>(x + d, max(0, p.dim - d));
      if (res) rawr_r[k][v] = vec_raw<T, 8>(res + d, max(0, p.dim - d));
      if (gate) rawg_r[k][v] = vec_raw<T, 8>(gate + d, max(0, p.dim - d));
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) vec_load<T, 8>(static_cast<const T*>(p.weight) + (v * TPR + t) * 8, max(0, p.dim - (v * TPR + t) * 8), w[v]);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const long row = ((long)blockIdx.x * R + k) * RPB + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const auto& raw = raw_r[k];
    const auto& rawr = rawr_r[k];
    const auto& rawg = rawg_r[k];
    const bool res = p.residual != nullptr, gate = p.gate != nullptr;
    // x + residual in 64 bits
    auto wide = [&](int v, double (&out)[8]) __attribute__((always_inline)) {
      float f[8], g[8];
      VecIO<T, 8>::up(raw[v], f);
      if (res) VecIO<T, 8>::up(rawr[v], g);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        // (the asm keeps the values from being made once and held for all uses)
        if (QUANT) asm volatile("" : "+v"(f[c]));
        out[c] = res ? (double)f[c] + (double)g[c] : (double)f[c];
      }
    };
    float h[NV][8], ss = 0.f, unused = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      VecIO<T, 8>::up(raw[v], h[v]);
      if (res) {
        float f[8];
        VecIO<T, 8>::up(rawr[v], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) h[v][c] += f[c];
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) ss = fmaf(h[v][c], h[v][c], ss);
    }
    // to 8 bits, rows of several waves are summed in 64 bits, for the borders
    // below; others are then where a value lies next to one
    double ssd = 0.0;
    if constexpr (QUANT && TPR > 64) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        double hd[8];
        wide(v, hd);
#pragma unroll
        for (int c = 0; c < 8; ++c) ssd = fma(hd[c], hd[c], ssd);
      }
      ssd = row_sum_d<TPR>(ssd, red_d);
      ss = (float)ssd;
    } else {
      row_sum2<TPR>(ss, unused, red);
    }
    const float r = rsqrt_f(fmaf(ss, p.inv_dim, p.eps));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = min(8, p.dim - d);
      if (p.h_out && live && nd > 0) vec_store<T, 8>(static_cast<T*>(p.h_out) + row * p.dim + d, nd, h[v]);
      float y[8], low = 0.f;   // low: how far below zero the lane's gates reach
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] = h[v][c] * r * w[v][c];
      if (gate) {
        float g[8];
        VecIO<T, 8>::up(rawg[v], g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          y[c] *= g[c] * sigmoid_f(g[c]);
          if (QUANT) low = fmaxf(low, -g[c]);
        }
      }
      if constexpr (QUANT) {
        // a group of 128 values is 16 lanes of 8; the largest magnitude is taken
        // on the bits, where a NaN is above everything
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) m = max(m, c < nd ? (__builtin_bit_cast(uint32_t, y[c]) & 0x7fffffffu) : 0u);
        m = max16_u32(m);
        m = max(m, __builtin_bit_cast(uint32_t, kQuantTiny));
        float scale = __builtin_bit_cast(float, m) * (1.f / kE4M3Max);
        // y / scale rounded to e4m3 (from its fp32 rounding).  A value next to a
        // border between two of them may be on either side by fp32's own
        // roundings: where both ends of the range that these may move it over
        // round to the same value (no compare and no clamp is needed: 448 (1 +
        // 2^-16) still rounds to 448), it is right; else the wave takes its
        // groups again in 64 bits (by the density of the borders, 8 an octave,
        // one wave of 512 values in 90, in 45 with gates about zero).
        // The range, in u = 2^-24: r is in y and in the group's largest value,
        // and cancels; h, h r and w leave 3 u in each of the two, 1 / 448, scale,
        // inv and the products with it 6 (the reciprocal's ulp is 2 u), and the
        // scale's rounding beside the exact one 1: 13, 16 are taken.  A gate
        // leaves 7.4 u more in each (exp2, 1 + e, reciprocal, two products, and
        // the exponent's rounding at gates above zero), and below zero e^-g is
        // off by 1.23 |g| u, the rounding of g log2 e: 28 + 2.45 |g| u in all, 32
        // + 2.5 |g| are taken.  From 80 on e^-g nears fp32's end: 64 bits.
        // (262144 x 128 with gates of std 1: 37 us; with the range of 2^-20 for
        // all, which left 1 in 3e5 values wrong at gates of -30 to -40, 35.5.)
        float margin = 0x1p-20f;
        bool far = false;
        if (gate) {
          low = __builtin_bit_cast(float, max16_u32(__builtin_bit_cast(uint32_t, low) & 0x7fffffffu));   // (the larger of 0 and -0 may be -0)
          margin = fmaf(low, 2.5f * 0x1p-24f, 0x1p-19f);
          far = low > 80.f;
        }
        const float inv = __builtin_amdgcn_rcpf(scale), inv0 = inv * (1.f - margin), inv1 = inv * (1.f + margin);
        int q[2] = {0, 0}, q1[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] * inv0, y[4 * i + 1] * inv0, q[i], false);
          q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] * inv0, y[4 * i + 3] * inv0, q[i], true);
          q1[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] * inv1, y[4 * i + 1] * inv1, q1[i], false);
          q1[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] * inv1, y[4 * i + 3] * inv1, q1[i], true);
        }
        auto leave = [&](const int (&q)[2], float scale) __attribute__((always_inline)) {
          if (nd <= 0 || !live) return;
          uint8_t* out = static_cast<uint8_t*>(p.y) + row * p.dim + d;
          if (nd == 8) {
            *reinterpret_cast<u32x2_u1*>(out) = u32x2_u1{(uint32_t)q[0], (uint32_t)q[1]};
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (c < nd) out[c] = (uint8_t)((uint32_t)q[c / 4] >> (8 * (c % 4)));
          }
          if ((t & 15) == 0) p.scales[row * ((p.dim + 127) / 128) + d / 128] = scale;
        };
        // The wave takes all of its groups again, and writes only those that need
        // it a second time: a row's values and scales are its own alone, whatever
        // rows share the wave.  (Written first, the values take no registers
        // meanwhile.)
        const uint64_t again = __builtin_amdgcn_ballot_w64(far || q[0] != q1[0] || q[1] != q1[1]);
        leave(q, scale);
        if (again != 0) {
          double sd = ssd;
          if constexpr (TPR <= 64) {
            sd = 0.0;
#pragma unroll
            for (int u = 0; u < NV; ++u) {
              double hd[8];
              wide(u, hd);
#pragma unroll
              for (int c = 0; c < 8; ++c) sd = fma(hd[c], hd[c], sd);
            }
            sd = row_sum_d<TPR>(sd, nullptr);
          }
          const double rd = 1.0 / sqrt(sd / (double)p.dim + (double)p.eps);
          float z[8];
          if (gate) VecIO<T, 8>::up(rawg[v], z);
          double yd[8], md = kQuantTiny;
          wide(v, yd);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            yd[c] = yd[c] * rd * (double)w[v][c];
            if (gate) yd[c] *= (double)z[c] / (1.0 + exp(-(double)z[c]));
            const double ad = fabs(yd[c]);
            if (c < nd) md = max_nan(md, ad);
          }
          md = max_nan(md, dpp_d<0xB1>(md));
          md = max_nan(md, dpp_d<0x4E>(md));
          md = max_nan(md, dpp_d<0x141>(md));
          md = max_nan(md, dpp_d<0x140>(md));
          scale = (float)(md / (double)kE4M3Max);
          const double inv_d = 1.0 / (double)scale;
          float f[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] = (float)(yd[c] * inv_d);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], q[i], false);
            q[i] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], q[i], true);
          }
          if ((again >> (lane_id() & 48) & 0xffff) != 0) leave(q, scale);
        }
      } else {
        if (nd > 0 && live) vec_store<T, 8>(static_cast<T*>(p.y) + row * p.dim + d, nd, y);
      }
    }
  }
}

// Gradient at h:  u = dy silu(gate) w,  dh = r (u - n mean(u n)) + d_res with
// n = h r;  dw = sum of dy silu(gate) n over the rows;  dgate = dy n w silu'.
// Persistent workgroups keep their rows' sums for dw in registers and leave
// one partial row each; a second kernel adds those in order.  The next row is
// on its way while one is worked on: 16384 x 4096 with d_res in bf16 take 96 us
// (5.6 TB/s, the rate of a copy), 131 without that and with more workgroups
// than are resident at once.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_bwd(NormParams p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  __shared__ float red[2][NT / 64][2];
  __shared__ float fold[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * NV * 8 : 1];
  const int t = threadIdx.x & (TPR - 1), sub = threadIdx.x / TPR;
  typedef typename VecIO<T, 8>::raw raw_t;
  float dw[NV][8];
  raw_t wr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * TPR + t) * 8;
    wr[v] = vec_raw<T, 8>(static_cast<const T*>(p.weight) + d, max(0, p.dim - d));
#pragma unroll
    for (int c = 0; c < 8; ++c) dw[v][c] = 0.f;
  }
  const float inv = p.inv_dim;
  const bool gate = p.gate != nullptr, dres = p.dres != nullptr;
  raw_t hn[NV], gn[NV], zn[NV], sn[NV];   // the next step's row, on its way
  auto fetch = [&](long row) {
    const long rr = row < p.rows ? row : 0;
    const T* h = static_cast<const T*>(p.x) + row_at(rr, p.inner, p.xo, p.xi);
    const T* dy = static_cast<const T*>(p.dy) + rr * p.dim;
    const T* z = static_cast<const T*>(p.gate) + (gate ? row_at(rr, p.inner, p.go, p.gi) : 0);
    const T* s = static_cast<const T*>(p.dres) + rr * p.dim;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = max(0, p.dim - d);
      hn[v] = vec_raw<T, 8>(h + d, nd);
      gn[v] = vec_raw<T, 8>(dy + d, nd);
      if (gate) zn[v] = vec_raw<T, 8>(z + d, nd);
      if (dres) sn[v] = vec_raw<T, 8>(s + d, nd);
    }
  };
  // 1024 lanes have 128 registers each: no room for a second row
  constexpr bool AHEAD = TPR < 1024;
  const long step = (long)gridDim.x * RPB;
  int buf = 0;
  if (AHEAD && (long)blockIdx.x * RPB < p.rows) fetch((long)blockIdx.x * RPB + sub);
  // every thread of the workgroup makes the same number of steps (barriers)
  for (long base = (long)blockIdx.x * RPB; base < p.rows; base += step, buf ^= 1) {
    const long row = base + sub;
    const bool live = row < p.rows;
    if (!AHEAD) fetch(row);
    float hf[NV][8], g[NV][8];
    raw_t zr[NV], sr[NV];
    float ss = 0.f, su = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w[8];
      VecIO<T, 8>::up(hn[v], hf[v]);
      VecIO<T, 8>::up(gn[v], g[v]);
      VecIO<T, 8>::up(wr[v], w);
      zr[v] = zn[v];
      sr[v] = sn[v];
      if (gate) {
        float z[8];
        VecIO<T, 8>::up(zr[v], z);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          ss = fmaf(hf[v][c], hf[v][c], ss);
          su = fmaf(g[v][c] * (z[c] * sigmoid_f(z[c])) * w[c], hf[v][c], su);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          ss = fmaf(hf[v][c], hf[v][c], ss);
          su = fmaf(g[v][c] * w[c], hf[v][c], su);
        }
      }
    }
    if (AHEAD && base + step < p.rows) fetch(row + step);
    row_sum2<TPR>(ss, su, red[buf]);   // two buffers: the next step's sums do not meet this step's readers
    const float r = rsqrt_f(fmaf(ss, inv, p.eps));
    const float m = su * r * inv;      // mean(u n)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = min(8, p.dim - d);
      float w[8], o[8];
      VecIO<T, 8>::up(wr[v], w);
      if (gate) {
        float z[8], dz[8];
        VecIO<T, 8>::up(zr[v], z);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float s = sigmoid_f(z[c]);
          dz[c] = g[v][c] * hf[v][c] * r * w[c] * (s * fmaf(z[c], 1.f - s, 1.f));
          g[v][c] *= z[c] * s;
        }
        if (live && nd > 0) vec_store<T, 8>(static_cast<T*>(p.dgate) + row * p.dim + d, nd, dz);
      }
      float s[8];
      if (dres) VecIO<T, 8>::up(sr[v], s);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float n = hf[v][c] * r;
        o[c] = r * (g[v][c] * w[c] - n * m) + (dres ? s[c] : 0.f);
        dw[v][c] += live ? g[v][c] * n : 0.f;
      }
      if (live && nd > 0) vec_store<T, 8>(static_cast<T*>(p.dh) + row * p.dim + d, nd, o);
    }
  }
  float* part = p.part + (long)blockIdx.x * p.dim;
  if constexpr (RPB > 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int c = 0; c < 8; ++c) fold[sub][(v * TPR + t) * 8 + c] = dw[v][c];
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += NT) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < RPB; ++i) s += fold[i][d];
      part[d] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = min(8, p.dim - d);
      if (nd > 0) vec_store<float, 8>(part + d, nd, dw[v]);
    }
  }
}

// dw: the workgroups' partial rows, in 64 strands of every 64th that are then
// added in order; 32 columns a workgroup (128-byte pieces of a row) keep the
// strands short and many compute units busy (512 x 4096: 5 us; 16 columns of
// 1024 rows a workgroup took 18).
template <typename T>
__global__ __launch_bounds__(512) void k_norm_dw(NormParams p) {
  __shared__ f32x4 acc[64][8];
  const int c = threadIdx.x & 7, strand = threadIdx.x >> 3;
  const int d = blockIdx.x * 32 + 4 * c, nd = min(4, p.dim - d);
  f32x4 s = zero4();
  if (nd > 0)
    for (int b = strand; b < p.blocks; b += 64) {
      float f[4];
      vec_load<float, 4>(p.part + (long)b * p.dim + d, nd, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += f[e];
    }
  acc[strand][c] = s;
  __syncthreads();
  if (strand != 0 || nd <= 0) return;
  s = zero4();
#pragma unroll 8
  for (int i = 0; i < 64; ++i) s += acc[i][c];
  const float o[4] = {s[0], s[1], s[2], s[3]};
  vec_store<T, 4>(static_cast<T*>(p.dw) + d, nd, o);
}

// Lanes per row and vectors per lane by the row's length.
#define NORM_DISPATCH(CALL)                    \
  if (p.dim <= 128) { CALL(16, 1); }           \
  else if (p.dim <= 256) { CALL(32, 1); }      \
  else if (p.dim <= 512) { CALL(64, 1); }      \
  else if (p.dim <= 1024) { CALL(128, 1); }    \
  else if (p.dim <= 2048) { CALL(256, 1); }    \
  else if (p.dim <= 4096) { CALL(256, 2); }    \
  else if (p.dim <= 8192) { CALL(512, 2); }    \
  else { CALL(1024, 2); }

template <typename T, int TPR, int NV, int R, bool QUANT>
static void norm_fwd_launch(const NormParams& p, hipStream_t st) {
  constexpr int NT = TPR < 256 ? 256 : TPR;
  const long per = (long)R * (NT / TPR);
  hipLaunchKernelGGL((k_norm_fwd<T, TPR, NV, R, QUANT>), dim3((unsigned)((p.rows + per - 1) / per)), dim3(NT), 0, st, p);
}
// Two rows a lane group where that still leaves eight workgroups a compute unit
// (262144 rows, bf16: 128 values with a gate 34.8 us, with one row 36.1; 64
// values without 18.8, with one 20.7).  To 8 bits both take the same, as the
// second look at values next to a border takes the registers: one row.
template <typename T, int TPR, int NV, bool QUANT>
static void norm_fwd_rows(const NormParams& p, hipStream_t st) {
  if constexpr (TPR <= 64 && !QUANT) {
    if (p.rows >= 2L * (256 / TPR) * 8 * kComputeUnits) return norm_fwd_launch<T, TPR, NV, 2, QUANT>(p, st);
  }
  norm_fwd_launch<T, TPR, NV, 1, QUANT>(p, st);
}
template <typename T, bool QUANT>
static hipError_t norm_fwd(const NormParams& p, hipStream_t st) {
  timing_before("norm_fwd", st);
#define CALL(TPR, NV) norm_fwd_rows<T, TPR, NV, QUANT>(p, st)
  NORM_DISPATCH(CALL);
#undef CALL
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_norm_fwd(DType dt, bool quant, const NormParams& p, hipStream_t st) {
  if (dt == DType::BF16) return quant ? norm_fwd<bf16, true>(p, st) : norm_fwd<bf16, false>(p, st);
  return quant ? norm_fwd<float, true>(p, st) : norm_fwd<float, false>(p, st);
}

// Workgroups of the backward: as many as are resident at once by the registers
// they take, fewer where the rows end first.
static int norm_rows_per_block(int dim) { return dim <= 128 ? 16 : dim <= 256 ? 8 : dim <= 512 ? 4 : dim <= 1024 ? 2 : 1; }
int norm_bwd_blocks(long rows, int dim) {
  const long want = dim <= 2048 ? 4 * kComputeUnits : dim <= 4096 ? 2 * kComputeUnits : kComputeUnits;
  const long most = (rows + norm_rows_per_block(dim) - 1) / norm_rows_per_block(dim);
  return (int)(most < want ? most : want);
}
template <typename T>
static hipError_t norm_bwd(const NormParams& p, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (p.blocks > 0) {
    timing_before("norm_bwd", st);
#define CALL(TPR, NV) \
  hipLaunchKernelGGL((k_norm_bwd<T, TPR, NV>), dim3((unsigned)p.blocks), dim3(TPR < 256 ? 256 : TPR), 0, st, p)
    NORM_DISPATCH(CALL);
#undef CALL
    e = hipGetLastError();
    timing_after(st);
    if (e != hipSuccess) return e;
  }
  timing_before("norm_dw", st);
  hipLaunchKernelGGL(k_norm_dw<T>, dim3((unsigned)((p.dim + 31) / 32)), dim3(512), 0, st, p);
  e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_norm_bwd(DType dt, const NormParams& p, hipStream_t st) {
  return dt == DType::BF16 ? norm_bwd<bf16>(p, st) : norm_bwd<float>(p, st);
}

}  // namespace gdr
