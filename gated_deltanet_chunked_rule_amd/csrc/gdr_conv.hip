// gdr_conv.hip -- short causal convolution: prompts, gradient, single tokens.
//
//   z_t = bias + sum_j w_j x_{t-W+1+j},   y_t = z_t or z_t sigmoid(z_t)
//
// All three are bound by memory: a thread owns VEC channels and walks down the
// tokens of a tile with the last W - 1 inputs in registers, so every input is
// read once (and W - 1 rows again at a tile's start).  8192 tokens x 8192
// channels in bf16 take 53 us (5.1 TB/s), the gradient of 32768 x 8192 338
// and 14 for its sums (4.6 TB/s), one token of 128 sequences 5.7 us, of which
// about 3 are a launch's own.
#include "gdr_layer.h"

namespace gdr {

template <typename T, int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvParams& p, int d, int nd, float (&w)[W][VEC], float (&b)[VEC]) {
  const T* wp = static_cast<const T*>(p.weight) + (long)d * W;
  float f[VEC * W];
#pragma unroll
  for (int i = 0; i < VEC * W / 4; ++i) {
    float q[4];
    vec_load<T, 4>(wp + 4 * i, max(0, min(4, nd * W - 4 * i)), q);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[4 * i + e] = q[e];
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][c] = f[c * W + j];
  if (p.bias) {
    vec_load<T, VEC>(static_cast<const T*>(p.bias) + d, nd, b);
  } else {
#pragma unroll
    for (int c = 0; c < VEC; ++c) b[c] = 0.f;
  }
}

// Row `t` of the extended input of the sequence that starts at `start`: an
// input token, or a row of the initial state before it.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_ext(const ConvParams& p, int n, int start, int t, int d, int nd, float (&f)[VEC]) {
  if (t >= start) {
    vec_load<T, VEC>(static_cast<const T*>(p.x) + (long)t * p.x_stride + d, nd, f);
  } else if (p.h0) {
    vec_load<T, VEC>(static_cast<const T*>(p.h0) + ((long)n * (W - 1) + (W - 1 + t - start)) * p.D + d, nd, f);
  } else {
#pragma unroll
    for (int c = 0; c < VEC; ++c) f[c] = 0.f;
  }
}

// Work items: (tile, channel group), channel groups fastest; then, where a
// final state is asked for, (sequence, channel group).
template <typename T, int W>
__global__ __launch_bounds__(256) void k_conv_fwd(ConvParams p) {
  constexpr int VEC = 8, U = 4;
  __shared__ int32_t cu_lds[kCuLds];
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  const int ncg = (p.D + VEC - 1) / VEC;
  const long item = (long)blockIdx.x * 256 + threadIdx.x;
  const long tile = item / ncg;
  const int d = (int)(item - tile * ncg) * VEC, nd = min(VEC, p.D - d);
  T* y = static_cast<T*>(p.y);
  if (tile >= p.tiles) {
    const long n = tile - p.tiles;
    if (!p.ht || n >= p.s.N) return;
    const int start = sf.at((int)n), end = max(start, sf.at((int)n + 1));
    T* out = static_cast<T*>(p.ht) + n * (W - 1) * p.D + d;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      float f[VEC];
      load_ext<T, VEC, W>(p, (int)n, start, end - (W - 1) + i, d, nd, f);
      vec_store<T, VEC>(out + (long)i * p.D, nd, f);
    }
    return;
  }
  float w[W][VEC], b[VEC];
  load_taps<T, VEC, W>(p, d, nd, w, b);
  const T* x = static_cast<const T*>(p.x) + d;
  int t = (int)tile * p.tile;
  const int t1 = min(t + p.tile, p.s.Ttot);
  while (t < t1) {
    int start, end;
    const int n = sf.find(t, start, end);
    end = min(end, t1);
    if (n < 0) {
      const float zero[VEC] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (; t < end; ++t) vec_store<T, VEC>(y + (long)t * p.D + d, nd, zero);
      continue;
    }
    float xs[W - 1 + U][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) load_ext<T, VEC, W>(p, n, start, t - (W - 1) + i, d, nd, xs[i]);
    for (; t < end; t += U) {
      typename VecIO<T, VEC>::raw r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = vec_raw<T, VEC>(x + (long)min(t + u, end - 1) * p.x_stride, nd);
#pragma unroll
      for (int u = 0; u < U; ++u) VecIO<T, VEC>::up(r[u], xs[W - 1 + u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float z[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          z[c] = b[c];
#pragma unroll
          for (int j = 0; j < W; ++j) z[c] = fmaf(w[j][c], xs[u + j][c], z[c]);
          if (p.act) z[c] *= sigmoid_f(z[c]);
        }
        if (t + u < end) vec_store<T, VEC>(y + (long)(t + u) * p.D + d, nd, z);
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) xs[i][c] = xs[U + i][c];
    }
    t = end;
  }
}

// Gradient.  A thread walks its tile's tokens and W - 1 beyond it (inside the
// sequence), recomputing z; dx_t leaves once dz_{t + W - 1} is known, and the
// tile's own tokens add to its partial sums of dw and db, which a second
// kernel adds over the tiles in order.  Four channels a thread: the windows,
// taps and sums of eight would leave two waves a SIMD.
template <typename T, int W>
__global__ __launch_bounds__(256) void k_conv_bwd(ConvParams p) {
  constexpr int VEC = 4;
  __shared__ int32_t cu_lds[kCuLds];
  const SeqFinder sf = seq_finder(p.s, cu_lds);
  const int ncg = (p.D + VEC - 1) / VEC;
  const long item = (long)blockIdx.x * 256 + threadIdx.x;
  const long tile = item / ncg;
  const int d = (int)(item - tile * ncg) * VEC, nd = min(VEC, p.D - d);
  const T* x = static_cast<const T*>(p.x) + d;
  const T* dy = static_cast<const T*>(p.dy) + d;
  T* dx = static_cast<T*>(p.dx) + d;
  const T* dht = static_cast<const T*>(p.dht);
  if (tile >= p.tiles + (p.dh0 ? p.s.N : 0)) return;
  float w[W][VEC], b[VEC];
  load_taps<T, VEC, W>(p, d, nd, w, b);
  auto dact = [&](const float (&win)[W][VEC], const float (&g)[VEC], float (&dz)[VEC]) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      float z = b[c];
#pragma unroll
      for (int j = 0; j < W; ++j) z = fmaf(w[j][c], win[j][c], z);
      if (p.act) {
        const float s = sigmoid_f(z);
        dz[c] = g[c] * (s * fmaf(z, 1.f - s, 1.f));
      } else {
        dz[c] = g[c];
      }
    }
  };
  if (tile >= p.tiles) {
    // dh0 row i meets tap j of token i - j; rows that the final state still
    // holds (sequences shorter than W - 1) get its gradient too
    const int n = (int)(tile - p.tiles);
    const int start = sf.at(n), len = max(0, sf.at(n + 1) - start);
    float g0[W - 1][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) g0[i][c] = 0.f;
      if (dht && i >= len) vec_load<T, VEC>(dht + ((long)n * (W - 1) + i - len) * p.D + d, nd, g0[i]);
    }
#pragma unroll
    for (int u = 0; u < W - 1; ++u) {
      if (u < len) {
        float win[W][VEC], g[VEC], dz[VEC];
#pragma unroll
        for (int j = 0; j < W; ++j) load_ext<T, VEC, W>(p, n, start, start + u - (W - 1) + j, d, nd, win[j]);
        vec_load<T, VEC>(dy + (long)(start + u) * p.D, nd, g);
        dact(win, g, dz);
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (u + j < W - 1)
#pragma unroll
            for (int c = 0; c < VEC; ++c) g0[u + j][c] = fmaf(w[j][c], dz[c], g0[u + j][c]);
      }
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) vec_store<T, VEC>(static_cast<T*>(p.dh0) + ((long)n * (W - 1) + i) * p.D + d, nd, g0[i]);
    return;
  }
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    db[c] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][c] = 0.f;
  }
  int t = (int)tile * p.tile;
  const int t1 = min(t + p.tile, p.s.Ttot);
  while (t < t1) {
    int start, end;
    const int n = sf.find(t, start, end);
    const int own_end = min(end, t1);
    if (n < 0) {
      const float zero[VEC] = {0.f, 0.f, 0.f, 0.f};
      for (; t < own_end; ++t) vec_store<T, VEC>(dx + (long)t * p.D, nd, zero);
      continue;
    }
    constexpr int U = 4;
    float win[W - 1 + U][VEC];       // inputs u - W + 1 .. u + U - 1
    float dzs[W - 1 + U][VEC];       // dz of the same tokens (zero outside the run)
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      load_ext<T, VEC, W>(p, n, start, t - (W - 1) + i, d, nd, win[i]);
#pragma unroll
      for (int c = 0; c < VEC; ++c) dzs[i][c] = 0.f;
    }
    // a step of U tokens: their loads together, then the work of each
    auto load_step = [&](int u0, typename VecIO<T, VEC>::raw (&rx)[U], typename VecIO<T, VEC>::raw (&rg)[U]) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = min(u0 + i, end - 1);
        rx[i] = vec_raw<T, VEC>(x + (long)v * p.x_stride, nd);
        rg[i] = vec_raw<T, VEC>(dy + (long)v * p.D, nd);
      }
    };
    const int stop = own_end + W - 1;   // dx of own_end - 1 needs dz up to stop - 1
    for (int u0 = t; u0 < stop; u0 += U) {
      typename VecIO<T, VEC>::raw rx[U], rg[U];
      load_step(u0, rx, rg);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int u = u0 + i;
        float g[VEC], dz[VEC];
        VecIO<T, VEC>::up(rx[i], win[W - 1 + i]);
        VecIO<T, VEC>::up(rg[i], g);
        float wv[W][VEC];
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int c = 0; c < VEC; ++c) wv[j][c] = win[i + j][c];
        dact(wv, g, dz);
        const bool in = u < end;          // tokens of this sequence
        const bool mine = u < own_end;    // tokens of this tile
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          dz[c] = in ? dz[c] : 0.f;
          dzs[W - 1 + i][c] = dz[c];
          if (mine) {
            db[c] += dz[c];
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][c] = fmaf(dz[c], wv[j][c], dw[j][c]);
          }
        }
        const int td = u - (W - 1);
        if (td >= t && td < own_end) {
          float gx[VEC];
#pragma unroll
          for (int c = 0; c < VEC; ++c) gx[c] = 0.f;
          if (dht && td >= end - (W - 1)) vec_load<T, VEC>(dht + ((long)n * (W - 1) + td - (end - (W - 1))) * p.D + d, nd, gx);
#pragma unroll
          for (int c = 0; c < VEC; ++c)
#pragma unroll
            for (int j = 0; j < W; ++j) gx[c] = fmaf(w[j][c], dzs[i + W - 1 - j][c], gx[c]);
          vec_store<T, VEC>(dx + (long)td * p.D, nd, gx);
        }
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          win[i][c] = win[U + i][c];
          dzs[i][c] = dzs[U + i][c];
        }
    }
    t = own_end;
  }
  float* part = p.part + tile * (long)(W + 1) * p.D + d;
#pragma unroll
  for (int j = 0; j < W; ++j) vec_store<float, VEC>(part + (long)j * p.D, nd, dw[j]);
  vec_store<float, VEC>(part + (long)W * p.D, nd, db);
}

// dw[d][j], db[d]: the tiles' partial sums, in 32 strands of every 32nd tile
// that are then added in order; 32 columns a workgroup (128-byte pieces).
template <typename T, int W>
__global__ __launch_bounds__(256) void k_conv_dw(ConvParams p) {
  __shared__ f32x4 acc[32][W + 1][8];
  const int lane = threadIdx.x & 7, strand = threadIdx.x >> 3;
  const int d = blockIdx.x * 32 + 4 * lane, nd = min(4, p.D - d);
  f32x4 s[W + 1];
#pragma unroll
  for (int j = 0; j <= W; ++j) s[j] = zero4();
  if (nd > 0)
    for (int tile = strand; tile < p.tiles; tile += 32) {
      const float* q = p.part + (long)tile * (W + 1) * p.D + d;
#pragma unroll
      for (int j = 0; j <= W; ++j) {
        float f[4];
        vec_load<float, 4>(q + (long)j * p.D, nd, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] += f[e];
      }
    }
#pragma unroll
  for (int j = 0; j <= W; ++j) acc[strand][j][lane] = s[j];
  __syncthreads();
  // thread (j, column group) adds the strands
  const int j = threadIdx.x >> 3;
  if (j > W || nd <= 0) return;
  f32x4 v = zero4();
#pragma unroll 8
  for (int i = 0; i < 32; ++i) v += acc[i][j][lane];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < nd) {
      if (j < W) static_cast<T*>(p.dw)[(long)(d + e) * W + j] = from_f<T>(v[e]);
      else if (p.db) static_cast<T*>(p.db)[d + e] = from_f<T>(v[e]);
    }
}

// One new token per row: blocks of one wave walk the channels of one row.
template <typename T, int W>
__global__ __launch_bounds__(64) void k_conv_step(ConvParams p, int blocks_per_row) {
  constexpr int VEC = 8;
  const int row = blockIdx.x / blocks_per_row;
  const int d = ((blockIdx.x - row * blocks_per_row) * 64 + lane_id()) * VEC;
  const int nd = min(VEC, p.D - d);
  const int slot = step_slot(p.slots, row, p.num_slots);
  if (nd <= 0) return;
  T* y = static_cast<T*>(p.y) + (long)row * p.D + d;
  float z[VEC];
  if (slot < 0) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) z[c] = 0.f;
    vec_store<T, VEC>(y, nd, z);
    return;
  }
  T* state = static_cast<T*>(p.state) + (long)slot * (W - 1) * p.D + d;
  typename VecIO<T, VEC>::raw r[W];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) r[i] = vec_raw<T, VEC>(state + (long)i * p.D, nd);
  r[W - 1] = vec_raw<T, VEC>(static_cast<const T*>(p.x) + (long)row * p.x_stride + d, nd);
  float w[W][VEC];
  load_taps<T, VEC, W>(p, d, nd, w, z);
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float f[VEC];
    VecIO<T, VEC>::up(r[j], f);
#pragma unroll
    for (int c = 0; c < VEC; ++c) z[c] = fmaf(w[j][c], f[c], z[c]);
    if (j > 0) vec_store<T, VEC>(state + (long)(j - 1) * p.D, nd, f);
  }
  if (p.act)
#pragma unroll
    for (int c = 0; c < VEC; ++c) z[c] *= sigmoid_f(z[c]);
  vec_store<T, VEC>(y, nd, z);
}

// Tokens per tile: as long as the tiles still give every SIMD several waves.
static int tile_for(long groups, int tokens, long threads, int lo, int hi) {
  int tile = hi;
  while (tile > lo && groups * ((tokens + tile - 1) / tile) < threads) tile /= 2;
  return tile;
}
// The gradient: 32768 x 8192 take 338 + 14 us (sums) in tiles of 128 tokens, 354
// + 9 in tiles of 256, 368 + 7 in tiles of 512.
int conv_bwd_tile(int tokens, int D) { return tile_for((D + 3) / 4, tokens, 1L << 19, 16, 256); }

template <typename T, int W>
static hipError_t conv_fwd(ConvParams p, hipStream_t st) {
  const long ncg = (p.D + 7) / 8;
  p.tile = tile_for(ncg, p.s.Ttot, 1L << 18, 4, 32);
  p.tiles = (p.s.Ttot + p.tile - 1) / p.tile;
  const long items = ncg * (p.tiles + (p.ht ? p.s.N : 0));
  if (items == 0) return hipSuccess;
  timing_before("conv_fwd", st);
  hipLaunchKernelGGL((k_conv_fwd<T, W>), dim3((unsigned)((items + 255) / 256)), dim3(256), 0, st, p);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
template <typename T, int W>
static hipError_t conv_bwd(const ConvParams& p, hipStream_t st) {
  const long ncg = (p.D + 3) / 4;
  const long items = ncg * (p.tiles + (p.dh0 ? p.s.N : 0));
  hipError_t e = hipSuccess;
  if (items > 0) {
    timing_before("conv_bwd", st);
    hipLaunchKernelGGL((k_conv_bwd<T, W>), dim3((unsigned)((items + 255) / 256)), dim3(256), 0, st, p);
    e = hipGetLastError();
    timing_after(st);
    if (e != hipSuccess) return e;
  }
  timing_before("conv_dw", st);
  hipLaunchKernelGGL((k_conv_dw<T, W>), dim3((unsigned)((p.D + 31) / 32)), dim3(256), 0, st, p);
  e = hipGetLastError();
  timing_after(st);
  return e;
}
template <typename T, int W>
static hipError_t conv_step(int rows, const ConvParams& p, hipStream_t st) {
  const int per = (p.D + 511) / 512;
  timing_before("conv_step", st);
  hipLaunchKernelGGL((k_conv_step<T, W>), dim3((unsigned)rows * per), dim3(64), 0, st, p, per);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}

#define CONV_DISPATCH(fn, ...)                                              \
  if (dt == DType::BF16) {                                                  \
    if (W == 2) return fn<bf16, 2>(__VA_ARGS__);                            \
    return W == 3 ? fn<bf16, 3>(__VA_ARGS__) : fn<bf16, 4>(__VA_ARGS__);    \
  }                                                                         \
  if (W == 2) return fn<float, 2>(__VA_ARGS__);                             \
  return W == 3 ? fn<float, 3>(__VA_ARGS__) : fn<float, 4>(__VA_ARGS__)

hipError_t launch_conv_fwd(DType dt, int W, const ConvParams& p, hipStream_t st) { CONV_DISPATCH(conv_fwd, p, st); }
hipError_t launch_conv_bwd(DType dt, int W, const ConvParams& p, hipStream_t st) { CONV_DISPATCH(conv_bwd, p, st); }
hipError_t launch_conv_step(DType dt, int W, int rows, const ConvParams& p, hipStream_t st) { CONV_DISPATCH(conv_step, rows, p, st); }

}  // namespace gdr
