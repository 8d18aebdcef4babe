// gdr_block_norm.hip -- the norm behind a block with its gate and scale, the
// residual's addition and the norm before the next block, in one pass; their
// gradient; and the sums over partial rows that gradients of vectors end in.
//
//   p = x / rms(x) w_post silu(gate),  h = residual + scale p,  y = h / rms(h) w_pre
//   rms(v) = sqrt(mean(v^2) + eps)
//
// Bound by memory: TPR lanes hold a row's operands in registers (NV vectors of
// 8 values each), so every operand is read once and the row's two sums need
// nothing from memory.  Sums are fp32 over unrounded values; y is made from the
// unrounded h.
#include "gdr_layer.h"

namespace gdr {

// Sums of N values over the TPR lanes of a row (a power of two, 16 to 1024),
// the same on every lane; rows of more than a wave meet in LDS.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&a)[N], float (*lds)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = row16_sum(a[i]);
#pragma unroll
    for (int m = 16; m < (TPR < 64 ? TPR : 64); m <<= 1) a[i] += __shfl_xor(a[i], m);
  }
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    if (lane_id() == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) lds[w][i] = a[i];
    lds_barrier();
    const int first = (threadIdx.x / TPR) * (TPR / 64);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = 0.f;
#pragma unroll
      for (int j = 0; j < TPR / 64; ++j) a[i] += lds[first + j][i];
    }
  }
}

template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_block_norm_fwd(BlockNormParams p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  typedef typename VecIO<T, 8>::raw raw_t;
  __shared__ float red[2][NT / 64][1];
  const int t = threadIdx.x & (TPR - 1);
  const long row = (long)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < p.rows;   // rows behind the last read row 0 and write nothing
  const long rr = live ? row : 0;
  const T* x = static_cast<const T*>(p.x) + rr * p.x_stride;
  const T* res = static_cast<const T*>(p.residual) + rr * p.r_stride;
  const T* gate = static_cast<const T*>(p.gate) + rr * p.g_stride;
  raw_t xr[NV], sr[NV], zr[NV], wr[NV], cr[NV], vr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * TPR + t) * 8, nd = max(0, p.dim - d);
    xr[v] = vec_raw<T, 8>(x + d, nd);
    sr[v] = vec_raw<T, 8>(res + d, nd);
    if (p.gate) zr[v] = vec_raw<T, 8>(gate + d, nd);
    wr[v] = vec_raw<T, 8>(static_cast<const T*>(p.post) + d, nd);
    if (p.scale) cr[v] = vec_raw<T, 8>(static_cast<const T*>(p.scale) + d, nd);
    vr[v] = vec_raw<T, 8>(static_cast<const T*>(p.pre) + d, nd);
  }
  float h[NV][8], ss[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    VecIO<T, 8>::up(xr[v], h[v]);
#pragma unroll
    for (int c = 0; c < 8; ++c) ss[0] = fmaf(h[v][c], h[v][c], ss[0]);
  }
  row_sums<TPR, 1>(ss, red[0]);
  const float rx = __builtin_amdgcn_rsqf(fmaf(ss[0], p.inv_dim, p.eps));   // an ulp
  ss[0] = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float w[8], s[8];
    VecIO<T, 8>::up(wr[v], w);
    VecIO<T, 8>::up(sr[v], s);
#pragma unroll
    for (int c = 0; c < 8; ++c) h[v][c] = h[v][c] * rx * w[c];
    if (p.gate) {
      float z[8];
      VecIO<T, 8>::up(zr[v], z);
#pragma unroll
      for (int c = 0; c < 8; ++c) h[v][c] *= z[c] * sigmoid_f(z[c]);
    }
    if (p.scale) {
      float k[8];
      VecIO<T, 8>::up(cr[v], k);
#pragma unroll
      for (int c = 0; c < 8; ++c) h[v][c] = fmaf(h[v][c], k[c], s[c]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) h[v][c] += s[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) ss[0] = fmaf(h[v][c], h[v][c], ss[0]);
  }
  row_sums<TPR, 1>(ss, red[1]);
  const float rh = __builtin_amdgcn_rsqf(fmaf(ss[0], p.inv_dim, p.eps));
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * TPR + t) * 8, nd = min(8, p.dim - d);
    if (!live || nd <= 0) continue;
    float w[8];
    VecIO<T, 8>::up(vr[v], w);
    vec_store<T, 8>(static_cast<T*>(p.h_out) + row * p.dim + d, nd, h[v]);
#pragma unroll
    for (int c = 0; c < 8; ++c) h[v][c] = h[v][c] * rh * w[c];
    vec_store<T, 8>(static_cast<T*>(p.y) + row * p.dim + d, nd, h[v]);
  }
}

// Gradient at x and h, from dy and the gradient of h from elsewhere:
//   n = h rh,  u = dy w_pre,  dh = rh (u - n mean(u n)) + d_res   (of residual too)
//   q = x rx,  c = silu(gate),  dp = dh scale c,  v = dp w_post
//   dx = rx (v - q mean(v q)),  dgate = dh scale q w_post silu'(gate)
//   dw_pre = sum dy n,  dw_post = sum dp q,  dscale = sum dh q w_post c
// Persistent workgroups keep the three vectors' sums in registers and leave one
// partial row of each.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_block_norm_bwd(BlockNormParams p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  typedef typename VecIO<T, 8>::raw raw_t;
  __shared__ float red3[2][NT / 64][3];
  __shared__ float red1[2][NT / 64][1];
  __shared__ float fold[RPB > 1 ? RPB : 1][RPB > 1 ? TPR * NV * 8 : 1];
  const int t = threadIdx.x & (TPR - 1), sub = threadIdx.x / TPR;
  const bool gate = p.gate != nullptr, scale = p.scale != nullptr, dres = p.dres != nullptr;
  raw_t post[NV], pre[NV], sc[NV];
  float dpost[NV][8], dpre[NV][8], dsc[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * TPR + t) * 8, nd = max(0, p.dim - d);
    post[v] = vec_raw<T, 8>(static_cast<const T*>(p.post) + d, nd);
    pre[v] = vec_raw<T, 8>(static_cast<const T*>(p.pre) + d, nd);
    if (scale) sc[v] = vec_raw<T, 8>(static_cast<const T*>(p.scale) + d, nd);
#pragma unroll
    for (int c = 0; c < 8; ++c) dpost[v][c] = dpre[v][c] = dsc[v][c] = 0.f;
  }
  int buf = 0;
  // every thread of the workgroup makes the same number of steps (barriers)
  for (long base = (long)blockIdx.x * RPB; base < p.rows; base += (long)gridDim.x * RPB, buf ^= 1) {
    const long row = base + sub;
    const bool live = row < p.rows;
    const long rr = live ? row : 0;
    const T* x = static_cast<const T*>(p.x) + rr * p.x_stride;
    const T* hh = static_cast<const T*>(p.h) + rr * p.r_stride;
    const T* z = static_cast<const T*>(p.gate) + rr * p.g_stride;
    raw_t xr[NV], hr[NV], yr[NV], zr[NV], sr[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = max(0, p.dim - d);
      hr[v] = vec_raw<T, 8>(hh + d, nd);
      yr[v] = vec_raw<T, 8>(static_cast<const T*>(p.dy) + rr * p.dim + d, nd);
      xr[v] = vec_raw<T, 8>(x + d, nd);
      if (gate) zr[v] = vec_raw<T, 8>(z + d, nd);
      if (dres) sr[v] = vec_raw<T, 8>(static_cast<const T*>(p.dres) + rr * p.dim + d, nd);
    }
    float s3[3] = {0.f, 0.f, 0.f};   // h^2, u h, x^2
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float h[8], g[8], w[8], q[8];
      VecIO<T, 8>::up(hr[v], h);
      VecIO<T, 8>::up(yr[v], g);
      VecIO<T, 8>::up(pre[v], w);
      VecIO<T, 8>::up(xr[v], q);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        s3[0] = fmaf(h[c], h[c], s3[0]);
        s3[1] = fmaf(g[c] * w[c], h[c], s3[1]);
        s3[2] = fmaf(q[c], q[c], s3[2]);
      }
    }
    row_sums<TPR, 3>(s3, red3[buf]);   // two buffers: the next row's sums do not meet this one's readers
    const float rh = __builtin_amdgcn_rsqf(fmaf(s3[0], p.inv_dim, p.eps)), mh = s3[1] * rh * p.inv_dim;
    const float rx = __builtin_amdgcn_rsqf(fmaf(s3[2], p.inv_dim, p.eps));
    float dh[NV][8], s1[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = min(8, p.dim - d);
      float h[8], g[8], w[8], q[8], wp[8], s[8], k[8], zz[8];
      VecIO<T, 8>::up(hr[v], h);
      VecIO<T, 8>::up(yr[v], g);
      VecIO<T, 8>::up(pre[v], w);
      VecIO<T, 8>::up(xr[v], q);
      VecIO<T, 8>::up(post[v], wp);
      if (dres) VecIO<T, 8>::up(sr[v], s);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float n = h[c] * rh;
        dh[v][c] = rh * (g[c] * w[c] - n * mh) + (dres ? s[c] : 0.f);
        dpre[v][c] += live ? g[c] * n : 0.f;
        q[c] *= rx;
      }
      if (live && nd > 0) vec_store<T, 8>(static_cast<T*>(p.dh) + row * p.dim + d, nd, dh[v]);
      if (scale) VecIO<T, 8>::up(sc[v], k);
      if (gate) {
        float dz[8];
        VecIO<T, 8>::up(zr[v], zz);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float e = sigmoid_f(zz[c]), cc = scale ? dh[v][c] * k[c] : dh[v][c];
          dz[c] = cc * q[c] * wp[c] * (e * fmaf(zz[c], 1.f - e, 1.f));
          zz[c] *= e;
        }
        if (live && nd > 0) vec_store<T, 8>(static_cast<T*>(p.dgate) + row * p.dim + d, nd, dz);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float act = gate ? dh[v][c] * zz[c] : dh[v][c];   // dh silu(gate)
        if (scale) dsc[v][c] += live ? act * q[c] * wp[c] : 0.f;
        const float dp = scale ? act * k[c] : act;
        dpost[v][c] += live ? dp * q[c] : 0.f;
        dh[v][c] = dp * wp[c];                                  // the gradient of q
        s1[0] = fmaf(dh[v][c], q[c], s1[0]);
      }
    }
    row_sums<TPR, 1>(s1, red1[buf]);
    const float mx = s1[0] * p.inv_dim;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * TPR + t) * 8, nd = min(8, p.dim - d);
      float q[8];
      VecIO<T, 8>::up(xr[v], q);
#pragma unroll
      for (int c = 0; c < 8; ++c) q[c] = rx * (dh[v][c] - q[c] * rx * mx);
      if (live && nd > 0) vec_store<T, 8>(static_cast<T*>(p.dx) + row * p.dim + d, nd, q);
    }
  }
  auto leave = [&](const float (&sum)[NV][8], float* part) __attribute__((always_inline)) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int c = 0; c < 8; ++c) fold[sub][(v * TPR + t) * 8 + c] = sum[v][c];
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
        if (nd > 0) vec_store<float, 8>(part + d, nd, sum[v]);
      }
    }
  };
  float* part = p.part + (long)blockIdx.x * (scale ? 3 : 2) * p.dim;
  leave(dpost, part);
  leave(dpre, part + p.dim);
  if (scale) leave(dsc, part + 2L * p.dim);
}

// Sums of partial rows, [rows][outputs][dim], in 64 strands of every 64th that
// are then added in order; 32 columns a workgroup.
template <typename T>
__global__ __launch_bounds__(512) void k_rows_sum(RowsSum p) {
  __shared__ f32x4 acc[64][8];
  const int c = threadIdx.x & 7, strand = threadIdx.x >> 3;
  const int d = blockIdx.x * 32 + 4 * c, nd = min(4, p.dim - d);
  const float* part = p.part + (long)blockIdx.y * p.dim + d;
  const long step = (long)gridDim.y * p.dim;
  f32x4 s = zero4();
  if (nd > 0)
    for (int b = strand; b < p.rows; b += 64) {
      float f[4];
      vec_load<float, 4>(part + b * step, nd, f);
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
  T* out = static_cast<T*>(blockIdx.y == 0 ? p.out[0] : blockIdx.y == 1 ? p.out[1] : p.out[2]);
  vec_store<T, 4>(out + d, nd, o);
}
hipError_t launch_rows_sum(DType dt, int outputs, const RowsSum& p, hipStream_t st) {
  timing_before("rows_sum", st);
  const dim3 grid((unsigned)((p.dim + 31) / 32), outputs);
  if (dt == DType::BF16) hipLaunchKernelGGL(k_rows_sum<bf16>, grid, dim3(512), 0, st, p);
  else hipLaunchKernelGGL(k_rows_sum<float>, grid, dim3(512), 0, st, p);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}

// Lanes per row and vectors per lane by the row's length.
#define BLOCK_NORM_DISPATCH(CALL)              \
  if (p.dim <= 128) { CALL(16, 1); }           \
  else if (p.dim <= 256) { CALL(32, 1); }      \
  else if (p.dim <= 512) { CALL(64, 1); }      \
  else if (p.dim <= 1024) { CALL(128, 1); }    \
  else if (p.dim <= 2048) { CALL(256, 1); }    \
  else if (p.dim <= 4096) { CALL(256, 2); }    \
  else if (p.dim <= 8192) { CALL(512, 2); }    \
  else { CALL(1024, 2); }

template <typename T>
static hipError_t block_norm_fwd(const BlockNormParams& p, hipStream_t st) {
  timing_before("block_norm_fwd", st);
#define CALL(TPR, NV)                                                                                          \
  constexpr int NT = TPR < 256 ? 256 : TPR;                                                                    \
  hipLaunchKernelGGL((k_block_norm_fwd<T, TPR, NV>), dim3((unsigned)((p.rows + NT / TPR - 1) / (NT / TPR))),   \
                     dim3(NT), 0, st, p)
  BLOCK_NORM_DISPATCH(CALL);
#undef CALL
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_block_norm_fwd(DType dt, const BlockNormParams& p, hipStream_t st) {
  return dt == DType::BF16 ? block_norm_fwd<bf16>(p, st) : block_norm_fwd<float>(p, st);
}

static int block_norm_rows_per_block(int dim) { return dim <= 128 ? 16 : dim <= 256 ? 8 : dim <= 512 ? 4 : dim <= 1024 ? 2 : 1; }
int block_norm_bwd_blocks(long rows, int dim) {
  const long want = dim <= 4096 ? 2 * kComputeUnits : kComputeUnits;
  const long most = (rows + block_norm_rows_per_block(dim) - 1) / block_norm_rows_per_block(dim);
  return (int)(most < want ? most : want);
}
template <typename T>
static hipError_t block_norm_bwd(const BlockNormParams& p, hipStream_t st) {
  if (p.blocks > 0) {
    timing_before("block_norm_bwd", st);
#define CALL(TPR, NV) \
  hipLaunchKernelGGL((k_block_norm_bwd<T, TPR, NV>), dim3((unsigned)p.blocks), dim3(TPR < 256 ? 256 : TPR), 0, st, p)
    BLOCK_NORM_DISPATCH(CALL);
#undef CALL
    const hipError_t e = hipGetLastError();
    timing_after(st);
    if (e != hipSuccess) return e;
  }
  RowsSum s = {};
  s.part = p.part;
  s.rows = p.blocks;
  s.dim = p.dim;
  s.out[0] = p.dpost;
  s.out[1] = p.dpre;
  s.out[2] = p.dscale;
  return launch_rows_sum(sizeof(T) == 2 ? DType::BF16 : DType::F32, p.scale ? 3 : 2, s, st);
}
hipError_t launch_block_norm_bwd(DType dt, const BlockNormParams& p, hipStream_t st) {
  return dt == DType::BF16 ? block_norm_bwd<bf16>(p, st) : block_norm_bwd<float>(p, st);
}

}  // namespace gdr
