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
//
// 16384 x 4096 in bf16 with gate and scale: 121 us (5.5 TB/s; plain streams, four
// read to two written, move 5.7), the gradient 211 (5.1; four to three 5.4) with
// its sums of partial rows 7; 64 rows 8.8 a call.
#include "gdr_layer.h"

namespace gdr {

// Sums of N values over the lanes of a row, the same on every lane: TPR lanes up
// to 256 (a power of two), the whole workgroup (of up to TPR lanes) from 512 on.
// Rows of more than a wave meet in LDS.
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
    if constexpr (TPR > 256) {
      const int u = threadIdx.x & 15;   // up to 16 waves: one a lane
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] = row16_sum(u < (int)(blockDim.x >> 6) ? lds[u][i] : 0.f);
    } else {
      const int first = (threadIdx.x / TPR) * (TPR / 64);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        a[i] = 0.f;
#pragma unroll
        for (int j = 0; j < TPR / 64; ++j) a[i] += lds[first + j][i];
      }
    }
  }
}
// Values from d on: one 32-bit offset in a register for all rows.
template <typename T, typename V> __device__ __forceinline__ T* values_at(V* row, int d) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
  return reinterpret_cast<T*>(reinterpret_cast<byte*>(row) + (uint32_t)d * (uint32_t)sizeof(T));
}
// A thread's place in its row, its row in the workgroup, and the lanes of a row.
template <int TPR> __device__ __forceinline__ int row_lane() { return TPR > 256 ? threadIdx.x : threadIdx.x & (TPR - 1); }
template <int TPR> __device__ __forceinline__ int row_sub() { return TPR > 256 ? 0 : threadIdx.x / TPR; }
template <int TPR> __device__ __forceinline__ int row_lanes() { return TPR > 256 ? blockDim.x : TPR; }

template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_block_norm_fwd(BlockNormParams p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  typedef typename VecIO<T, 8>::raw raw_t;
  __shared__ float red[2][NT / 64][1];
  const int t = row_lane<TPR>(), lanes = row_lanes<TPR>();
  const long row = (long)blockIdx.x * RPB + row_sub<TPR>();
  const bool live = row < p.rows;   // rows behind the last read row 0 and write nothing
  const long rr = live ? row : 0;
  const T* x = static_cast<const T*>(p.x) + rr * p.x_stride;
  const T* res = static_cast<const T*>(p.residual) + rr * p.r_stride;
  const T* gate = static_cast<const T*>(p.gate) + rr * p.g_stride;
  raw_t xr[NV], sr[NV], zr[NV], wr[NV], cr[NV], vr[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * lanes + t) * 8, nd = max(0, p.dim - d);
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
  const float rx = rsqrt_f(fmaf(ss[0], p.inv_dim, p.eps));
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
  const float rh = rsqrt_f(fmaf(ss[0], p.inv_dim, p.eps));
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * lanes + t) * 8, nd = min(8, p.dim - d);
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
  // From 8193 values on a lane has 128 registers.  LDS holds the sums of two of
  // the vectors, and row and vectors are read again (from L2) where they are used
  // a second time: 4096 x 16384 in bf16 464 us, 2048 x 16384 in fp32 370.  With x
  // for the gate and h for d_res 411 and 336, where all of it in registers (736
  // bytes a lane spilled) took 1516 and 805.
  constexpr bool BIG = TPR == 1024;
  __shared__ f32x4 far[BIG ? 2 * NV : 1][2][BIG ? TPR : 1];   // [sum and vector][half][lane]
  const int t = row_lane<TPR>(), sub = row_sub<TPR>(), lanes = row_lanes<TPR>();
  const bool gate = p.gate != nullptr, scale = p.scale != nullptr, dres = p.dres != nullptr;
  raw_t post[NV], pre[NV], sc[NV];
  float dpost[NV][8], dpre[NV][8], dsc[NV][8];
  auto vectors = [&](int v) __attribute__((always_inline)) {
    const int d = (v * lanes + t) * 8, nd = max(0, p.dim - d);
    post[v] = vec_raw<T, 8>(values_at<const T>(p.post, d), nd);
    pre[v] = vec_raw<T, 8>(values_at<const T>(p.pre, d), nd);
    sc[v] = vec_raw<T, 8>(values_at<const T>(p.scale, d), scale ? nd : 0);
  };
  // sums of a lane's own columns: no other lane reads or writes them
  auto far_sum = [&](int k, const float (&f)[8]) __attribute__((always_inline)) {
    far[k][0][t] += f32x4{f[0], f[1], f[2], f[3]};
    far[k][1][t] += f32x4{f[4], f[5], f[6], f[7]};
  };
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (BIG) far[2 * v][0][t] = far[2 * v][1][t] = far[2 * v + 1][0][t] = far[2 * v + 1][1][t] = zero4();
    else vectors(v);
#pragma unroll
    for (int c = 0; c < 8; ++c) dpost[v][c] = dpre[v][c] = dsc[v][c] = 0.f;
  }
  int buf = 0;
  // every thread of the workgroup makes the same number of steps (barriers)
  for (long base = (long)blockIdx.x * RPB; base < p.rows; base += (long)gridDim.x * RPB, buf ^= 1) {
    // a row of its own for the workgroup: in scalar registers, and not as one
    // running address of 64 bits a lane for each tensor and vector
    const long row = RPB == 1 ? (long)__builtin_amdgcn_readfirstlane((int)base) : base + sub;
    const bool live = row < p.rows;
    const long rr = live ? row : 0;
    const T* x = static_cast<const T*>(p.x) + rr * p.x_stride;
    const T* hh = static_cast<const T*>(p.h) + rr * p.r_stride;
    const T* z = static_cast<const T*>(p.gate) + rr * p.g_stride;
    raw_t xr[NV], hr[NV], yr[NV], zr[NV], sr[NV];
    auto sums_of = [&](int v) __attribute__((always_inline)) {   // what the first sums take
      const int d = (v * lanes + t) * 8, nd = max(0, p.dim - d);
      hr[v] = vec_raw<T, 8>(values_at<const T>(hh, d), nd);
      yr[v] = vec_raw<T, 8>(values_at<const T>(static_cast<const T*>(p.dy) + rr * p.dim, d), nd);
      xr[v] = vec_raw<T, 8>(values_at<const T>(x, d), nd);
    };
    auto others = [&](int v) __attribute__((always_inline)) {
      const int d = (v * lanes + t) * 8, nd = max(0, p.dim - d);
      zr[v] = vec_raw<T, 8>(values_at<const T>(z, d), gate ? nd : 0);
      sr[v] = vec_raw<T, 8>(values_at<const T>(static_cast<const T*>(p.dres) + rr * p.dim, d), dres ? nd : 0);
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      sums_of(v);
      if constexpr (!BIG) others(v);
    }
    float s3[3] = {0.f, 0.f, 0.f};   // h^2, u h, x^2
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (BIG) {
        asm volatile("" ::: "memory");
        vectors(v);
      }
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
    const float rh = rsqrt_f(fmaf(s3[0], p.inv_dim, p.eps)), mh = s3[1] * rh * p.inv_dim;
    const float rx = rsqrt_f(fmaf(s3[2], p.inv_dim, p.eps));
    float dh[NV][8], s1[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * lanes + t) * 8, nd = min(8, p.dim - d);
      if constexpr (BIG) vectors(v);
      if constexpr (BIG) {
        asm volatile("" ::: "memory");   // a second read, and not registers that hold the first
        sums_of(v);
        others(v);
      }
      float h[8], g[8], w[8], q[8], wp[8], s[8], k[8], z[8];
      VecIO<T, 8>::up(hr[v], h);
      VecIO<T, 8>::up(yr[v], g);
      VecIO<T, 8>::up(pre[v], w);
      VecIO<T, 8>::up(xr[v], q);
      VecIO<T, 8>::up(post[v], wp);
      VecIO<T, 8>::up(sr[v], s);
      VecIO<T, 8>::up(sc[v], k);
      VecIO<T, 8>::up(zr[v], z);
      float dz[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        // an absent vector counts as what leaves the others as they are, so that nothing here branches
        const float n = h[c] * rh, qc = q[c] * rx, e = sigmoid_f(z[c]), kc = scale ? k[c] : 1.f, act = gate ? z[c] * e : 1.f;
        const float f = rh * (g[c] * w[c] - n * mh) + s[c], qw = qc * wp[c], fq = f * qw;
        dz[c] = fq * kc * (e * fmaf(z[c], 1.f - e, 1.f));
        const float dp = f * act * kc;
        dh[v][c] = f;
        dpre[v][c] = (BIG ? 0.f : dpre[v][c]) + (live ? g[c] * n : 0.f);
        dpost[v][c] = (BIG ? 0.f : dpost[v][c]) + (live ? dp * qc : 0.f);
        dsc[v][c] += live ? fq * act : 0.f;
        h[c] = dp * wp[c];                                  // the gradient of q
        s1[0] = fmaf(h[c], qc, s1[0]);
      }
      if constexpr (BIG) {
        far_sum(2 * v, dpre[v]);
        far_sum(2 * v + 1, dpost[v]);
      }
      if (live && nd > 0) {
        vec_store<T, 8>(values_at<T>(static_cast<T*>(p.dh) + row * p.dim, d), nd, dh[v]);
        if (gate) vec_store<T, 8>(values_at<T>(static_cast<T*>(p.dgate) + row * p.dim, d), nd, dz);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) dh[v][c] = h[c];
    }
    row_sums<TPR, 1>(s1, red1[buf]);
    const float mx = s1[0] * p.inv_dim;
    if constexpr (BIG)
#pragma unroll
      for (int v = 0; v < NV; ++v) xr[v] = vec_raw<T, 8>(values_at<const T>(x, (v * lanes + t) * 8), max(0, p.dim - (v * lanes + t) * 8));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int d = (v * lanes + t) * 8, nd = min(8, p.dim - d);
      float q[8];
      VecIO<T, 8>::up(xr[v], q);
#pragma unroll
      for (int c = 0; c < 8; ++c) q[c] = rx * (dh[v][c] - q[c] * rx * mx);
      if (live && nd > 0) vec_store<T, 8>(values_at<T>(static_cast<T*>(p.dx) + row * p.dim, d), nd, q);
    }
  }
  auto leave = [&](const float (&sum)[NV][8], float* part) __attribute__((always_inline)) {
    if constexpr (RPB > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int c = 0; c < 8; ++c) fold[sub][(v * lanes + t) * 8 + c] = sum[v][c];
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
        const int d = (v * lanes + t) * 8, nd = min(8, p.dim - d);
        if (nd > 0) vec_store<float, 8>(part + d, nd, sum[v]);
      }
    }
  };
  if constexpr (BIG) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        dpre[v][c] = far[2 * v][c / 4][t][c % 4];
        dpost[v][c] = far[2 * v + 1][c / 4][t][c % 4];
      }
  }
  float* part = p.part + (long)blockIdx.x * (scale ? 3 : 2) * p.dim;
  leave(dpost, part);
  leave(dpre, part + p.dim);
  if (scale) leave(dsc, part + 2L * p.dim);
}

// Sums of partial rows, [rows][outputs][dim], in 64 strands of every 64th that
// are then added in order; 32 columns a workgroup.  512 rows of 3 x 4096: 7 us (25
// MB, from the last-level cache); bound by the few workgroups that so few columns
// make, and by the launch.
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

// Lanes per row and vectors per lane by the row's length; from 2049 values on as
// many waves as its vectors need.  The gradient holds its registers for two
// (two vectors) or three (one) waves a SIMD.  It in bf16, 2^26 values, us: rows of
// 2304 370 in two, 522 in one, 3000 306 and 447, 4096 211 and 246, 5120 269 and
// 237, 6144 248 and 225 (a few waves of two vectors leave SIMDs idle).  In fp32,
// 2^25 values: 246 and 341, 228 and 311, 217 and 209, 214 and 212, 216 and 216:
// the same choice.  The forward's differ less, and both types share the plan: bf16
// 137 and 155, 128 and 144, 117 and 113, 116 and 120, 116 and 116, fp32 157 and
// 129, 146 and 124, 133 and 120, 149 and 136, 142 and 130.  Two vectors within the
// registers of three waves a SIMD spill: 4096 336, where these took 173 (x for the
// gate, h for d_res).
static bool block_norm_single(int dim) { return dim <= 2048 || (dim > 4096 && dim <= 6144); }
int block_norm_threads(int dim) { return dim <= 2048 ? 256 : block_norm_single(dim) ? (dim + 511) / 512 * 64 : (dim + 1023) / 1024 * 64; }
#define BLOCK_NORM_DISPATCH(CALL)              \
  if (p.dim <= 128) { CALL(16, 1); }           \
  else if (p.dim <= 256) { CALL(32, 1); }      \
  else if (p.dim <= 512) { CALL(64, 1); }      \
  else if (p.dim <= 1024) { CALL(128, 1); }    \
  else if (p.dim <= 2048) { CALL(256, 1); }    \
  else if (p.dim <= 4096) { CALL(512, 2); }    \
  else if (p.dim <= 6144) { CALL(768, 1); }    \
  else if (p.dim <= 8192) { CALL(512, 2); }    \
  else { CALL(1024, 2); }

template <typename T>
static hipError_t block_norm_fwd(const BlockNormParams& p, hipStream_t st) {
  timing_before("block_norm_fwd", st);
#define CALL(TPR, NV)                                                                                          \
  constexpr int NT = TPR < 256 ? 256 : TPR;                                                                    \
  hipLaunchKernelGGL((k_block_norm_fwd<T, TPR, NV>), dim3((unsigned)((p.rows + NT / TPR - 1) / (NT / TPR))),   \
                     dim3(block_norm_threads(p.dim)), 0, st, p)
  BLOCK_NORM_DISPATCH(CALL);
#undef CALL
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_block_norm_fwd(DType dt, const BlockNormParams& p, hipStream_t st) {
  return dt == DType::BF16 ? block_norm_fwd<bf16>(p, st) : block_norm_fwd<float>(p, st);
}

int block_norm_rows_per_block(int dim) { return dim <= 128 ? 16 : dim <= 256 ? 8 : dim <= 512 ? 4 : dim <= 1024 ? 2 : 1; }
int block_norm_bwd_blocks(long rows, int dim) {
  const int resident = (dim > 2048 && block_norm_single(dim) ? 768 : 512) / block_norm_threads(dim);   // workgroups resident on a compute unit
  const long want = (resident < 1 ? 1 : resident) * kComputeUnits;
  const long most = (rows + block_norm_rows_per_block(dim) - 1) / block_norm_rows_per_block(dim);
  return (int)(most < want ? most : want);
}
template <typename T>
static hipError_t block_norm_bwd(const BlockNormParams& p, hipStream_t st) {
  if (p.blocks > 0) {
    timing_before("block_norm_bwd", st);
#define CALL(TPR, NV) \
  hipLaunchKernelGGL((k_block_norm_bwd<T, TPR, NV>), dim3((unsigned)p.blocks), dim3(block_norm_threads(p.dim)), 0, st, p)
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
