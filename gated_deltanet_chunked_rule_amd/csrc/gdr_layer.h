// gdr_layer.h -- parameter blocks, launchers and device helpers of the
// operators around the rule (convolution, single-token steps, state space
// scan, linear recurrence, norms, integer products); internal to libgdr.
#pragma once

#include "../../include/gdr.h"
#include "gdr_device.h"

namespace gdr {

// Records the message of a refused call; returns `s` (gdr_api.cpp).
gdr_status set_error(gdr_status s, const char* msg) noexcept;

constexpr int kComputeUnits = 256;

// Token ranges of the sequences, read on the device.  Offsets are clamped to
// [0, Ttot]: whatever cu holds, ranges stay inside the tensors.
struct SeqRanges {
  const int32_t* cu;   // nullable: N rows of T tokens
  int N, T;
  int Ttot;
};

struct ConvParams {
  SeqRanges s;
  const void *x, *weight, *bias, *h0;
  const void *dy, *dht;      // backward
  void *y, *ht;
  void *dx, *dw, *db, *dh0;  // backward
  float* part;               // backward: [tiles][W + 1][D] fp32 partial sums of dw and db
  void* state;               // step
  const int32_t* slots;
  int num_slots;
  long x_stride;
  int D, act;
  int tile, tiles;           // tokens per tile, tiles over the token axis
};

struct StepParams {          // rule: q, k, v, g, beta; scan: q = C, k = B, v = x, dt, A, bias, skip
  const void *q, *k, *v, *dt;
  const float *g, *beta, *A, *bias, *skip;
  float* state;
  const int32_t* slots;
  void* o;
  long q_stride, k_stride, v_stride, dt_stride;
  int rows, Hq, Hv, K, V, num_slots, softplus;
  float scale;
};

struct SsmParams {
  SeqRanges s;
  const void *x, *dt, *B, *C;
  const float *A, *D, *bias, *h0;
  void* y;
  float* ht;
  float* seg_state;          // [segs - 1][H][N][P]: transition offsets, then the states at the segment ends
  float* seg_decay;          // [segs - 1][H]: log-decay over the segment, -inf where its end does not depend on its start
  long x_stride, dt_stride, b_stride, c_stride;
  int H, G, P, N, softplus;
  int seg, segs;             // tokens per segment (a multiple of the chunk), segments
  int wgs;                   // workgroups per segment
};

struct NormParams {
  long rows;
  int inner, dim;
  float eps, inv_dim;            // inv_dim = 1 / dim
  const void *x, *residual, *gate, *weight;
  long xo, xi, ro, ri, go, gi;   // outer and inner strides of x, residual, gate
  void *y, *h_out;
  float* scales;
  const void *dy, *dres;         // backward
  void *dh, *dgate, *dw;
  float* part;                   // backward: [blocks][dim] partial sums of dw
  int blocks;
};

struct LinParams {               // linear scan; the step: Ttot rows, ht the pool of states
  SeqRanges s;
  const void *x, *r, *i, *dy;
  const float *A, *h0, *dht;
  void *y, *dx, *dr, *di;
  float *ht, *dh0, *dA;
  float *P, *S, *Q, *part;       // [tiles][D] each
  uint64_t* words;               // [tiles][D]: (P, S) of the tiles that are there, in one pass
  uint32_t* ends;                // [groups][D]: states at the ends of groups of tiles
  int* ticket;
  const int32_t* slots;
  long x_stride, r_stride, i_stride;
  int D, tiles, cols, num_slots; // tiles of tokens, columns of channels
};

struct BlockNormParams {
  long rows;
  int dim, blocks;
  float eps, inv_dim;
  const void *x, *residual, *gate, *post, *pre, *scale;
  const void *h, *dy, *dres;     // backward; h has residual's stride
  long x_stride, r_stride, g_stride;
  void *y, *h_out;
  void *dx, *dh, *dgate, *dpost, *dpre, *dscale;
  float* part;                   // [blocks][2 or 3][dim]: sums for dpost, dpre, dscale
};

struct RowsSum {
  const float* part;             // [rows][outputs][dim]
  int rows, dim;
  void* out[3];
};

struct QuantParams {
  long rows;
  int dim, pad;                  // values of a row, and with the zeros behind them
  const void* x;
  int8_t* q;
  float* scales;
  long x_stride, q_stride;
};

struct I8Params {
  const int8_t *x, *w;           // [M][K], [N][K]
  const float *xs, *ws, *bias;
  void* y;
  long x_stride, w_stride;
  int M, N, K;
  int tm, tn, tiles;             // tiles of x and the weight
};

hipError_t launch_conv_fwd(DType dt, int W, const ConvParams& p, hipStream_t st);
hipError_t launch_conv_bwd(DType dt, int W, const ConvParams& p, hipStream_t st);
hipError_t launch_conv_step(DType dt, int W, int rows, const ConvParams& p, hipStream_t st);
int conv_bwd_tile(int tokens, int D);       // tokens per tile of the backward
hipError_t launch_rule_step(DType dt, const StepParams& p, hipStream_t st);
hipError_t launch_ssm_step(DType dt, const StepParams& p, hipStream_t st);
void ssm_plan(DType dt, SsmParams& p);      // segments and workgroups
hipError_t launch_ssm_scan(DType dt, const SsmParams& p, hipStream_t st);
hipError_t launch_norm_fwd(DType dt, bool quant, const NormParams& p, hipStream_t st);
hipError_t launch_norm_bwd(DType dt, const NormParams& p, hipStream_t st);
int norm_bwd_blocks(long rows, int dim);
int lin_tiles(DType dt, int tokens);        // tiles of the token axis
int lin_bwd_tiles(int tokens);
int lin_cols(int D);
size_t lin_fwd_bytes(DType dt, int tokens, int D);
hipError_t launch_lin_fwd(DType dt, const LinParams& p, void* workspace, hipStream_t st);
hipError_t launch_lin_bwd(DType dt, const LinParams& p, hipStream_t st);
hipError_t launch_lin_step(DType dt, const LinParams& p, hipStream_t st);
hipError_t launch_block_norm_fwd(DType dt, const BlockNormParams& p, hipStream_t st);
hipError_t launch_block_norm_bwd(DType dt, const BlockNormParams& p, hipStream_t st);
int block_norm_bwd_blocks(long rows, int dim);
int block_norm_threads(int dim);            // of a workgroup
int block_norm_rows_per_block(int dim);
hipError_t launch_quant_rows(DType dt, const QuantParams& p, hipStream_t st);
hipError_t launch_i8_matmul(DType dt, const I8Params& p, hipStream_t st);
hipError_t launch_rows_sum(DType dt, int outputs, const RowsSum& p, hipStream_t st);   // dt: of the outputs

// ------------------------------------------------------------- device part --
// VEC consecutive elements that need the alignment of one element only:
// global accesses of 8 and 16 bytes work at any element address on gfx950, so
// odd row lengths take the same path.
typedef uint32_t u32x4_u2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_u4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T, int VEC> struct VecIO;
template <> struct VecIO<bf16, 8> {
  typedef u32x4_u2 raw;
  static __device__ __forceinline__ void up(raw r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = r[i];   // bit_cast of a vector element lvalue drops the index
      f[2 * i] = __builtin_bit_cast(float, u << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ raw down(const float (&f)[8]) {
    raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x2 b = {static_cast<bf16>(f[2 * i]), static_cast<bf16>(f[2 * i + 1])};
      r[i] = __builtin_bit_cast(uint32_t, b);
    }
    return r;
  }
};
template <> struct VecIO<bf16, 4> {
  typedef u32x2_u2 raw;
  static __device__ __forceinline__ void up(raw r, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = r[i];
      f[2 * i] = __builtin_bit_cast(float, u << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ raw down(const float (&f)[4]) {
    raw r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bf16x2 b = {static_cast<bf16>(f[2 * i]), static_cast<bf16>(f[2 * i + 1])};
      r[i] = __builtin_bit_cast(uint32_t, b);
    }
    return r;
  }
};
template <> struct VecIO<float, 4> {
  typedef u32x4_u4 raw;
  static __device__ __forceinline__ void up(raw r, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = r[i];
      f[i] = __builtin_bit_cast(float, u);
    }
  }
  static __device__ __forceinline__ raw down(const float (&f)[4]) {
    raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_bit_cast(uint32_t, f[i]);
    return r;
  }
};
typedef uint32_t u32x2_u4 __attribute__((ext_vector_type(2), aligned(4)));
template <> struct VecIO<float, 2> {
  typedef u32x2_u4 raw;
  static __device__ __forceinline__ void up(raw r, float (&f)[2]) {
    const uint32_t u = r[0], v = r[1];
    f[0] = __builtin_bit_cast(float, u);
    f[1] = __builtin_bit_cast(float, v);
  }
  static __device__ __forceinline__ raw down(const float (&f)[2]) {
    return raw{__builtin_bit_cast(uint32_t, f[0]), __builtin_bit_cast(uint32_t, f[1])};
  }
};
typedef uint32_t u32x1_u2 __attribute__((ext_vector_type(1), aligned(2)));
template <> struct VecIO<bf16, 2> {
  typedef u32x1_u2 raw;
  static __device__ __forceinline__ void up(raw r, float (&f)[2]) {
    const uint32_t u = r[0];
    f[0] = __builtin_bit_cast(float, u << 16);
    f[1] = __builtin_bit_cast(float, u & 0xffff0000u);
  }
  static __device__ __forceinline__ raw down(const float (&f)[2]) {
    const bf16x2 b = {static_cast<bf16>(f[0]), static_cast<bf16>(f[1])};
    return raw{__builtin_bit_cast(uint32_t, b)};
  }
};
struct raw_f8 { u32x4_u4 a, b; };
template <> struct VecIO<float, 8> {
  typedef raw_f8 raw;
  static __device__ __forceinline__ void up(raw r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = r.a[i], v = r.b[i];
      f[i] = __builtin_bit_cast(float, u);
      f[4 + i] = __builtin_bit_cast(float, v);
    }
  }
  static __device__ __forceinline__ raw down(const float (&f)[8]) {
    raw r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = __builtin_bit_cast(uint32_t, f[i]);
      r.b[i] = __builtin_bit_cast(uint32_t, f[4 + i]);
    }
    return r;
  }
};

// The first n <= VEC elements at p (the others are zero); the whole vector in
// one access where n == VEC.
template <typename T, int VEC>
__device__ __forceinline__ typename VecIO<T, VEC>::raw vec_raw(const T* p, int n) {
  if (n >= VEC) return *reinterpret_cast<const typename VecIO<T, VEC>::raw*>(p);
  float f[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
  return VecIO<T, VEC>::down(f);
}
template <typename T, int VEC>
__device__ __forceinline__ void vec_load(const T* p, int n, float (&f)[VEC]) {
  VecIO<T, VEC>::up(vec_raw<T, VEC>(p, n), f);
}
template <typename T, int VEC>
__device__ __forceinline__ void vec_store(T* p, int n, const float (&f)[VEC]) {
  if (n >= VEC) {
    *reinterpret_cast<typename VecIO<T, VEC>::raw*>(p) = VecIO<T, VEC>::down(f);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) p[i] = from_f<T>(f[i]);
  }
}

__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
// 1 / (1 + e^-x), with the hardware's exp2 and reciprocal (one ulp each)
__device__ __forceinline__ float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.f + exp_f(-x)); }
// 1 / sqrt(v) for v >= 0, an ulp.  The instruction takes what lies below the normal
// numbers as zero, so small v are scaled by 2^64 and the root's 2^32 taken back.
__device__ __forceinline__ float rsqrt_f(float v) {
  const bool small = v < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v);
  return small ? r * 0x1p32f : r;
}
// log(1 + e^x); above 20 it equals x in fp32.  With u = e^x and w = 1 + u
// rounded, log(w) u / (w - 1) takes back the rounding of w (the correction of
// Goldberg's "What every computer scientist should know about floating-point
// arithmetic", theorem 4), so that small steps keep their relative accuracy.
__device__ __forceinline__ float softplus_f(float x) {
  const float u = exp_f(x), w = 1.f + u, d = w - 1.f;
  const float v = d == 0.f ? u : __builtin_amdgcn_logf(w) * 0.6931471805599453f * (u * __builtin_amdgcn_rcpf(d));
  return x > 20.f ? x : v;
}

// Tables of offsets: staged in LDS below this many sequences.
constexpr int kCuLds = 1024;
struct SeqFinder {
  const int32_t* cu;   // global, or the staged copy
  int N, T, Ttot;
  bool packed;
  __host__ __device__ __forceinline__ int at(int n) const {
    if (!packed) return n * T;
    const int v = cu[n] < 0 ? 0 : cu[n];
    return v < Ttot ? v : Ttot;
  }
  // The run of tokens from t on (t < Ttot) that share a sequence: [start, end)
  // with start <= t < end, returns n; outside every sequence returns -1 and
  // end is the first token to look at again.  Where offsets decrease, start
  // may lie before the run that ended at t: 0 <= start <= t < end <= Ttot and
  // 0 <= n < N are all that holds for any table.
  __host__ __device__ __forceinline__ int find(int t, int& start, int& end) const {
    if (!packed) {
      const int n = t / T;
      start = n * T;
      end = start + T;
      return n;
    }
    start = t;
    if (at(0) > t) {
      end = at(0);
      return -1;
    }
    int lo = 0, hi = N - 1;
    while (lo < hi) {
      const int mid = lo + ((hi - lo + 1) >> 1);   // their sum may leave an int
      if (at(mid) <= t) lo = mid; else hi = mid - 1;
    }
    const int e = at(lo + 1);
    if (e <= t) {   // behind the last sequence (or offsets that decrease)
      end = lo == N - 1 ? Ttot : t + 1;
      return -1;
    }
    start = at(lo);
    end = e;
    return lo;
  }
  // Whether the run found at t goes on from a piece [.., piece) of the token
  // axis that another workgroup walked: its state is then that piece's.  Only
  // at the piece's own first token, and never at token 0, whatever the table.
  static __host__ __device__ __forceinline__ bool goes_on(int t, int piece, int start) { return t == piece && start < t; }
};
// f(n) of the sequences without a token among first, first + step, ...  (Their
// numbers plus a step may leave an int.)
template <typename F>
__host__ __device__ __forceinline__ void empty_sequences(const SeqFinder& sf, long first, long step, F f) {
  if (!sf.packed && sf.T > 0) return;
  for (long n = first; n < sf.N; n += step)
    if (sf.at((int)n + 1) <= sf.at((int)n)) f(n);
}
// What happens at the `count` (below 32) tokens from t0 on, as bits: first: the
// token starts a run that does not go on from the tokens before t0; last: it
// ends its sequence; gap: it belongs to none, or lies behind the last token.
// seq[k] is the sequence of a token that starts or ends one, in [0, N)
// whatever the table (where offsets decrease, a run's tokens may find
// different ones, or none: such a token ends nothing).
struct TokenRuns { uint32_t first, last, gap; };
__host__ __device__ __forceinline__ TokenRuns token_runs(const SeqFinder& sf, int t0, int count, int* seq) {
  TokenRuns m = {0, 0, 0};
  const int t1 = t0 + count < sf.Ttot ? t0 + count : sf.Ttot;
  for (int t = t0; t < t1;) {
    int start, end;
    const int n = sf.find(t, start, end), stop = end < t1 ? end : t1;
    if (n < 0) {
      m.gap |= ((1u << (stop - t)) - 1u) << (t - t0);
    } else {
      int s, e;
      const int ends = end > t1 ? -1 : end == t + 1 ? n : sf.find(end - 1, s, e);
      if (!SeqFinder::goes_on(t, t0, start)) {
        m.first |= 1u << (t - t0);
        seq[t - t0] = n;
      }
      if (ends >= 0) {
        m.last |= 1u << (end - 1 - t0);
        seq[end - 1 - t0] = ends;
      }
    }
    t = stop;
  }
  const int live = t1 > t0 ? t1 - t0 : 0;
  if (live < count) m.gap |= ~0u << live;
  return m;
}
// Linear recurrence: a column of kLinCh channels is a wave's, kLinVec a lane, from
// lin_base on.  The last column's last lanes are moved back onto the last
// channels, which they share with the lane before: they compute and store the
// same values, and no access needs a mask.  Fewer than kLinVec channels are
// held by every lane, in its first places.
constexpr int kLinVec = 2, kLinCh = 64 * kLinVec;
__host__ __device__ __forceinline__ int lin_base(int first, int D) {
  const int last = D < kLinVec ? 0 : D - kLinVec;
  return first < last ? first : last;
}
// Value c < kLinCh of a column is that of lane c / kLinVec in its place
// lin_place, and of the channel lin_channel, which is there for every c.
__host__ __device__ __forceinline__ int lin_place(int c, int D) {
  const int k = c % kLinVec;
  return k < D ? k : D - 1;
}
__host__ __device__ __forceinline__ int lin_channel(int col, int c, int D) {
  return lin_base(col * kLinCh + c / kLinVec * kLinVec, D) + lin_place(c, D);
}
// Every thread of the workgroup calls this (barrier inside).
template <int STAGE = kCuLds>
__device__ __forceinline__ SeqFinder seq_finder(const SeqRanges& s, int32_t* lds) {
  SeqFinder f;
  f.cu = s.cu;
  f.N = s.N;
  f.T = s.T;
  f.Ttot = s.Ttot;
  f.packed = s.cu != nullptr;
  if (s.cu && s.N < STAGE) {
    for (int i = threadIdx.x; i <= s.N; i += blockDim.x) lds[i] = s.cu[i];
    __syncthreads();
    f.cu = lds;
  }
  return f;
}

// Slot of a step's row, or -1 for padding: outside the pool, or named by an
// earlier row.  The lanes of a wave share one row.
__device__ __forceinline__ int step_slot(const int32_t* slots, int row, int num_slots) {
  if (!slots) return row;
  const int s = __builtin_amdgcn_readfirstlane(slots[row]);
  bool dup = false;
  for (int j = lane_id(); j < row; j += 64) dup |= slots[j] == s;
  if (__builtin_amdgcn_ballot_w64(dup) != 0 || s < 0 || s >= num_slots) return -1;
  return s;
}

}  // namespace gdr
