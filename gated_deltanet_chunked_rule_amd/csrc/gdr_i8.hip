// gdr_i8.hip -- rows quantised to 8-bit integers, and the product of such rows
// with a weight that holds one scale for each output channel.
//
//   scale = max(max |x|, 2^-100) / 127,  q = round(x / scale)      per row
//   y[m, n] = (sum over k of q[m, k] w[n, k]) xs[m] ws[n] + bias[n]
//
// The sums are exact (int32; K < 2^17 keeps 127 * 127 K, and 128 * 128 K, below
// 2^31); the three fp32 operations behind them round.  Both operands' rows run
// along k, so that a fragment of V_MFMA_I32_16X16X64_I8 is 16 consecutive bytes
// of a row: lane l holds row l % 16, k = 16 (l / 16) + j of each 64.  (Which k
// a lane holds does not matter as long as both operands agree.)  The weight is
// the first operand: a lane then holds four consecutive n of one m.
#include "gdr_layer.h"

namespace gdr {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_u1 __attribute__((ext_vector_type(2), aligned(1)));

constexpr float kRowTiny = 0x1p-100f;   // an all-zero row gets the scale kRowTiny / 127

__device__ __forceinline__ float max_bits(float a, float b) {   // of magnitudes; a NaN is above everything
  return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)));
}

// TPR lanes hold a row (NV vectors of 8 values each), as the norms do.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_quant_rows(QuantParams p) {
  constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
  __shared__ float red[NT / 64];
  const int t = threadIdx.x & (TPR - 1);
  const long row = (long)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < p.rows;   // rows behind the last read row 0 and write nothing
  const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.x_stride;
  typename VecIO<T, 8>::raw raw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * TPR + t) * 8;
    raw[v] = vec_raw<T, 8>(x + d, max(0, p.dim - d));
  }
  float m = kRowTiny;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float f[8];
    VecIO<T, 8>::up(raw[v], f);
#pragma unroll
    for (int c = 0; c < 8; ++c) m = max_bits(m, fabsf(f[c]));
  }
  m = max_bits(m, dpp_f<0xB1>(m));
  m = max_bits(m, dpp_f<0x4E>(m));
  m = max_bits(m, dpp_f<0x141>(m));
  m = max_bits(m, dpp_f<0x140>(m));
#pragma unroll
  for (int s = 16; s < (TPR < 64 ? TPR : 64); s <<= 1) m = max_bits(m, __shfl_xor(m, s));
  if constexpr (TPR > 64) {
    if (lane_id() == 0) red[threadIdx.x >> 6] = m;
    lds_barrier();
    const int first = (threadIdx.x / TPR) * (TPR / 64);
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) m = max_bits(m, red[first + i]);
  }
  if (!live) return;
  // a row with an infinity or a NaN is NaN: its scale is, and its values are zero
  const bool sound = __builtin_bit_cast(uint32_t, m) < 0x7f800000u;
  const float scale = sound ? m / 127.f : __builtin_nanf("");
  if (t == 0) p.scales[row] = scale;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int d = (v * TPR + t) * 8;
    if (d >= p.pad) continue;
    float f[8];
    VecIO<T, 8>::up(raw[v], f);
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      // the quotient is the correctly rounded one (an IEEE division), so that
      // the rounded value is what its fp32 quotient rounds to, ties to even
      const int q = sound ? (int)rintf(f[c] / scale) : 0;
      o[c / 4] |= (uint32_t)(q & 255) << (8 * (c % 4));
    }
    int8_t* out = p.q + row * p.q_stride + d;
    const int nd = p.pad - d;
    if (nd >= 8) *reinterpret_cast<u32x2_u1*>(out) = u32x2_u1{o[0], o[1]};
    else
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < nd) out[c] = (int8_t)(o[c / 4] >> (8 * (c % 4)));
  }
}

// ---------------------------------------------------------------- product --
// Bytes of a descriptor over `rows` rows: up to the 16-byte piece that holds
// the last row's last value.
__device__ __forceinline__ long i8_range(int rows, long stride, int K) { return rows <= 0 ? 0 : (rows - 1) * stride + (K + 15) / 16 * 16; }
// The bytes of a fragment that lie before K (k: of its first byte).
__device__ __forceinline__ i32x4 i8_head(i32x4 f, int k, int K) {
  const int n = K - k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = n - 4 * i;
    f[i] = b >= 4 ? f[i] : b <= 0 ? 0 : f[i] & (int)((1u << (8 * b)) - 1u);
  }
  return f;
}
__device__ __forceinline__ i32x4 i8_mma(i32x4 a, i32x4 b, i32x4 c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }

// y of N consecutive n from n0 on of row m
template <typename T, int N>
__device__ __forceinline__ void i8_leave(const I8Params& p, int m, int n0, const int (&acc)[N], float xs, const float (&ws)[N], const float (&bias)[N]) {
  const int nd = min(N, p.N - n0);
  if (m >= p.M || nd <= 0) return;
  float f[N];
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = (float)acc[e] * xs * ws[e] + bias[e];
  T* y = static_cast<T*>(p.y) + (long)m * p.N + n0;
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    float g[4] = {f[e], f[e + 1], f[e + 2], f[e + 3]};
    if (nd > e) vec_store<T, 4>(y + e, nd - e, g);
  }
}

// Few rows of x: the weight is streamed once from memory into registers, and
// nothing is staged.  A workgroup takes 16 NT rows of the weight and 16 MT of
// x; its waves share k in pieces of 64 U bytes and add up in LDS.
template <typename T, int MT, int NT, int U, int NW>
__global__ __launch_bounds__(64 * NW) void k_i8_few(I8Params p) {
  constexpr int TILES = MT * NT;
  __shared__ i32x4 part[NW][TILES][64];
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const rsrc_t rw = make_rsrc_u(p.w + (long)n0 * p.w_stride, i8_range(min(16 * NT, p.N - n0), p.w_stride, p.K));
  const rsrc_t rx = make_rsrc_u(p.x + (long)m0 * p.x_stride, i8_range(min(16 * MT, p.M - m0), p.x_stride, p.K));
  const uint32_t ow = (uint32_t)(c * p.w_stride) + 16 * g, ox = (uint32_t)(c * p.x_stride) + 16 * g;
  const uint32_t sw = (uint32_t)(16 * p.w_stride), sx = (uint32_t)(16 * p.x_stride);
  i32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  for (int k0 = w * 64 * U; k0 < p.K; k0 += NW * 64 * U) {
    i32x4 fw[U][NT], fx[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < NT; ++i) fw[u][i] = __builtin_bit_cast(i32x4, buf_load16(rw, ow + i * sw + k0 + 64 * u));
#pragma unroll
      for (int j = 0; j < MT; ++j) fx[u][j] = __builtin_bit_cast(i32x4, buf_load16(rx, ox + j * sx + k0 + 64 * u));
    }
    if (k0 + 64 * U > p.K) {   // wave-uniform
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NT; ++i) fw[u][i] = i8_head(fw[u][i], k0 + 64 * u + 16 * g, p.K);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = i8_mma(fw[u][i], fx[u][j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[w][i * MT + j][l] = acc[i][j];
  __syncthreads();
  for (int tile = w; tile < TILES; tile += NW) {
    i32x4 s = part[0][tile][l];
#pragma unroll
    for (int u = 1; u < NW; ++u) s += part[u][tile][l];
    const int i = tile / MT, j = tile - i * MT, m = m0 + 16 * j + c, n = n0 + 16 * i + 4 * g;
    if (m >= p.M || n >= p.N) continue;
    float ws[4], bias[4] = {0.f, 0.f, 0.f, 0.f};
    vec_load<float, 4>(p.ws + n, p.N - n, ws);
    if (p.bias) vec_load<float, 4>(p.bias + n, p.N - n, bias);
    const int a[4] = {s[0], s[1], s[2], s[3]};
    i8_leave<T, 4>(p, m, n, a, p.xs[m], ws, bias);
  }
}

// Many rows: BN rows of the weight by BM rows of x a workgroup, in steps of 128
// bytes of k that direct copies bring into two LDS buffers.  Row r's 16-byte
// piece c stands at c ^ (r % 8).  Row r of a wave's 16 NT weight rows in LDS is
// n = 4 NT ((r % 16) / 4) + 4 (r / 16) + r % 4, so that a lane's values of one
// m over its NT tiles are 4 NT consecutive n.
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_i8_many(I8Params p) {
  constexpr int NW = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16, KS = 128;
  constexpr int CW = BN / 8 / NW, CX = BM / 8 / NW;   // 1 KB copies a wave
  static_assert(CW * 8 * NW == BN && CX * 8 * NW == BM, "whole copies for each wave");
  __shared__ __align__(1024) int8_t lds[2][(BM + BN) * KS];
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int id = xcd_remap(blockIdx.x, p.tiles);
  if (id >= p.tiles) return;
  // groups of p.group rows of tiles, column by column, so that the tiles that
  // run at once on an XCD share rows of both operands
  const int per = p.group * p.tn, grp = id / per, in = id - grp * per;
  const int gm = min(p.group, p.tm - grp * p.group);
  const int m0 = (grp * p.group + in % gm) * BM, n0 = in / gm * BN;
  const i32x4v rw = rsrc_words(p.w + (long)n0 * p.w_stride, i8_range(min(BN, p.N - n0), p.w_stride, p.K));
  const i32x4v rx = rsrc_words(p.x + (long)m0 * p.x_stride, i8_range(min(BM, p.M - m0), p.x_stride, p.K));
  uint32_t ow[CW], ox[CX];
#pragma unroll
  for (int j = 0; j < CW; ++j) {
    const int r = (w * CW + j) * 8 + (l >> 3), in_wave = r % (16 * NT);
    const int n = r - in_wave + 4 * NT * (in_wave % 16 / 4) + 4 * (in_wave / 16) + in_wave % 4;
    ow[j] = (uint32_t)(n * p.w_stride) + 16 * ((l & 7) ^ (r & 7));
  }
#pragma unroll
  for (int j = 0; j < CX; ++j) {
    const int r = (w * CX + j) * 8 + (l >> 3);
    ox[j] = (uint32_t)(r * p.x_stride) + 16 * ((l & 7) ^ (r & 7));
  }
  auto copy = [&](int k0, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < CW; ++j) lds_copy16(rw, ow[j] + k0, lds_addr(&lds[buf][(w * CW + j) * 8 * KS]));
#pragma unroll
    for (int j = 0; j < CX; ++j) lds_copy16(rx, ox[j] + k0, lds_addr(&lds[buf][(BN + (w * CX + j) * 8) * KS]));
  };
  const int wm = w % WM, wn = w / WM;
  const int aw = (wn * 16 * NT + c) * KS, ax = (BN + wm * 16 * MT + c) * KS;
  i32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto products = [&](int k0, int buf, auto tail) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < KS / 64; ++kk) {
      const int at = 16 * ((4 * kk + g) ^ (c & 7));
      i32x4 fw[NT], fx[MT];
#pragma unroll
      for (int i = 0; i < NT; ++i) fw[i] = *reinterpret_cast<const i32x4*>(&lds[buf][aw + i * 16 * KS + at]);
#pragma unroll
      for (int j = 0; j < MT; ++j) fx[j] = *reinterpret_cast<const i32x4*>(&lds[buf][ax + j * 16 * KS + at]);
      if constexpr (decltype(tail)::value) {
#pragma unroll
        for (int i = 0; i < NT; ++i) fw[i] = i8_head(fw[i], k0 + 64 * kk + 16 * g, p.K);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = i8_mma(fw[i], fx[j], acc[i][j]);
    }
  };
  copy(0, 0);
  int buf = 0, k0 = 0;
  for (; k0 + KS < p.K; k0 += KS, buf ^= 1) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // this wave's copies have landed
    lds_barrier();                        // and everybody's; the other buffer is free
    copy(k0 + KS, buf ^ 1);
    products(k0, buf, std::false_type{});
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
  lds_barrier();
  if (k0 + KS > p.K) products(k0, buf, std::true_type{});
  else products(k0, buf, std::false_type{});
  const int n = n0 + wn * 16 * NT + 4 * NT * g;
  float ws[4 * NT], bias[4 * NT];
#pragma unroll
  for (int e = 0; e < 4 * NT; e += 4) {
    float f[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
    if (n + e < p.N) {
      vec_load<float, 4>(p.ws + n + e, p.N - n - e, f);
      if (p.bias) vec_load<float, 4>(p.bias + n + e, p.N - n - e, b);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ws[e + i] = f[i];
      bias[e + i] = b[i];
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = m0 + wm * 16 * MT + 16 * j + c;
    int a[4 * NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[4 * i + e] = acc[i][j][e];
    i8_leave<T, 4 * NT>(p, m, n, a, m < p.M ? p.xs[m] : 0.f, ws, bias);
  }
}

#define QUANT_DISPATCH(CALL)                   \
  if (p.pad <= 128) { CALL(16, 1); }           \
  else if (p.pad <= 256) { CALL(32, 1); }      \
  else if (p.pad <= 512) { CALL(64, 1); }      \
  else if (p.pad <= 1024) { CALL(128, 1); }    \
  else if (p.pad <= 2048) { CALL(256, 1); }    \
  else if (p.pad <= 4096) { CALL(256, 2); }    \
  else if (p.pad <= 8192) { CALL(512, 2); }    \
  else if (p.pad <= 16384) { CALL(1024, 2); }  \
  else { CALL(1024, 4); }

template <typename T>
static hipError_t quant_rows(const QuantParams& p, hipStream_t st) {
  timing_before("quantize_rows", st);
#define CALL(TPR, NV)                                                                                      \
  constexpr int NT = TPR < 256 ? 256 : TPR;                                                                \
  hipLaunchKernelGGL((k_quant_rows<T, TPR, NV>), dim3((unsigned)((p.rows + NT / TPR - 1) / (NT / TPR))),   \
                     dim3(NT), 0, st, p)
  QUANT_DISPATCH(CALL);
#undef CALL
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_quant_rows(DType dt, const QuantParams& p, hipStream_t st) {
  return dt == DType::BF16 ? quant_rows<bf16>(p, st) : quant_rows<float>(p, st);
}

template <typename T, int MT, int NT, int U>
static void i8_few(const I8Params& p, hipStream_t st) {
  hipLaunchKernelGGL((k_i8_few<T, MT, NT, U, 8>), dim3((p.N + 16 * NT - 1) / (16 * NT), (p.M + 16 * MT - 1) / (16 * MT)), dim3(512), 0, st, p);
}
template <typename T, int BM, int BN, int WM, int WN>
static void i8_many(I8Params p, hipStream_t st) {
  p.tm = (p.M + BM - 1) / BM;
  p.tn = (p.N + BN - 1) / BN;
  p.tiles = p.tm * p.tn;
  p.group = 4;
  hipLaunchKernelGGL((k_i8_many<T, BM, BN, WM, WN>), dim3((p.tiles + 7) / 8 * 8), dim3(64 * WM * WN), 0, st, p);
}
template <typename T>
static hipError_t i8_matmul(const I8Params& p, hipStream_t st) {
  timing_before("matmul_i8", st);
  auto tiles = [&](long bm, long bn) { return ((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn); };
  if (p.M <= 16) i8_few<T, 1, 1, 4>(p, st);
  else if (p.M <= 32) i8_few<T, 2, 1, 4>(p, st);
  else if (p.M <= 64) i8_few<T, 4, 1, 2>(p, st);
  else if (p.M <= 128 || tiles(128, 128) < kComputeUnits) i8_few<T, 8, 2, 1>(p, st);
  else if (tiles(256, 256) < kComputeUnits) i8_many<T, 128, 128, 2, 2>(p, st);
  else i8_many<T, 256, 256, 2, 4>(p, st);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_i8_matmul(DType dt, const I8Params& p, hipStream_t st) {
  return dt == DType::BF16 ? i8_matmul<bf16>(p, st) : i8_matmul<float>(p, st);
}

}  // namespace gdr
