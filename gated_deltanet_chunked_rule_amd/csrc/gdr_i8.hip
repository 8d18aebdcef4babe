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

// TPR lanes hold a row (NV vectors of 8 values each), as the norms do: the row is
// read once.  Bound by memory: 8192 x 4096 in bf16 24 us (4.2 TB/s), 16384 x 4096
// 36 (5.7); 1 row 6.9 a call.
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

// The waves' sums of a workgroup's tiles ([wave][tile][lane], tile = MT i + j),
// added and left in y.
template <typename T, int MT, int TILES, int NW>
__device__ __forceinline__ void i8_finish(const I8Params& p, const i32x4* part, int m0, int n0, int w) {
  const int l = lane_id(), c = l & 15, g = l >> 4;
  for (int tile = w; tile < TILES; tile += NW) {
    i32x4 s = part[tile * 64 + l];
#pragma unroll
    for (int u = 1; u < NW; ++u) s += part[(u * TILES + tile) * 64 + l];
    const int i = tile / MT, j = tile - i * MT, m = m0 + 16 * j + c, n = n0 + 16 * i + 4 * g;
    if (m >= p.M || n >= p.N) continue;
    float ws[4], bias[4] = {0.f, 0.f, 0.f, 0.f};
    vec_load<float, 4>(p.ws + n, p.N - n, ws);
    if (p.bias) vec_load<float, 4>(p.bias + n, p.N - n, bias);
    const float xs = p.xs[m];
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (float)s[e] * xs * ws[e] + bias[e];
    vec_store<T, 4>(static_cast<T*>(p.y) + (long)m * p.N + n, p.N - n, f);
  }
}

// The s_waitcnt that lets N of the wave's copies be under way.
template <int N>
__device__ __forceinline__ void i8_landed() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
}

// Some rows: 16 NT rows of the weight by 16 MT of x a workgroup, in steps of 256
// bytes of k of which each of the four waves multiplies 64.  Direct copies of
// whole rows bring the steps into LDS, ST - 1 ahead; nothing in LDS is read
// twice, and the waves' sums meet at the end.  Row r's 16-byte piece c stands
// at c ^ stage_swz<16>(r % 16).  4096 -> 8192, 1 row 8.9 us (bound by the weight:
// 5.1 at the rate of reads alone, and the launch), 100 rows 12.3, 256 rows 17.4.
// Operands read straight into registers took 8.8, 19.4 and 41 (a lane's 16 bytes of
// 16 rows are 64 requests); more steps ahead (9, 6 and 4 buffers for 6, 4 and 3)
// 9.2, 12.8 and 18.5.  What bounds 100 rows is not shown: the 655 KB that a compute
// unit copies are 4.3 us at 64 bytes a clock, its round takes 8; 1.08 million
// requests of 128 bytes to L2 (a quarter of them on to memory) return after 490
// clocks each, which the two steps of 40 KB ahead would cover, and waves wait to
// issue for 45 % of their time.
template <typename T, int MT, int NT, int ST>
__global__ __launch_bounds__(256) void k_i8_some(I8Params p) {
  constexpr int NW = 4, KS = 64 * NW, R = 16 * (MT + NT), C = R / 4 / NW, TILES = MT * NT;   // C: 1 KB copies a wave and step
  static_assert(C * 4 * NW == R, "whole copies for each wave");
  constexpr int STAGE = R * KS, PART = NW * TILES * 1024;
  __shared__ __align__(1024) int8_t lds[ST * STAGE > PART ? ST * STAGE : PART];
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int bn = (p.N + 16 * NT - 1) / (16 * NT), bm = blockIdx.x / bn;
  const int n0 = (blockIdx.x - bm * bn) * 16 * NT, m0 = bm * 16 * MT;
  const i32x4v rw = rsrc_words(p.w + (long)n0 * p.w_stride, i8_range(min(16 * NT, p.N - n0), p.w_stride, p.K));
  const i32x4v rx = rsrc_words(p.x + (long)m0 * p.x_stride, i8_range(min(16 * MT, p.M - m0), p.x_stride, p.K));
  // rows of the weight first; a copy's four rows are all of one operand
  uint32_t off[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int first = (j * NW + w) * 4, r = first + (l >> 4);
    off[j] = (uint32_t)(first < 16 * NT ? r * p.w_stride : (r - 16 * NT) * p.x_stride) + 16 * ((l & 15) ^ stage_swz<16>(r & 15));
  }
  const int steps = (p.K + KS - 1) / KS;
  // steps behind the last are copied from behind the descriptors' ranges: zeros
  auto copy = [&](int s, int buf) __attribute__((always_inline)) {
    const uint32_t k0 = s < steps ? (uint32_t)(s * KS) : 0x80000000u;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int first = (j * NW + w) * 4;
      lds_copy16(first < 16 * NT ? rw : rx, off[j] + k0, lds_addr(&lds[buf * STAGE + first * KS]));
    }
  };
  i32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) copy(s, s);
  const int at = c * KS + 16 * ((4 * w + g) ^ stage_swz<16>(c));
  int buf = 0;
  for (int s = 0; s < steps; ++s) {
    i8_landed<(ST - 2) * C>();   // of step s, this wave's copies
    lds_barrier();               // and everybody's; the buffer of step s - 1 is free
    copy(s + ST - 1, buf == 0 ? ST - 1 : buf - 1);
    i32x4 fw[NT], fx[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) fw[i] = *reinterpret_cast<const i32x4*>(&lds[buf * STAGE + at + i * 16 * KS]);
#pragma unroll
    for (int j = 0; j < MT; ++j) fx[j] = *reinterpret_cast<const i32x4*>(&lds[buf * STAGE + at + (NT + j) * 16 * KS]);
    if ((s + 1) * KS > p.K) {
#pragma unroll
      for (int i = 0; i < NT; ++i) fw[i] = i8_head(fw[i], s * KS + 64 * w + 16 * g, p.K);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = i8_mma(fw[i], fx[j], acc[i][j]);
    buf = buf == ST - 1 ? 0 : buf + 1;
  }
  i8_landed<0>();
  lds_barrier();   // the stages' place is free for the sums
  i32x4* part = reinterpret_cast<i32x4*>(lds);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[(w * TILES + i * MT + j) * 64 + l] = acc[i][j];
  lds_barrier();
  i8_finish<T, MT, TILES, NW>(p, part, m0, n0, w);
}

// Many rows: BN rows of the weight by BM rows of x a workgroup, in steps of 128
// bytes of k that direct copies bring into two LDS buffers.  A step is two
// products of 64 k; the operands of the next one are read into a second set of
// registers while a product runs.  Row r's 16-byte piece c stands at c ^
// stage_swz<8>(r % 16).  Row r of a wave's 16 NT weight rows in LDS is n = 4 NT
// ((r % 16) / 4) + 4 (r / 16) + r % 4, so that a lane's values of one m over its
// NT tiles are 4 NT consecutive n.
//
// 8192 x 4096 -> 8192: 223 to 251 us by the data and the run (2.2e15 to 2.5e15
// operations a second; outputs in fp32 282), 8192^3 410 (2.7e15).  The matrix unit
// is busy 54 % of that; products alone, from registers, reach 3.9e15 with 16 or
// more accumulators a wave (2.2e15 to 2.6e15 with 8 and fewer), and so do those of
// 32 x 32 x 32.  Of its variants, where this loop took 249: operands read where
// they are used 304; steps of 64 k in four buffers 346 (rows of 64 bytes are read
// at half the rate); copies between the products, or behind an earlier second
// barrier, 273 and 265; persistent workgroups with the next tile's first copies
// ahead of the outputs 272; waves of 64 x 128 288.
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_i8_many(I8Params p) {
  constexpr int NW = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16, KS = 128;
  constexpr int CW = BN / 8 / NW, CX = BM / 8 / NW, C = CW + CX;   // 1 KB copies a wave and step
  static_assert(CW * 8 * NW == BN && CX * 8 * NW == BM, "whole copies for each wave");
  __shared__ __align__(1024) int8_t lds[2][(BM + BN) * KS];
  const int w = wave_id(), l = lane_id(), c = l & 15, g = l >> 4;
  const int id = xcd_remap(blockIdx.x, p.tiles);
  if (id >= p.tiles) return;
  // groups of four rows of tiles, column by column, so that the tiles that run
  // at once on an XCD share rows of both operands
  const int per = 4 * p.tn, grp = id / per, in = id - grp * per, gm = min(4, p.tm - grp * 4);
  const int m0 = (grp * 4 + in % gm) * BM, n0 = in / gm * BN;
  const i32x4v rw = rsrc_words(p.w + (long)n0 * p.w_stride, i8_range(min(BN, p.N - n0), p.w_stride, p.K));
  const i32x4v rx = rsrc_words(p.x + (long)m0 * p.x_stride, i8_range(min(BM, p.M - m0), p.x_stride, p.K));
  uint32_t ow[CW], ox[CX];
#pragma unroll
  for (int j = 0; j < CW; ++j) {
    const int r = (w * CW + j) * 8 + (l >> 3), in_wave = r % (16 * NT);
    const int n = r - in_wave + 4 * NT * (in_wave % 16 / 4) + 4 * (in_wave / 16) + in_wave % 4;
    ow[j] = (uint32_t)(n * p.w_stride) + 16 * ((l & 7) ^ stage_swz<8>(r & 15));
  }
#pragma unroll
  for (int j = 0; j < CX; ++j) {
    const int r = (w * CX + j) * 8 + (l >> 3);
    ox[j] = (uint32_t)(r * p.x_stride) + 16 * ((l & 7) ^ stage_swz<8>(r & 15));
  }
  const int steps = (p.K + KS - 1) / KS;
  // steps behind the last are copied from behind the descriptors' ranges: zeros
  auto copy_one = [&](int j, uint32_t k0, int buf) __attribute__((always_inline)) {
    if (j < CW) lds_copy16(rw, ow[j < CW ? j : 0] + k0, lds_addr(&lds[buf][(w * CW + j) * 8 * KS]));
    else lds_copy16(rx, ox[j < CW ? 0 : j - CW] + k0, lds_addr(&lds[buf][(BN + (w * CX + j - CW) * 8) * KS]));
  };
  auto copy_at = [&](int s) { return s < steps ? (uint32_t)(s * KS) : 0x80000000u; };
  const int wm = w % WM, wn = w / WM;
  const int aw = (wn * 16 * NT + c) * KS, ax = (BN + wm * 16 * MT + c) * KS;
  i32x4 acc[NT][MT], fw[2][NT], fx[2][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto read = [&](int buf, auto half) __attribute__((always_inline)) {
    constexpr int H = decltype(half)::value;
    const int at = 16 * ((4 * H + g) ^ stage_swz<8>(c));
#pragma unroll
    for (int i = 0; i < NT; ++i) fw[H][i] = *reinterpret_cast<const i32x4*>(&lds[buf][aw + i * 16 * KS + at]);
#pragma unroll
    for (int j = 0; j < MT; ++j) fx[H][j] = *reinterpret_cast<const i32x4*>(&lds[buf][ax + j * 16 * KS + at]);
  };
  auto products = [&](auto half) __attribute__((always_inline)) {
    constexpr int H = decltype(half)::value;
#pragma unroll
    for (int k = 0; k < NT * MT; ++k) acc[k / MT][k % MT] = i8_mma(fw[H][k / MT], fx[H][k % MT], acc[k / MT][k % MT]);
  };
  auto copy = [&](int s, int buf) __attribute__((always_inline)) {
    const uint32_t k0 = copy_at(s);
#pragma unroll
    for (int j = 0; j < C; ++j) copy_one(j, k0, buf);
  };
  copy(0, 0);
  copy(1, 1);
  i8_landed<C>();
  lds_barrier();
  read(0, ic<0>{});
  int buf = 0;
  for (int s = 0; s + 1 < steps; ++s) {
    read(buf, ic<1>{});
    products(ic<0>{});
    i8_landed<0>();    // of the next step, this wave's copies; and its reads of this one are done
    lds_barrier();     // and everybody's
    copy(s + 2, buf);
    buf ^= 1;
    read(buf, ic<0>{});
    products(ic<1>{});
  }
  read(buf, ic<1>{});
  if (steps * KS > p.K) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      fw[0][i] = i8_head(fw[0][i], (steps - 1) * KS + 16 * g, p.K);
      fw[1][i] = i8_head(fw[1][i], (steps - 1) * KS + 64 + 16 * g, p.K);
    }
  }
  products(ic<0>{});
  products(ic<1>{});
  i8_landed<0>();   // no copy outlives the wave
  // a lane's 4 NT values of a row one after another, so that cache lines fill at
  // once (in two turns of 16 bytes each was written twice: 267 MB for 134)
  constexpr int V = sizeof(T) == 2 ? 8 : 4;   // 16 bytes of y
  auto leave = [&](auto all) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(all)::value;   // every n of the tile is there
    const int n = n0 + wn * 16 * NT + 4 * NT * g;
    float ws[4 * NT], bias[4 * NT];
#pragma unroll
    for (int e = 0; e < 4 * NT; e += 4) {
      float f[4], h[4] = {0.f, 0.f, 0.f, 0.f};
      vec_load<float, 4>(p.ws + n + e, WHOLE ? 4 : max(0, p.N - n - e), f);
      if (p.bias) vec_load<float, 4>(p.bias + n + e, WHOLE ? 4 : max(0, p.N - n - e), h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ws[e + i] = f[i];
        bias[e + i] = h[i];
      }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int m = m0 + wm * 16 * MT + 16 * j + c;
      if (m >= p.M) continue;
      const float xs = p.xs[m];
#pragma unroll
      for (int e = 0; e < 4 * NT; e += V) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (float)acc[(e + i) / 4][j][i % 4] * xs * ws[e + i] + bias[e + i];
        vec_store<T, V>(static_cast<T*>(p.y) + (long)m * p.N + n + e, WHOLE ? V : p.N - n - e, f);
      }
    }
  };
  if (n0 + BN <= p.N) leave(std::true_type{});
  else leave(std::false_type{});
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

template <typename T, int MT, int NT, int ST>
static void i8_some(const I8Params& p, hipStream_t st) {
  hipLaunchKernelGGL((k_i8_some<T, MT, NT, ST>), dim3((unsigned)(((p.N + 16L * NT - 1) / (16 * NT)) * ((p.M + 16L * MT - 1) / (16 * MT)))), dim3(256), 0, st, p);
}
template <typename T, int BM, int BN, int WM, int WN>
static void i8_many(I8Params p, hipStream_t st) {
  p.tm = (p.M + BM - 1) / BM;
  p.tn = (p.N + BN - 1) / BN;
  p.tiles = p.tm * p.tn;
  hipLaunchKernelGGL((k_i8_many<T, BM, BN, WM, WN>), dim3((p.tiles + 7) / 8 * 8), dim3(64 * WM * WN), 0, st, p);
}
// The variant with the shortest rounds: workgroups over compute units, rounded
// up, times what a round takes (k = 4096, bf16, us beside the launch, which is
// some 3 for all):
//   x rows by weight rows    32 x 32   64 x 32   128 x 32   128 x 64   128 x 128   256 x 256
//   a round                     6         7         8         12.5        20           57
// The order of the rounds is that of other k too: of 56 cases (k of 512, 1024,
// 4096 and 16384, 1 to 2048 rows, 2048 and 8192 columns) this choice was within 0.8
// us or 4 % of the fastest in all but one (1024 rows, 512 -> 2048: 10.5 us, 8.0 in
// 128 x 128).
// Measured, us a call, 4096 -> 8192: 17 rows 9.3 (64 x 32: 9.8), 40 rows 10.0 (32
// x 32: 14, 128 x 32: 11.3), 100 rows 12.5 (64 x 32: 17.4, 128 x 64: 16.5), 256
// rows 18.1 (128 x 32: 26, 128 x 128: 24.9), 512 rows 27.8 (128 x 64: 33.5, 256 x
// 256: 46), 1024 rows 41 (48), 2048 rows 62 (128 x 128: 80); 4096 -> 2048: 256
// rows 7.8 (128 x 32: 11.3), 1024 rows 17.3 (64 x 32: 26, 128 x 128: 25).  A
// launch is below 2^32 threads: from 2^29 columns on small tiles are none.
template <typename T>
static hipError_t i8_matmul(const I8Params& p, hipStream_t st) {
  timing_before("matmul_i8", st);
  const struct { int bm, bn; float round; } kinds[] = {{32, 32, 6.f}, {64, 32, 7.f}, {128, 32, 8.f}, {128, 64, 12.5f}, {128, 128, 20.f}, {256, 256, 57.f}};
  int best = 5;
  float least = __builtin_inff();
  for (int k = 0; k < 6; ++k) {
    const long tiles = ((p.M + kinds[k].bm - 1L) / kinds[k].bm) * ((p.N + kinds[k].bn - 1L) / kinds[k].bn);
    const float cost = (float)((tiles + kComputeUnits - 1) / kComputeUnits) * kinds[k].round;
    if (tiles * 256 < 1L << 32 && cost < least) {
      best = k;
      least = cost;
    }
  }
  switch (best) {
    case 0: i8_some<T, 2, 2, 6>(p, st); break;
    case 1: i8_some<T, 4, 2, 4>(p, st); break;
    case 2: i8_some<T, 8, 2, 3>(p, st); break;
    case 3: i8_some<T, 8, 4, 3>(p, st); break;
    case 4: i8_many<T, 128, 128, 2, 2>(p, st); break;
    default: i8_many<T, 256, 256, 2, 4>(p, st);
  }
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_i8_matmul(DType dt, const I8Params& p, hipStream_t st) {
  return dt == DType::BF16 ? i8_matmul<bf16>(p, st) : i8_matmul<float>(p, st);
}

}  // namespace gdr
