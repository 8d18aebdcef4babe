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
// A workgroup takes one segment of the token axis and 16 channels (x columns of
// one group's heads) for each of its waves, up to 256 channels in at most 4
// heads; a wave keeps its [N, 16] block of the state in fp32 accumulators.
// The scores C B^T of a chunk are the same for every head of the group: a
// wave computes a 16 x 16 tile of them and leaves it in LDS with each head's
// decays applied, so that nothing of it is computed twice; the gates of the
// next chunk are made meanwhile by waves without a tile.  16 waves of 128
// registers hide each other's latencies: their output pass takes 65 us (8192
// tokens, 64 heads of 64, N = 128), and took 68 where 8 waves of 32 channels
// took 76, 4 of 64 channels 89, and two workgroups of 8 waves a compute unit 78.
// What bounds it: the three-term state update (19 us of it), the chunk's
// products and decays (21) and the tiles' movement (31) share two barriered
// phases and overlap in part only.
//
// Long prompts are cut into segments that run side by side: a first pass
// computes what each segment adds to the state and its decay, k_ssm_join
// turns those into the states at the segment ends, and the output pass starts
// from them, all exact.  Segments are cut on the packed token axis, so that
// ragged batches balance by themselves.
#include "gdr_layer.h"

namespace gdr {

constexpr int SC = 64;        // chunk

// Staged tiles: SC rows of NCH 16-byte pieces, unpadded (they are filled by
// direct global -> LDS copies); piece c of row r stands at c ^ ssm_swz(r),
// which takes the low four bits of r only.
template <typename T, int NCH>
__device__ __forceinline__ int ssm_swz(int r) {
  if constexpr (sizeof(T) == 4) return r & (NCH < 16 ? NCH - 1 : 15);
  else return stage_swz<NCH>(r & 15);
}

// A contraction block of 32 indices.  Over the state (n): lane group
// q = lane / 16 holds n = 8 q + e, e < 8, a contiguous piece of a row of B or
// C; the two accumulator tiles of the block hold n = 8 q + 4 u + e % 4 in tile
// u, so that their registers are the other operand as they stand.  Over the
// tokens (j): lane group q holds j = 16 (e / 4) + 4 q + e % 4, the rows of two
// score tiles, one above the other.
template <typename T> struct Blk;
template <> struct Blk<bf16> {
  typedef bf16x8 frag;
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pair(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), bf16x2));
  }
  typedef uint2 quad;   // four values, as they stand in an operand
  static __device__ __forceinline__ quad four(const f32x4& x) { return make_uint2(pair(x[0], x[1]), pair(x[2], x[3])); }
  static __device__ __forceinline__ frag join(quad x, quad y) { return __builtin_bit_cast(frag, make_uint4(x.x, x.y, y.x, y.y)); }
  static __device__ __forceinline__ frag acc(const f32x4& x, const f32x4& y) {
    return __builtin_bit_cast(frag, make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(y[0], y[1]), pair(y[2], y[3])));
  }
  static __device__ __forceinline__ float get(const frag& f, int e) {
    const uint4 u = __builtin_bit_cast(uint4, f);
    const uint32_t v = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
    return __builtin_bit_cast(float, e & 1 ? v & 0xffff0000u : v << 16);
  }
  // NaN if a value is not finite (0 * it), else 0
  static __device__ __forceinline__ float unsound(const frag& f, float sum) {
    const uint4 u = __builtin_bit_cast(uint4, f);
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v[i]), __builtin_bit_cast(bf16x2, 0u), sum, false);
    return sum;
  }
  static __device__ __forceinline__ void set(frag& f, int e, float v) { f[e] = (bf16)v; }
};
template <> struct Blk<float> {
  struct frag { float v[8]; };
  static __device__ __forceinline__ f32x4 mma(const frag& a, const frag& b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  typedef f32x4 quad;
  static __device__ __forceinline__ quad four(const f32x4& x) { return x; }
  static __device__ __forceinline__ frag join(const quad& x, const quad& y) { return acc(x, y); }
  static __device__ __forceinline__ frag acc(const f32x4& x, const f32x4& y) {
    return frag{{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
  }
  static __device__ __forceinline__ float get(const frag& f, int e) { return f.v[e]; }
  static __device__ __forceinline__ float unsound(const frag& f, float sum) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(f.v[e], 0.f, sum);
    return sum;
  }
  static __device__ __forceinline__ void set(frag& f, int e, float v) { f.v[e] = v; }
};

// Operand reads from staged tiles.  A lane's byte address is its row's start
// plus (constant of the block) ^ (constant of the lane), and constant row
// steps that the instruction's offset holds: a few registers for all of them.
template <typename T, int NB, int NX> struct Reader;
template <int NB, int NX> struct Reader<bf16, NB, NX> {
  int arow, ax, brow, bx, xrow, xx;
  __device__ __forceinline__ Reader(int w) {
    const int l = lane_id(), c = l & 15, q = l >> 4, r = 4 * q + (c >> 2), s = c & 3, wx = 32 * (w & 7);
    arow = c * NB * 16;
    ax = 16 * (q ^ ssm_swz<bf16, NB>(c));
    brow = r * NB * 16;
    bx = 16 * (s ^ ssm_swz<bf16, NB>(r));
    xrow = r * NX * 16 + 8 * (s & 1);
    xx = wx ^ (16 * ((s >> 1) ^ ssm_swz<bf16, NX>(r)));
  }
  // four channels 4 q of this wave's columns of x, of token c of the first tile; further tiles 256 NX bytes on
  static __device__ __forceinline__ const char* own_x(const bf16* t, int w, int c, int q) {
    return reinterpret_cast<const char*>(t) + c * NX * 16 + ((32 * (w & 7)) ^ (16 * ((q >> 1) ^ ssm_swz<bf16, NX>(c)))) + 8 * (q & 1);
  }
  static __device__ __forceinline__ f32x4 x4(const char* a) {
    const uint2 u = *reinterpret_cast<const uint2*>(a);
    return f32x4{__builtin_bit_cast(float, u.x << 16), __builtin_bit_cast(float, u.x & 0xffff0000u),
                 __builtin_bit_cast(float, u.y << 16), __builtin_bit_cast(float, u.y & 0xffff0000u)};
  }
  // n along row 16 it + c
  __device__ __forceinline__ bf16x8 along(const bf16* t, int it, int kb) const {
    return *reinterpret_cast<const bf16x8*>(reinterpret_cast<const char*>(t) + arow + ((64 * kb) ^ ax) + it * 256 * NB);
  }
  static __device__ __forceinline__ bf16x8 tr(const char* a, int step) {
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    return cat4(__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)a), __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(a + step)));
  }
  // tokens of block jb down the columns 32 kb + 8 (c / 4) + 4 u + c % 4
  __device__ __forceinline__ bf16x8 down_b(const bf16* t, int jb, int kb, int u) const {
    return tr(reinterpret_cast<const char*>(t) + brow + ((64 * kb) ^ bx) + 8 * u + jb * 512 * NB, 256 * NB);
  }
  // and down this wave's 16 columns of x
  __device__ __forceinline__ bf16x8 down_x(const bf16* t, int jb) const {
    return tr(reinterpret_cast<const char*>(t) + xrow + xx + jb * 512 * NX, 256 * NX);
  }
};
template <int NB, int NX> struct Reader<float, NB, NX> {
  typedef Blk<float>::frag frag;
  int arow, ax, brow, bx, xrow, xx;
  __device__ __forceinline__ Reader(int w) {
    const int l = lane_id(), c = l & 15, q = l >> 4, wx = 64 * (w & 7);
    arow = c * NB * 16;
    ax = 16 * ((2 * q) ^ ssm_swz<float, NB>(c));
    brow = 4 * q * NB * 16 + 4 * (c & 3);
    bx = 16 * ((2 * (c >> 2)) ^ ssm_swz<float, NB>(4 * q));
    xrow = 4 * q * NX * 16 + 4 * (c & 3);
    xx = wx ^ (16 * ((c >> 2) ^ ssm_swz<float, NX>(4 * q)));
  }
  static __device__ __forceinline__ const char* own_x(const float* t, int w, int c, int q) {
    return reinterpret_cast<const char*>(t) + c * NX * 16 + ((64 * (w & 7)) ^ (16 * (q ^ ssm_swz<float, NX>(c))));
  }
  static __device__ __forceinline__ f32x4 x4(const char* a) { return *reinterpret_cast<const f32x4*>(a); }
  __device__ __forceinline__ frag along(const float* t, int it, int kb) const {
    const char* p = reinterpret_cast<const char*>(t) + arow + it * 256 * NB;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p + ((128 * kb) ^ ax)), hi = *reinterpret_cast<const f32x4*>(p + ((128 * kb + 16) ^ ax));
    return Blk<float>::acc(lo, hi);
  }
  // row 4 q + 16 (e / 4) + e % 4 of a block: its swizzle is that of 4 q, ^ e % 4
  static __device__ __forceinline__ frag rows(const char* p, int x, int pitch) {
    frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = *reinterpret_cast<const float*>(p + (x ^ (16 * (e % 4))) + (16 * (e / 4) + e % 4) * pitch);
    return f;
  }
  __device__ __forceinline__ frag down_b(const float* t, int jb, int kb, int u) const {
    return rows(reinterpret_cast<const char*>(t) + brow + jb * 512 * NB, (128 * kb + 16 * u) ^ bx, NB * 16);
  }
  __device__ __forceinline__ frag down_x(const float* t, int jb) const {
    return rows(reinterpret_cast<const char*>(t) + xrow + jb * 512 * NX, xx, NX * 16);
  }
};

// One wave's share of a tile's copy: blocks w, w + NW, ... of 64 pieces.
// Offsets are per lane and the same for every chunk; columns from `cols` on
// point behind any buffer and read as zero, as do rows behind the descriptor.
template <typename T, int NCH, int NW>
struct TileCopy {
  static constexpr int VEC = 16 / (int)sizeof(T), BLOCKS = SC * NCH / 64, NV = (BLOCKS + NW - 1) / NW;
  uint32_t off[NV];
  __device__ __forceinline__ void plan(long stride, int cols) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = 64 * (wave_id() + NW * i) + lane_id(), r = p / NCH, c = (p % NCH) ^ ssm_swz<T, NCH>(r);
      off[i] = c * VEC < cols ? (uint32_t)(r * (int)stride + c * VEC) * (uint32_t)sizeof(T) : 0x80000000u;
    }
  }
  __device__ __forceinline__ void issue(T* lds, const T* base, long stride, int rows, int cols) const {
    const i32x4v rs = rsrc_words(base, ((long)(rows - 1) * stride + cols) * (long)sizeof(T));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int blk = wave_id() + NW * i;
      if (BLOCKS % NW == 0 || blk < BLOCKS) lds_copy16(rs, off[i], lds_addr(lds + 64 * blk * VEC));
    }
  }
};

// A double moved between lanes by a DPP control; lanes without a source, and
// rows outside the mask, get 0.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Inclusive sum over the lanes of a wave: shifts within the rows of 16, then
// the last lane of the rows before (no LDS: a sixth of the latency of shuffles).
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp_f64<0x111>(x);        // row_shr 1, 2, 4, 8
  x += dpp_f64<0x112>(x);
  x += dpp_f64<0x114>(x);
  x += dpp_f64<0x118>(x);
  x += dpp_f64<0x142, 0xA>(x);   // lane 15 of a row to rows 1 and 3
  x += dpp_f64<0x143, 0xC>(x);   // lane 31 to rows 2 and 3
  return x;
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane) << 32) |
                                        (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane));
}

constexpr int SHEADS = 4;       // heads of a workgroup, at most
constexpr int SCU = 128;        // staged sequence offsets

template <typename T, int ND, int NW, bool OUT>
struct SsmLds {
  static constexpr int VEC = 16 / (int)sizeof(T);
  static constexpr int NB = ND / VEC, NX = 128 / VEC;              // pieces of a row of B or C, of x (128 channels)
  static constexpr int XT = NW / 8;                                // x tiles of 128 channels
  static constexpr int NBUF = sizeof(T) == 2 ? 2 : 1;              // fp32 fills the LDS with one
  static constexpr int REM = OUT && sizeof(T) == 4;
  // per head, tiles (jt <= it) of the decayed scores, by lane: rows j, columns i
  typename Blk<T>::quad score[OUT ? SHEADS : 1][OUT ? 10 * 64 : 1];
  // per head and token: gam as a float (and its remainder, fp32), d, and two
  // weights: at the end of the token's tile of 16, and in the chunk's end
  // state.  Rings: while one chunk is read, the next one's scores are made
  // from its gates, and the gates of the one after that are made.
  float gam[3][SHEADS][SC], wt[3][SHEADS][SC];
  float d[2][OUT ? SHEADS : 1][OUT ? SC : 1], ut[2][OUT ? SHEADS : 1][OUT ? SC : 1];
  float rem[3][REM ? SHEADS : 1][REM ? SC : 1];
  int32_t cu[SCU];
  // the tiles last: what stands before them is in reach of an LDS access's
  // offset field, and needs no address registers of its own
  alignas(16) T b[NBUF][SC * ND];
  alignas(16) T x[OUT ? 1 : NBUF][XT][SC * 128];
  alignas(16) T c[OUT ? NBUF : 1][OUT ? SC * ND : 8];
  // a chunk of y, to leave in whole rows (bf16): the 16 channels of wave w in
  // row r stand at w ^ (r % NW), their halves swapped in rows 8 to 15 of 16, so
  // that the rows of a tile are written to different banks (65.8 us for 67.7)
  static constexpr bool STAGE = OUT && sizeof(T) == 2;
  alignas(16) T y[STAGE ? SC * 16 * NW : 8];
};

template <typename T, int ND, int NW, bool OUT>
__global__ __launch_bounds__(64 * NW, 1) void k_ssm(SsmParams p, int total) {
  typedef Blk<T> K;
  typedef typename K::frag frag;
  typedef SsmLds<T, ND, NW, OUT> Lds;
  constexpr int NK = ND / 32, NB = Lds::NB, NX = Lds::NX, COLS = 16 * NW;
  constexpr bool F32 = sizeof(T) == 4;
  __shared__ __align__(16) Lds lds;
  // workgroups of one segment share B and C: keep them on one XCD
  const int id = xcd_remap(blockIdx.x, total);
  if (id >= total) return;
  const SeqFinder sf = seq_finder<SCU>(p.s, lds.cu);
  // quotients come from vector instructions: the same for every lane, they and
  // the addresses that follow from them go to scalar registers
  auto div = [](int a, int b) { return __builtin_amdgcn_readfirstlane(a / b); };
  const int hp = div(p.H, p.G) * p.P;                   // channels of a group
  const int per_group = (hp + COLS - 1) / COLS;
  const int seg = div(id, p.wgs), wi = id - seg * p.wgs;
  const int g = div(wi, per_group), col0 = (wi - g * per_group) * COLS;
  const int cols = min(COLS, hp - col0);
  const int w = wave_id(), l = lane_id(), c = l & 15, q = l >> 4;
  const bool live = 16 * w < cols;                      // waves without channels still help with copies, scores and gates
  const int chan0 = g * hp + col0;                      // the workgroup's first channel: the first of a head
  const int head0 = div(chan0, p.P), heads = div(cols, p.P);
  const int chan = chan0 + (live ? 16 * w : 0);
  const int head = div(chan, p.P), hd = head - head0, pc = chan - head * p.P;
  const long sstride = (long)p.N * p.P;
  const T* x = static_cast<const T*>(p.x);
  const T* dt = static_cast<const T*>(p.dt);
  const T* Bp = static_cast<const T*>(p.B) + (long)g * ND;
  const T* Cp = static_cast<const T*>(p.C) + (long)g * ND;
  T* y = static_cast<T*>(p.y);
  const long HP = (long)p.H * p.P;
  // the last waves make the gates, one head each
  const int ghd = NW - 1 - w;
  const bool gater = ghd < heads;
  const int ghead = head0 + (gater ? ghd : 0);
  const float A = p.A[ghead], bias = p.bias ? p.bias[ghead] : 0.f;

  // element e of tile h[kb][u]: state row 32 kb + 8 q + 4 u + e, column c
  f32x4 h[NK][2];
  auto state_at = [&](const float* s) { return s + (long)head * sstride + pc; };
  auto each_state = [&](auto f) __attribute__((always_inline)) {
    // made here each time (the asm hides that it is always the same): the
    // addresses kept over the chunk loop would spill the state itself
    int at0 = 8 * q * p.P + c;
    asm volatile("" : "+v"(at0));
#pragma unroll
    for (int kb = 0; kb < NK; ++kb)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) h[kb][u][e] = f(h[kb][u][e], at0 + (32 * kb + 4 * u + e) * p.P);
  };
  auto load_state = [&](const float* s) __attribute__((always_inline)) {
    each_state([&](float, int at) __attribute__((always_inline)) { return s ? s[at] : 0.f; });
  };
  auto store_state = [&](float* s) __attribute__((always_inline)) {
    if (live) each_state([&](float v, int at) __attribute__((always_inline)) { s[at] = v; return v; });
  };

  if constexpr (OUT) {
    // Final states of empty sequences: the segments' workgroups copy them, each
    // its share (workgroups of their own would wait for a compute unit each; by
    // the first segment's alone, 64 empty ones beside a prompt of 8192 tokens of
    // 64 heads took the pass from 67 to 578 us, so 118, of which their bytes are 52).
    if (p.ht) {
      const int every = max(p.segs, 1);
      for (int n0 = 0; n0 < p.s.N; n0 += 64 * every) {
        const int m = n0 + l * every + seg;
        uint64_t empty = __builtin_amdgcn_ballot_w64(m < p.s.N && sf.at(min(m, p.s.N - 1) + 1) <= sf.at(min(m, p.s.N - 1)));
        for (; empty; empty &= empty - 1) {
          const int n = n0 + __builtin_ctzll(empty) * every + seg;
          load_state(p.h0 ? state_at(p.h0 + n * (long)p.H * sstride) : nullptr);
          store_state(const_cast<float*>(state_at(p.ht + n * (long)p.H * sstride)));
        }
      }
    }
  }

  const float skip = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(OUT && p.D ? __builtin_bit_cast(int, p.D[head]) : 0));

  const int seg0 = seg * p.seg, seg1 = min(seg0 + p.seg, p.s.Ttot);
  float total_gam = 0.f;
  const Reader<T, NB, NX> rd(w);
  const uint32_t dt_off = (uint32_t)(l * (int)p.dt_stride * (int)sizeof(T));
  const uint32_t y_off = (uint32_t)((c * (int)HP + chan + 4 * q) * (int)sizeof(T));
  TileCopy<T, NB, NW> cb, cc;
  TileCopy<T, NX, NW> cx[Lds::XT];
  cb.plan(p.b_stride, ND);
  if constexpr (OUT) cc.plan(p.c_stride, ND);
#pragma unroll
  for (int i = 0; i < Lds::XT; ++i) cx[i].plan(p.x_stride, cols - 128 * i);

  // The sequence of token t is the same for every lane: told so, the compiler
  // keeps what follows from it in scalar registers.
  auto find = [&](int t, int& start, int& end) {
    const int n = __builtin_amdgcn_readfirstlane(sf.find(t, start, end));
    start = __builtin_amdgcn_readfirstlane(start);
    end = __builtin_amdgcn_readfirstlane(end);
    return n;
  };
  // One run of tokens [t0, t1) of a sequence, from the state in h.
  auto run = [&](int t0, int t1) __attribute__((always_inline)) {
    uint32_t rdt = 0;
    auto copy_b = [&](int t, int buf) __attribute__((always_inline)) {
      cb.issue(lds.b[buf], Bp + (long)t * p.b_stride, p.b_stride, min(SC, t1 - t), ND);
    };
    auto copy_c = [&](int t, int buf) __attribute__((always_inline)) {
      cc.issue(lds.c[buf], Cp + (long)t * p.c_stride, p.c_stride, min(SC, t1 - t), ND);
    };
    auto copy_x = [&](int t, int buf) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < Lds::XT; ++i)
        cx[i].issue(lds.x[buf][i], x + (long)t * p.x_stride + chan0 + 128 * i, p.x_stride, min(SC, t1 - t), max(cols - 128 * i, 0));
    };
    auto load_dt = [&](int t) __attribute__((always_inline)) {   // tokens behind the run read as zero
      if (!gater || t >= t1) return;
      const rsrc_t r = make_rsrc_u(dt + (long)t * p.dt_stride + ghead, ((long)(min(SC, t1 - t) - 1) * p.dt_stride + 1) * (long)sizeof(T));
      if constexpr (F32) rdt = __builtin_amdgcn_raw_buffer_load_b32(r, dt_off, 0, 0);
      else rdt = __builtin_amdgcn_raw_buffer_load_b16(r, dt_off, 0, 0);   // widened where it is used: here it would be waited for
    };
    // the gates of the chunk at t, lane l its token l, from the dt loaded for it
    auto gates = [&](int t, int gb, int db) __attribute__((always_inline)) {
      float d = __builtin_bit_cast(float, F32 ? rdt : rdt << 16) + bias;
      if (p.softplus) d = softplus_f(d);
      if (t + l >= t1) d = 0.f;
      // gam in 64 bits: a difference of two far sums keeps fp32's accuracy.  A
      // token that forgets everything counts as e^-256, which is zero in fp32
      // (and stays so behind any growth that fp32 could hold): with its own sum,
      // gam behind it would lose the small differences of the tokens that follow
      // (bf16, which keeps gam without its remainder: 3 % where it was -1e6).
      double step = (double)d * (double)A;
      if (step < -256.0) step = -256.0;   // a NaN stays
      const double gam = wave_scan(step);
      const float gf = (float)gam;
      lds.gam[gb][ghd][l] = gf;
      lds.wt[gb][ghd][l] = exp_f((float)(lane_f64(gam, 63) - gam)) * d;   // tokens behind the last have d = 0
      if constexpr (OUT) {
        lds.d[db][ghd][l] = d;
        lds.ut[db][ghd][l] = exp_f((float)(dpp_f64<0x15F>(gam) - gam)) * d;   // row_newbcast 15
        if constexpr (F32) lds.rem[gb][ghd][l] = (float)(gam - (double)gf);
      }
    };
    // Scores, transposed: tile (jt, it) holds B_j . C_i, rows j, columns i, with
    // each head's decays.  Tiles left of the diagonal take e^{gam_i - gam_j} as
    // two factors at the end of tile jt, both at most 1: one exponential for
    // four values.
    auto scores = [&](int buf, int gb, int db) __attribute__((always_inline)) {
      const T* tb = lds.b[buf];
      const T* tc = lds.c[OUT ? buf : 0];
      // the four on the diagonal first, which take longest: one for each SIMD
      for (int o = w; o < 10; o += NW) {
        const int it = o < 4 ? o : o >= 7 ? 3 : o >= 5 ? 2 : 1, jt = o < 4 ? o : o - 4 - it * (it - 1) / 2;
        const int idx = it * (it + 1) / 2 + jt;
        f32x4 s = zero4();
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) s = K::mma(rd.along(tb, jt, kb), rd.along(tc, it, kb), s);
        if (jt < it) {
#pragma unroll 2
          for (int k = 0; k < heads; ++k) {
            const f32x4 uj = *reinterpret_cast<const f32x4*>(&lds.ut[db][k][16 * jt + 4 * q]);
            float df = lds.gam[gb][k][16 * it + c] - lds.gam[gb][k][16 * jt + 15];
            if constexpr (F32) df += lds.rem[gb][k][16 * it + c] - lds.rem[gb][k][16 * jt + 15];
            lds.score[k][idx * 64 + l] = K::four(s * (uj * exp_f(df)));
          }
        } else {
#pragma unroll 2
          for (int k = 0; k < heads; ++k) {
            const float gi = lds.gam[gb][k][16 * it + c];
            const f32x4 gj = *reinterpret_cast<const f32x4*>(&lds.gam[gb][k][16 * jt + 4 * q]);
            const f32x4 dj = *reinterpret_cast<const f32x4*>(&lds.d[db][k][16 * jt + 4 * q]);
            f32x4 rj = zero4();
            float ri = 0.f;
            if constexpr (F32) {
              rj = *reinterpret_cast<const f32x4*>(&lds.rem[gb][k][16 * jt + 4 * q]);
              ri = lds.rem[gb][k][16 * it + c];
            }
            f32x4 pm;
#pragma unroll
            for (int e = 0; e < 4; ++e) pm[e] = 4 * q + e <= c ? s[e] * (exp_f(gi - gj[e] + (ri - rj[e])) * dj[e]) : 0.f;
            lds.score[k][idx * 64 + l] = K::four(pm);
          }
        }
      }
    };
    auto next = [](int gb) { return gb == 2 ? 0 : gb + 1; };

    // Two phases a chunk, a barrier before each.  The first reads C, x and the
    // chunk's scores; the second reads B, and makes the next chunk's scores
    // (ten waves) and the gates of the one after that (others).  Tiles are
    // copied where the phase before has given up their place: B in the first
    // phase, for the second; C and x in the second, C for the next but one.
    // The states pass has the second phase only, with two places for each.
    lds_barrier();   // the tiles of the run before are no longer read
    load_dt(t0);
    copy_b(t0, 0);
    copy_x(t0, 0);
    if constexpr (OUT) {
      copy_c(t0, 0);
      if (Lds::NBUF == 2 && t0 + SC < t1) copy_c(t0 + SC, 1);
    }
    if (gater) gates(t0, 0, 0);
    load_dt(t0 + SC);
    if (gater && t0 + SC < t1) gates(t0 + SC, 1, 1);
    load_dt(t0 + 2 * SC);
    int buf = 0, gb = 0, db = 0;
    if constexpr (OUT) {
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
      lds_barrier();
      scores(0, 0, 0);
    }
    for (int t = t0; t < t1; t += SC) {
      const int len = min(SC, t1 - t);
      const bool more = t + SC < t1;
      const int buf1 = Lds::NBUF == 2 ? buf ^ 1 : 0;
      // This wave's copies of x, C (and B) have landed: vmcnt counts down in
      // order, and two stores at least were issued behind them.
      if (Lds::STAGE && t > t0) __builtin_amdgcn_s_waitcnt(0x0F72);
      else __builtin_amdgcn_s_waitcnt(0x0F70);
      lds_barrier();   // everyone's have, and the scores are there
      // dt for the gates of the next but one has landed too: taken here, before
      // further copies, as the wait for it would be one for them
      asm volatile("" : "+v"(rdt));
      if (Lds::NBUF == 2 && more) {
        copy_b(t + SC, buf1);
        if constexpr (!OUT) copy_x(t + SC, buf1);
      }
      frag xf[2];   // x^T: this wave's columns, tokens 32 jb..
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) xf[jb] = rd.down_x(lds.x[OUT ? 0 : buf][w / 8], jb);
      // h' = e^{gam_n} h + B^T (w x), w_j = e^{gam_n - gam_j} d_j.  The fp32
      // product w x is taken as three bf16 terms of 8 bits each, so that the
      // state is as exact as fp32 operands would make it (one term would leave
      // 2^-8, two 2^-16); B and x are bf16 as they are.  All but the products
      // is done before the barrier, where the other waves' products leave the
      // vector unit idle.
      constexpr int TERMS = F32 ? 1 : 3;
      frag wx[2][TERMS];
      auto weigh = [&]() __attribute__((always_inline)) {
        const float gend = lds.gam[gb][hd][SC - 1], en = exp_f(gend);
        total_gam += gend;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
          for (int u = 0; u < 2; ++u) h[kb][u] *= en;
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
          f32x4 u0 = *reinterpret_cast<const f32x4*>(&lds.wt[gb][hd][32 * jb + 4 * q]);
          f32x4 u1 = *reinterpret_cast<const f32x4*>(&lds.wt[gb][hd][32 * jb + 16 + 4 * q]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u0[e] *= K::get(xf[jb], e);
            u1[e] *= K::get(xf[jb], 4 + e);
          }
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            wx[jb][k] = K::acc(u0, u1);
            if (k + 1 < TERMS)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                u0[e] -= K::get(wx[jb][k], e);
                u1[e] -= K::get(wx[jb][k], 4 + e);
              }
          }
        }
      };
      if constexpr (OUT) {
        // A value of x that is not finite would reach the tokens before it too,
        // through the zeros above the diagonal: such a channel is NaN from the
        // token on (bit 4 it + e of nan_at), and the product takes a zero for it.
        const bool unsound = __builtin_amdgcn_ballot_w64(!(K::unsound(xf[1], K::unsound(xf[0], 0.f)) == 0.f)) != 0;
        uint32_t nan_at = 0;
        if (__builtin_expect(unsound, 0)) {
          int behind = 4 * q - c;
          asm volatile("" : "+v"(behind));   // nothing of this is kept over the chunk loop
#pragma unroll
          for (int jb = 0; jb < 2; ++jb)
#pragma unroll
            for (int e = 0; e < 8; ++e) K::set(xf[jb], e, K::get(xf[jb], e) * 0.f == 0.f ? 0.f : 1.f);
#pragma unroll 1
          for (int it = 3; it >= 0; --it) {
            f32x4 count = zero4();   // of them up to token i
#pragma unroll
            for (int jb = 0; jb < 2; ++jb) {
              frag upto;
#pragma unroll
              for (int e = 0; e < 8; ++e) K::set(upto, e, behind + 32 * jb + 16 * (e / 4) + e % 4 <= 16 * it ? 1.f : 0.f);
              count = K::mma(xf[jb], upto, count);
            }
#pragma unroll
            for (int e = 3; e >= 0; --e) nan_at = nan_at << 1 | (count[e] > 0.f);
          }
#pragma unroll
          for (int jb = 0; jb < 2; ++jb) {
            xf[jb] = rd.down_x(lds.x[0][w / 8], jb);
#pragma unroll
            for (int e = 0; e < 8; ++e) K::set(xf[jb], e, K::get(xf[jb], e) * 0.f == 0.f ? K::get(xf[jb], e) : 0.f);
          }
        }
        // y^T, rows = channels, columns = tokens: first e^{gam_i} h^T C_i
        const T* tc = lds.c[buf];
        f32x4 acc[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) acc[it] = zero4();
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
          const frag hf = K::acc(h[kb][0], h[kb][1]);
#pragma unroll
          for (int it = 0; it < 4; ++it) acc[it] = K::mma(hf, rd.along(tc, it, kb), acc[it]);
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) acc[it] *= exp_f(lds.gam[gb][hd][16 * it + c]);
        if (__builtin_expect(unsound, 0)) {
#pragma unroll
          for (int it = 0; it < 4; ++it)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[it][e] = nan_at >> (4 * it + e) & 1 ? __builtin_nanf("") : acc[it][e];
        }
        // then the tokens of the chunk up to i
        const typename K::quad* sc = lds.score[hd] + l;
        // and last D x_i, in fp32: on the scores' diagonal it would be rounded with
        // them (the usual layer's y 2.28e-3 off its 64-bit values for 1.72e-3, of
        // which its own rounding is 1.66e-3), and put first, the largest term, it
        // would have the others rounded to its last place (fp32: 1.3e-7 for 5.7e-8)
        int l1 = l;
        asm volatile("" : "+v"(l1));   // the address is made here: kept over the chunk loop it would spill
        const char* own = rd.own_x(lds.x[0][w / 8], w, l1 & 15, l1 >> 4);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          if (16 * it >= len) break;
#pragma unroll
          for (int jb = 0; 2 * jb <= it; ++jb) {
            const typename K::quad* s0 = sc + (it * (it + 1) / 2 + 2 * jb) * 64;
            acc[it] = K::mma(xf[jb], K::join(s0[0], 2 * jb < it ? s0[64] : K::four(zero4())), acc[it]);
          }
          acc[it] += skip * rd.x4(own + it * 256 * NX);
          if constexpr (Lds::STAGE) {
            *reinterpret_cast<typename K::quad*>(lds.y + ((16 * it + c) * NW + (w ^ (c % NW))) * 16 + 4 * (q ^ (c >> 3 << 1))) = K::four(acc[it]);
          } else if (live) {   // rows behind the chunk's last lie behind the descriptor
            const rsrc_t yr = make_rsrc_u(y + (long)(t + 16 * it) * HP, (long)(len - 16 * it) * HP * (long)sizeof(T));
            buf_store16(yr, y_off, __builtin_bit_cast(uint4, acc[it]));
          }
        }
        if (__builtin_expect(unsound, 0))
#pragma unroll
          for (int jb = 0; jb < 2; ++jb) xf[jb] = rd.down_x(lds.x[0][w / 8], jb);
        weigh();
        __builtin_amdgcn_s_waitcnt(0x0F70);   // B of the next chunk has landed
        lds_barrier();                        // second phase
        if (more) copy_x(t + SC, 0);
        if (Lds::NBUF == 2 && t + 2 * SC < t1) copy_c(t + 2 * SC, buf);
        if (Lds::NBUF == 2 && more) scores(buf1, next(gb), db ^ 1);
      }
      if (gater && t + 2 * SC < t1) gates(t + 2 * SC, next(next(gb)), db);
      if (t + 3 * SC < t1) load_dt(t + 3 * SC);

      if constexpr (!OUT) weigh();
      const T* tb = lds.b[buf];
#pragma unroll
      for (int jb = 0; jb < 2; ++jb) {
        if (32 * jb >= len) break;
        // two blocks at a time, term by term over their four tiles, so that no
        // product waits for the one before
#pragma unroll
        for (int kb = 0; kb < NK; kb += 2) {
          constexpr int KB = NK > 1 ? 2 : 1;
          frag bf[KB][2];
#pragma unroll
          for (int i = 0; i < KB; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) bf[i][u] = rd.down_b(tb, jb, kb + i, u);
#pragma unroll
          for (int k = 0; k < TERMS; ++k)
#pragma unroll
            for (int i = 0; i < KB; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) h[kb + i][u] = K::mma(bf[i][u], wx[jb][k], h[kb + i][u]);
          }
      }
      if constexpr (Lds::STAGE) {
        // whole rows of the workgroup's channels; those behind the last
        // token or channel lie behind the descriptor
        const rsrc_t yr = make_rsrc_u(y + (long)t * HP, (long)len * HP * (long)sizeof(T));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = (int)threadIdx.x + 64 * NW * k, r = i / (2 * NW), u = (i / 2) % NW, ch = 16 * (u ^ (r % NW)) + 8 * ((i ^ r >> 3) & 1);
          buf_store16(yr, ch < cols ? (uint32_t)((r * (int)HP + chan0 + ch) * 2) : 0x80000000u, *reinterpret_cast<const uint4*>(lds.y + i * 8));
        }
      }
      if constexpr (Lds::NBUF == 1) {
        // one place for B and C: the next chunk's come when this one's are read
        if (more) {
          lds_barrier();
          copy_b(t + SC, 0);
          if constexpr (OUT) copy_c(t + SC, 0);
          else copy_x(t + SC, 0);
          if constexpr (OUT) {
            __builtin_amdgcn_s_waitcnt(0x0F70);
            lds_barrier();
            scores(0, next(gb), db ^ 1);
          }
        }
      }
      buf = buf1;
      gb = next(gb);
      db ^= 1;
    }
  };

  if constexpr (!OUT) {
    int start, end;
    const int n = find(seg1 - 1, start, end);
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
      const int n = find(t, start, end);
      const int stop = min(end, seg1);
      if (n < 0) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (long i = threadIdx.x; i < (long)(stop - t) * (cols / 4); i += 64 * NW) {
          const long r = i / (cols / 4);
          vec_store<T, 4>(y + (t + r) * HP + chan0 + 4 * (i - r * (cols / 4)), 4, zero);
        }
      } else {
        if (SeqFinder::goes_on(t, seg0, start)) load_state(state_at(p.seg_state + (seg - 1) * (long)p.H * sstride));
        else load_state(p.h0 ? state_at(p.h0 + n * (long)p.H * sstride) : nullptr);
        run(t, stop);
        if (p.ht && stop == end) store_state(const_cast<float*>(state_at(p.ht + n * (long)p.H * sstride)));
      }
      t = stop;
    }
  }
}

// States at the segment ends, in place: end_s = b_s + e^{decay_s} end_{s-1}.
// One thread walks four values over the segments, their loads sixteen ahead
// (8192 tokens of 64 heads: 12.7 us, eight ahead 13.8).
__global__ __launch_bounds__(256) void k_ssm_join(SsmParams p) {
  const long per = (long)p.H * p.N * p.P;
  const long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= per) return;
  const int head = (int)(i / ((long)p.N * p.P));
  const int n = p.segs - 1;
  f32x4 cur = zero4();
  for (int s0 = 0; s0 < n; s0 += 16) {
    f32x4 b[16];
    float g[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int s = min(s0 + k, n - 1);
      b[k] = *reinterpret_cast<const f32x4*>(p.seg_state + s * per + i);
      g[k] = p.seg_decay[(long)s * p.H + head];
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
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

// Waves of a workgroup: 16 (256 channels share the tiles of B and C), or 8
// where a group has no more than 128 channels, where 256 would be more heads
// than the gates have room for, and in fp32, whose tiles take twice the LDS.
static int ssm_waves(DType dt, const SsmParams& p) {
  return dt == DType::BF16 && p.P >= 64 && p.H / p.G * p.P > 128 ? 16 : 8;
}

// Segments: enough workgroups for every compute unit, of one chunk at least.
// Up to three chunks (two in fp32) run as one segment: a further chunk takes 5
// us one after another, in fp32 9 to 13, the two further launches 6 to 8 (one
// segment / several, us a call: bf16, 64 heads of 64, N = 128, 3 chunks 23.9 /
// 28.8, 4 chunks 29.1 / 31.1, 6 chunks 39.3 / 37.4; 8 heads, 3 chunks 23.3 /
// 24.4, 4 chunks 28.5 / 24.5; fp32, 8 heads of 32, N = 64, 2 chunks 22.3 / 22.9,
// 3 chunks 31.2 / 23.0; 64 heads of 64, N = 128, 2 chunks 32.2 / 33.2, 3 chunks
// 45.4 / 35.0).
void ssm_plan(DType dt, SsmParams& p) {
  const int hp = p.H / p.G * p.P, cols = 16 * ssm_waves(dt, p);
  p.wgs = p.G * ((hp + cols - 1) / cols);
  const long chunks = ((long)p.s.Ttot + SC - 1) / SC;
  long segs = chunks <= (dt == DType::BF16 ? 3 : 2) ? 1 : (kComputeUnits + p.wgs - 1) / p.wgs;
  segs = segs > chunks ? chunks : segs;
  segs = segs < 1 ? 1 : segs;
  p.seg = (int)((chunks + segs - 1) / segs) * SC;
  if (p.seg < SC) p.seg = SC;
  p.segs = (int)(((long)p.s.Ttot + p.seg - 1) / p.seg);
}

template <typename T, int ND, int NW>
static hipError_t ssm_scan(const SsmParams& p, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (p.segs > 1) {
    const int total = (p.segs - 1) * p.wgs;
    timing_before("ssm_states", st);
    hipLaunchKernelGGL((k_ssm<T, ND, NW, false>), dim3((unsigned)((total + 7) / 8 * 8)), dim3(64 * NW), 0, st, p, total);
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
  // without a token in any sequence, one segment's workgroups copy the states
  const int total = (p.segs > 0 ? p.segs : p.ht ? 1 : 0) * p.wgs;
  if (total == 0) return hipSuccess;
  timing_before("ssm_scan", st);
  hipLaunchKernelGGL((k_ssm<T, ND, NW, true>), dim3((unsigned)((total + 7) / 8 * 8)), dim3(64 * NW), 0, st, p, total);
  e = hipGetLastError();
  timing_after(st);
  return e;
}
template <typename T, int NW>
static hipError_t ssm_scan_n(const SsmParams& p, hipStream_t st) {
  if (p.N == 32) return ssm_scan<T, 32, NW>(p, st);
  return p.N == 64 ? ssm_scan<T, 64, NW>(p, st) : ssm_scan<T, 128, NW>(p, st);
}
hipError_t launch_ssm_scan(DType dt, const SsmParams& p, hipStream_t st) {
  if (dt != DType::BF16) return ssm_scan_n<float, 8>(p, st);
  return ssm_waves(dt, p) == 16 ? ssm_scan_n<bf16, 16>(p, st) : ssm_scan_n<bf16, 8>(p, st);
}

}  // namespace gdr
