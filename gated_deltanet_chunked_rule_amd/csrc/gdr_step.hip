// gdr_step.hip -- one new token per row: the gated delta rule and the state
// space recurrence, on a pool of fp32 states, in place.
//
//   rule:  S' = e^g S;  p = S'^T k;  S = S' + k (beta (v - p))^T;  o = scale S^T q
//   scan:  S = e^{d A} S + B (d x)^T;                              y = S^T C + D x
//
// Bound by the state's memory traffic: a state column needs nothing of the
// others, so one wave takes 32 columns of one head's [KD, V] state, holds
// them in registers (8 lanes of 4 columns times 8 groups of KD / 8 rows),
// reads them once and writes them once.  Sums over the rows are a lane's own
// rows and then three exchanges between the row groups; no LDS, no barrier.
// In bf16 100 rows of 32 heads of 128 x 128 take 85 us with states that changed
// since (5.0 TB/s; 63 where part of them is still in the last-level cache), 64
// rows of 64 heads of 128 x 64 take 54 (41); one row of 32 heads takes 4.0.
#include "gdr_layer.h"

namespace gdr {

// Sum over the 8 row groups (lane bits 3, 4, 5).
__device__ __forceinline__ f32x4 groups_sum(f32x4 x) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v = x[e];
    v += __shfl_xor(v, 8);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    x[e] = v;
  }
  return x;
}

// N consecutive values of a 16-byte aligned row.
template <typename T, int N>
__device__ __forceinline__ void row_values(const T* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    float q[4];
    vec_load<T, 4>(p + 4 * i, 4, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[4 * i + e] = q[e];
  }
}

template <typename T, int KD, bool RULE>
__global__ __launch_bounds__(256) void k_step(StepParams p) {
  constexpr int R = KD / 8;   // rows per lane
  const int blocks = p.V / 32;
  const long unit = (long)blockIdx.x * (blockDim.x >> 6) + wave_id();
  const int head_block = p.Hv * blocks;
  const long row_l = unit / head_block;
  if (row_l >= p.rows) return;   // wave-uniform
  const int row = (int)row_l;
  const int hb = (int)(unit - row_l * head_block);
  const int h = hb / blocks, l = lane_id();
  const int col = (hb - h * blocks) * 32 + 4 * (l & 7), k0 = (l >> 3) * R;
  const int slot = step_slot(p.slots, row, p.num_slots);
  T* o = static_cast<T*>(p.o) + ((long)row * p.Hv + h) * p.V + col;
  if (slot < 0) {
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    if (l < 8) vec_store<T, 4>(o, 4, zero);
    return;
  }
  float* state = p.state + (((long)slot * p.Hv + h) * KD + k0) * p.V + col;
  f32x4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) s[i] = *reinterpret_cast<const f32x4*>(state + (long)i * p.V);
  const int hq = h / (p.Hv / p.Hq);
  float q[R], k[R], v[4];
  row_values<T, R>(static_cast<const T*>(p.k) + (long)row * p.k_stride + (long)hq * KD + k0, k);
  row_values<T, R>(static_cast<const T*>(p.q) + (long)row * p.q_stride + (long)hq * KD + k0, q);
  row_values<T, 4>(static_cast<const T*>(p.v) + (long)row * p.v_stride + (long)h * p.V + col, v);
  f32x4 out = zero4();
  if constexpr (RULE) {
    const float decay = expf(p.g[(long)row * p.Hv + h]), beta = p.beta[(long)row * p.Hv + h];
    f32x4 pk = zero4();
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] *= decay;
        pk[e] = fmaf(s[i][e], k[i], pk[e]);
      }
    pk = groups_sum(pk);
    f32x4 delta;
#pragma unroll
    for (int e = 0; e < 4; ++e) delta[e] = beta * (v[e] - pk[e]);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = fmaf(k[i], delta[e], s[i][e]);
        out[e] = fmaf(s[i][e], q[i], out[e]);
      }
  } else {
    float d = to_f(static_cast<const T*>(p.dt)[(long)row * p.dt_stride + h]) + (p.bias ? p.bias[h] : 0.f);
    if (p.softplus) d = softplus_f(d);
    const float decay = expf(d * p.A[h]);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = fmaf(k[i], d * v[e], decay * s[i][e]);
        out[e] = fmaf(s[i][e], q[i], out[e]);
      }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) *reinterpret_cast<f32x4*>(state + (long)i * p.V) = s[i];
  out = groups_sum(out);
  if (l < 8) {
    float y[4];
    const float skip = RULE ? 0.f : (p.skip ? p.skip[h] : 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = RULE ? out[e] * p.scale : (p.skip ? fmaf(skip, v[e], out[e]) : out[e]);
    vec_store<T, 4>(o, 4, y);
  }
}

template <typename T, bool RULE>
static hipError_t step(const StepParams& p, hipStream_t st) {
  const long units = (long)p.rows * p.Hv * (p.V / 32);
  // few units: one wave per workgroup spreads them over the compute units
  const int waves = units >= 8L * kComputeUnits ? 4 : 1;
  const dim3 grid((unsigned)((units + waves - 1) / waves)), block(64 * waves);
  timing_before(RULE ? "rule_step" : "ssm_step", st);
  if (p.K == 32) hipLaunchKernelGGL((k_step<T, 32, RULE>), grid, block, 0, st, p);
  else if (p.K == 64) hipLaunchKernelGGL((k_step<T, 64, RULE>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((k_step<T, 128, RULE>), grid, block, 0, st, p);
  const hipError_t e = hipGetLastError();
  timing_after(st);
  return e;
}
hipError_t launch_rule_step(DType dt, const StepParams& p, hipStream_t st) {
  return dt == DType::BF16 ? step<bf16, true>(p, st) : step<float, true>(p, st);
}
hipError_t launch_ssm_step(DType dt, const StepParams& p, hipStream_t st) {
  return dt == DType::BF16 ? step<bf16, false>(p, st) : step<float, false>(p, st);
}

}  // namespace gdr
