// gdr_layer_api.cpp -- C ABI of the operators around the rule: argument
// validation, workspaces and launches.  See include/gdr.h for the contract.
// Messages are literals and nothing here allocates host memory, so no C++
// exception can reach a C caller.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gdr.h"
#include "gdr_layer.h"

namespace {

using gdr::set_error;

// Token counts stay a little under 2^31, so that token numbers plus a tile fit an int.
constexpr long kMaxTokens = 0x7fff0000L;
// Launches hold at most 2^32 - 1 threads.
constexpr long kMaxThreads = 0xffffff00L;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t esize(gdr_dtype d) { return d == GDR_BF16 ? 2 : 4; }
gdr::DType dtype_of(gdr_dtype d) { return d == GDR_BF16 ? gdr::DType::BF16 : gdr::DType::F32; }
gdr_status invalid(const char* m) { return set_error(GDR_ERR_INVALID_ARG, m); }
gdr_status unsupported(const char* m) { return set_error(GDR_ERR_UNSUPPORTED, m); }
gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : set_error(GDR_ERR_HIP, hipGetErrorString(e)); }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

gdr_status check_tokens(int B, int T, bool packed, int num_seqs, gdr_dtype dtype) {
  if (B < 1 || T < 0) return invalid("B must be positive and T not negative");
  if (dtype != GDR_BF16 && dtype != GDR_F32) return unsupported("dtype must be GDR_BF16 or GDR_F32");
  if ((long)B * T > kMaxTokens) return unsupported("too many tokens");
  if (packed && B != 1) return invalid("packed mode (cu_seqlens) requires B == 1");
  if (packed && num_seqs < 1) return invalid("num_seqs must be >= 1 in packed mode");
  return GDR_OK;
}

gdr::SeqRanges ranges(int B, int T, int num_seqs, const int32_t* cu) {
  gdr::SeqRanges s;
  s.cu = cu;
  s.N = cu ? num_seqs : B;
  s.T = T;
  s.Ttot = B * T;
  return s;
}

// Lanes that a row of dim values takes in the norm's and the quantisation's kernels.
long row_threads(int dim) {
  return dim <= 128 ? 16 : dim <= 256 ? 32 : dim <= 512 ? 64 : dim <= 1024 ? 128 : dim <= 4096 ? 256 : dim <= 8192 ? 512 : 1024;
}

// ------------------------------------------------------------ convolution --
gdr_status conv_check(const gdr_conv_shape* sh, bool packed) {
  if (!sh) return invalid("shape is NULL");
  if (gdr_status st = check_tokens(sh->B, sh->T, packed, sh->num_seqs, sh->dtype)) return st;
  if (sh->D < 1) return invalid("D must be positive");
  // channel numbers plus a workgroup's channels (and an item's group of 8) fit an int
  if (sh->D > (1 << 30)) return unsupported("D must be at most 2^30");
  if (sh->W < 2 || sh->W > 4) return unsupported("W must be 2, 3 or 4");
  if (sh->activation != GDR_ACT_NONE && sh->activation != GDR_ACT_SILU) return invalid("unknown activation");
  if (sh->x_stride != 0 && sh->x_stride < sh->D) return invalid("x_stride must be 0 or at least D");
  const long groups = (sh->D + 3L) / 4;
  const long tokens = (long)sh->B * sh->T, seqs = packed ? sh->num_seqs : sh->B;
  if (groups * (tokens / 4 + 1 + seqs) > kMaxThreads) return unsupported("too many tokens times channels");
  return GDR_OK;
}
gdr::ConvParams conv_params(const gdr_conv_shape* sh, const void* x, const void* weight, const void* bias,
                            const void* h0, const int32_t* cu) {
  gdr::ConvParams p = {};
  p.s = ranges(sh->B, sh->T, sh->num_seqs, cu);
  p.x = x; p.weight = weight; p.bias = bias; p.h0 = h0;
  p.x_stride = sh->x_stride ? sh->x_stride : sh->D;
  p.D = sh->D;
  p.act = sh->activation == GDR_ACT_SILU;
  return p;
}
void conv_bwd_tiles(const gdr_conv_shape* sh, int& tile, int& tiles) {
  const int tokens = sh->B * sh->T;
  tile = gdr::conv_bwd_tile(tokens, sh->D);
  tiles = (tokens + tile - 1) / tile;
}
size_t conv_bwd_bytes(const gdr_conv_shape* sh) {
  int tile, tiles;
  conv_bwd_tiles(sh, tile, tiles);
  return align_up(((size_t)tiles * (sh->W + 1) * sh->D + 1) * 4);
}

// ------------------------------------------------------------------- scan --
gdr_status ssm_check(const gdr_ssm_shape* sh, bool packed) {
  if (!sh) return invalid("shape is NULL");
  if (gdr_status st = check_tokens(sh->B, sh->T, packed, sh->num_seqs, sh->dtype)) return st;
  if (sh->H < 1 || sh->G < 1) return invalid("H and G must be positive");
  if (sh->H % sh->G != 0) return invalid("H must be a multiple of G");
  if (sh->P != 32 && sh->P != 64 && sh->P != 128) return unsupported("P must be 32, 64 or 128");
  if (sh->N != 32 && sh->N != 64 && sh->N != 128) return unsupported("N must be 32, 64 or 128");
  // a chunk's 64 rows lie within 2 GiB
  if ((long)sh->H * sh->P > (1 << 22) || (long)sh->G * sh->N > (1 << 22)) return unsupported("H * P and G * N must be at most 2^22");
  if (sh->dt_softplus != 0 && sh->dt_softplus != 1) return invalid("dt_softplus must be 0 or 1");
  const int64_t st[4] = {sh->x_stride, sh->b_stride, sh->c_stride, sh->dt_stride};
  const int64_t least[4] = {(int64_t)sh->H * sh->P, (int64_t)sh->G * sh->N, (int64_t)sh->G * sh->N, sh->H};
  for (int i = 0; i < 4; ++i) {
    if (st[i] != 0 && st[i] < least[i]) return invalid("a token stride is smaller than its row");
    if (st[i] > (1 << 22)) return unsupported("a token stride is over 2^22 elements");
    if (i < 3 && st[i] * esize(sh->dtype) % 16 != 0) return invalid("rows of x, B and C must be 16-byte aligned");
  }
  return GDR_OK;
}
gdr::SsmParams ssm_params(const gdr_ssm_shape* sh, const int32_t* cu) {
  gdr::SsmParams p = {};
  p.s = ranges(sh->B, sh->T, sh->num_seqs, cu);
  p.x_stride = sh->x_stride ? sh->x_stride : (long)sh->H * sh->P;
  p.b_stride = sh->b_stride ? sh->b_stride : (long)sh->G * sh->N;
  p.c_stride = sh->c_stride ? sh->c_stride : (long)sh->G * sh->N;
  p.dt_stride = sh->dt_stride ? sh->dt_stride : sh->H;
  p.H = sh->H; p.G = sh->G; p.P = sh->P; p.N = sh->N;
  p.softplus = sh->dt_softplus;
  gdr::ssm_plan(dtype_of(sh->dtype), p);
  return p;
}
size_t ssm_state_bytes(const gdr::SsmParams& p) {
  return p.segs > 1 ? align_up((size_t)(p.segs - 1) * p.H * p.N * p.P * 4) : 0;
}
size_t ssm_bytes(const gdr::SsmParams& p) {
  return ssm_state_bytes(p) + align_up((size_t)(p.segs > 1 ? p.segs - 1 : 1) * p.H * 4);
}

// ------------------------------------------------------------------- norm --
gdr_status norm_check(const gdr_norm_shape* sh) {
  if (!sh) return invalid("shape is NULL");
  if (sh->dtype != GDR_BF16 && sh->dtype != GDR_F32) return unsupported("dtype must be GDR_BF16 or GDR_F32");
  if (sh->rows < 0 || sh->inner < 1 || sh->dim < 1) return invalid("rows must not be negative, inner and dim positive");
  if (sh->rows % sh->inner != 0) return invalid("rows must be a multiple of inner");
  if (sh->dim > 16384) return unsupported("dim must be at most 16384");
  if (!(std::isfinite(sh->eps) && sh->eps >= 0.f)) return invalid("eps must be finite and not negative");
  if (sh->quant != 0 && sh->quant != 1) return invalid("quant must be 0 or 1");
  if (sh->rows > (kMaxThreads - 1024) / row_threads(sh->dim)) return unsupported("too many rows");
  const gdr_row_stride* st[3] = {&sh->x_stride, &sh->residual_stride, &sh->gate_stride};
  for (const gdr_row_stride* s : st)
    if (s->outer < 0 || s->inner < 0) return invalid("row strides must not be negative");
  return GDR_OK;
}
void row_stride(const gdr_norm_shape* sh, const gdr_row_stride& s, long& outer, long& inner) {
  const bool dense = s.outer == 0 && s.inner == 0;
  outer = dense ? (long)sh->inner * sh->dim : s.outer;
  inner = dense ? sh->dim : s.inner;
}
gdr::NormParams norm_params(const gdr_norm_shape* sh) {
  gdr::NormParams p = {};
  p.rows = sh->rows; p.inner = sh->inner; p.dim = sh->dim; p.eps = sh->eps; p.inv_dim = 1.f / (float)sh->dim;
  row_stride(sh, sh->x_stride, p.xo, p.xi);
  row_stride(sh, sh->residual_stride, p.ro, p.ri);
  row_stride(sh, sh->gate_stride, p.go, p.gi);
  p.blocks = gdr::norm_bwd_blocks(sh->rows, sh->dim);
  return p;
}

// ----------------------------------------------------- linear recurrence --
gdr_status lin_check(const gdr_linear_scan_shape* sh, bool packed) {
  if (!sh) return invalid("shape is NULL");
  if (gdr_status st = check_tokens(sh->B, sh->T, packed, sh->num_seqs, sh->dtype)) return st;
  if (sh->D < 1) return invalid("D must be positive");
  // the gradient's join starts 64 threads a channel, and a row of 64-bit words lies within 2^32 bytes
  if (sh->D > (1 << 25)) return unsupported("D must be at most 2^25");
  const int64_t st[3] = {sh->x_stride, sh->r_stride, sh->i_stride};
  for (int64_t s : st)
    if (s != 0 && s < sh->D) return invalid("a token stride is smaller than its row");
  if ((long)gdr::lin_bwd_tiles(sh->B * sh->T) * gdr::lin_cols(sh->D) > kMaxThreads / 512) return unsupported("too many tokens times channels");
  return GDR_OK;
}
gdr::LinParams lin_params(const gdr_linear_scan_shape* sh, const void* x, const void* r, const void* i, const float* A,
                          const float* h0, const int32_t* cu) {
  gdr::LinParams p = {};
  p.s = ranges(sh->B, sh->T, sh->num_seqs, cu);
  p.x = x; p.r = r; p.i = i; p.A = A; p.h0 = h0;
  p.x_stride = sh->x_stride ? sh->x_stride : sh->D;
  p.r_stride = sh->r_stride ? sh->r_stride : sh->D;
  p.i_stride = sh->i_stride ? sh->i_stride : sh->D;
  p.D = sh->D;
  p.tiles = gdr::lin_tiles(dtype_of(sh->dtype), sh->B * sh->T);
  p.cols = gdr::lin_cols(sh->D);
  return p;
}
// One row of D fp32 values for each tile of tokens.
size_t lin_rows_bytes(const gdr_linear_scan_shape* sh) { return align_up((size_t)gdr::lin_bwd_tiles(sh->B * sh->T) * sh->D * 4); }

// ------------------------------------------------------ norms of a block --
gdr_status block_norm_check(const gdr_block_norm_shape* sh) {
  if (!sh) return invalid("shape is NULL");
  if (sh->dtype != GDR_BF16 && sh->dtype != GDR_F32) return unsupported("dtype must be GDR_BF16 or GDR_F32");
  if (sh->rows < 0 || sh->dim < 1) return invalid("rows must not be negative, dim positive");
  if (sh->dim > 16384) return unsupported("dim must be at most 16384");
  if (!(std::isfinite(sh->eps) && sh->eps >= 0.f)) return invalid("eps must be finite and not negative");
  const int64_t st[3] = {sh->x_stride, sh->residual_stride, sh->gate_stride};
  for (int64_t s : st)
    if (s != 0 && s < sh->dim) return invalid("a row stride is smaller than its row");
  if (sh->rows > kMaxThreads / gdr::block_norm_threads(sh->dim) * gdr::block_norm_rows_per_block(sh->dim)) return unsupported("too many rows");
  return GDR_OK;
}
gdr::BlockNormParams block_norm_params(const gdr_block_norm_shape* sh, const void* x, const void* gate, const void* post,
                                       const void* pre, const void* scale) {
  gdr::BlockNormParams p = {};
  p.rows = sh->rows; p.dim = sh->dim; p.eps = sh->eps; p.inv_dim = 1.f / (float)sh->dim;
  p.x = x; p.gate = gate; p.post = post; p.pre = pre; p.scale = scale;
  p.x_stride = sh->x_stride ? sh->x_stride : sh->dim;
  p.r_stride = sh->residual_stride ? sh->residual_stride : sh->dim;
  p.g_stride = sh->gate_stride ? sh->gate_stride : sh->dim;
  p.blocks = gdr::block_norm_bwd_blocks(sh->rows, sh->dim);
  return p;
}

template <size_t M>
bool all_aligned(const void* const (&p)[M], size_t a) {
  for (const void* q : p)
    if (!aligned(q, a)) return false;
  return true;
}

// The overlap that comes about most easily: an output in an input's place.
bool in_place(const void* out, const void* in) { return out != nullptr && out == in; }

}  // namespace

extern "C" {

gdr_status gdr_causal_conv_fwd(const gdr_conv_shape* shape, const void* x, const void* weight, const void* bias,
                               const void* initial_state, const int32_t* cu_seqlens, void* y, void* final_state,
                               void* stream) {
  if (gdr_status st = conv_check(shape, cu_seqlens != nullptr)) return st;
  if (!weight || (shape->T > 0 && (!x || !y))) return invalid("x, weight and y must be non-NULL");
  const void* ptrs[] = {x, weight, bias, initial_state, y, final_state};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !aligned(cu_seqlens, 4)) return invalid("device pointers must be aligned to their elements");
  if (in_place(y, x) || in_place(final_state, initial_state)) return invalid("y and final_state must not overlap x and initial_state");
  gdr::ConvParams p = conv_params(shape, x, weight, bias, initial_state, cu_seqlens);
  p.y = y;
  p.ht = final_state;
  return done(gdr::launch_conv_fwd(dtype_of(shape->dtype), shape->W, p, static_cast<hipStream_t>(stream)));
}

size_t gdr_causal_conv_bwd_workspace_size(const gdr_conv_shape* shape) {
  if (conv_check(shape, false) != GDR_OK) return 0;
  return conv_bwd_bytes(shape);
}

gdr_status gdr_causal_conv_bwd(const gdr_conv_shape* shape, const void* x, const void* weight, const void* bias,
                               const void* initial_state, const int32_t* cu_seqlens, const void* dy,
                               const void* dht, void* dx, void* dw, void* db, void* dh0, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (gdr_status st = conv_check(shape, cu_seqlens != nullptr)) return st;
  if (!weight || !dw || (shape->T > 0 && (!x || !dy || !dx))) return invalid("x, weight, dy, dx and dw must be non-NULL");
  const void* ptrs[] = {x, weight, bias, initial_state, dy, dht, dx, dw, db, dh0};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !aligned(cu_seqlens, 4)) return invalid("device pointers must be aligned to their elements");
  if (in_place(dx, x) || in_place(dx, dy) || in_place(dh0, initial_state) || in_place(dh0, dht))
    return invalid("dx and dh0 must not overlap x, dy, initial_state and dht");
  if (!workspace || workspace_bytes < conv_bwd_bytes(shape))
    return set_error(GDR_ERR_WORKSPACE, "workspace too small (see gdr_causal_conv_bwd_workspace_size)");
  if (!aligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  gdr::ConvParams p = conv_params(shape, x, weight, bias, initial_state, cu_seqlens);
  p.dy = dy; p.dht = dht; p.dx = dx; p.dw = dw; p.db = db; p.dh0 = dh0;
  p.part = static_cast<float*>(workspace);
  conv_bwd_tiles(shape, p.tile, p.tiles);
  return done(gdr::launch_conv_bwd(dtype_of(shape->dtype), shape->W, p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_causal_conv_step(const gdr_conv_shape* shape, const void* x, const void* weight, const void* bias,
                                void* state, int32_t num_slots, const int32_t* slots, void* y, void* stream) {
  if (gdr_status st = conv_check(shape, false)) return st;
  if (shape->T != 1) return invalid("a step takes T == 1 (B rows)");
  if (!x || !weight || !state || !y) return invalid("x, weight, state and y must be non-NULL");
  if (num_slots < 1 || (!slots && num_slots < shape->B)) return invalid("num_slots must cover the rows");
  const void* ptrs[] = {x, weight, bias, state, y};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !aligned(slots, 4)) return invalid("device pointers must be aligned to their elements");
  if ((long)shape->B * ((shape->D + 511L) / 512) * 64 > kMaxThreads) return unsupported("too many rows times channels");
  gdr::ConvParams p = conv_params(shape, x, weight, bias, nullptr, nullptr);
  p.y = y; p.state = state; p.slots = slots; p.num_slots = num_slots;
  return done(gdr::launch_conv_step(dtype_of(shape->dtype), shape->W, shape->B, p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_step(const gdr_shape* shape, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const void* v, int64_t v_stride, const float* g, const float* beta, float scale, float* state,
                    int32_t num_slots, const int32_t* slots, void* o, void* stream) {
  if (!shape) return invalid("shape is NULL");
  if (gdr_status st = check_tokens(shape->B, shape->T, false, 0, shape->dtype)) return st;
  if (shape->T != 1) return invalid("a step takes T == 1 (B rows)");
  if (shape->Hq < 1 || shape->Hv < 1 || shape->Hv % shape->Hq != 0) return invalid("Hv must be a multiple of Hq");
  if (shape->K != shape->V) return unsupported("K must equal V");
  if (shape->K != 32 && shape->K != 64 && shape->K != 128) return unsupported("K must be 32, 64 or 128");
  if (!(std::isfinite(scale) && scale > 0.f)) return invalid("scale must be finite and > 0");
  if (!q || !k || !v || !g || !beta || !state || !o) return invalid("q, k, v, g, beta, state and o must be non-NULL");
  if (num_slots < 1 || (!slots && num_slots < shape->B)) return invalid("num_slots must cover the rows");
  const int64_t qk = (int64_t)shape->Hq * shape->K, vv = (int64_t)shape->Hv * shape->V;
  if ((q_stride && q_stride < qk) || (k_stride && k_stride < qk) || (v_stride && v_stride < vv))
    return invalid("a row stride is smaller than its row");
  const size_t es = esize(shape->dtype);
  const void* ptrs[] = {q, k, v, state, o};
  if (!all_aligned(ptrs, 16) || q_stride * es % 16 || k_stride * es % 16 || v_stride * es % 16)
    return invalid("rows of q, k, v, o and the states must be 16-byte aligned");
  if (!aligned(g, 4) || !aligned(beta, 4) || !aligned(slots, 4)) return invalid("device pointers must be aligned to their elements");
  if ((long)shape->B * shape->Hv > kMaxThreads / (64 * 4)) return unsupported("too many rows times heads");
  gdr::StepParams p = {};
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.state = state; p.slots = slots; p.o = o;
  p.q_stride = q_stride ? q_stride : qk;
  p.k_stride = k_stride ? k_stride : qk;
  p.v_stride = v_stride ? v_stride : vv;
  p.rows = shape->B; p.Hq = shape->Hq; p.Hv = shape->Hv; p.K = shape->K; p.V = shape->V;
  p.num_slots = num_slots;
  p.scale = scale;
  return done(gdr::launch_rule_step(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

size_t gdr_ssm_scan_fwd_workspace_size(const gdr_ssm_shape* shape) {
  if (ssm_check(shape, false) != GDR_OK) return 0;
  return ssm_bytes(ssm_params(shape, nullptr));
}

gdr_status gdr_ssm_scan_fwd(const gdr_ssm_shape* shape, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const float* dt_bias,
                            const float* initial_state, const int32_t* cu_seqlens, void* y, float* final_state,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (gdr_status st = ssm_check(shape, cu_seqlens != nullptr)) return st;
  if (!A || (shape->T > 0 && (!x || !dt || !B || !C || !y))) return invalid("x, dt, A, B, C and y must be non-NULL");
  const void* wide[] = {x, B, C, y, initial_state, final_state, workspace};
  if (!all_aligned(wide, 16)) return invalid("x, B, C, y, the states and the workspace must be 16-byte aligned");
  const void* f32[] = {A, D, dt_bias, cu_seqlens};
  if (!all_aligned(f32, 4) || !aligned(dt, esize(shape->dtype))) return invalid("device pointers must be aligned to their elements");
  if (in_place(y, x) || in_place(final_state, initial_state)) return invalid("y and final_state must not overlap x and initial_state");
  gdr::SsmParams p = ssm_params(shape, cu_seqlens);
  if (!workspace || workspace_bytes < ssm_bytes(p))
    return set_error(GDR_ERR_WORKSPACE, "workspace too small (see gdr_ssm_scan_fwd_workspace_size)");
  if (((long)p.segs + 8) * p.wgs > kMaxThreads / 512) return unsupported("too many sequences times heads");
  p.x = x; p.dt = dt; p.A = A; p.B = B; p.C = C; p.D = D; p.bias = dt_bias; p.h0 = initial_state;
  p.y = y; p.ht = final_state;
  p.seg_state = static_cast<float*>(workspace);
  p.seg_decay = reinterpret_cast<float*>(static_cast<char*>(workspace) + ssm_state_bytes(p));
  return done(gdr::launch_ssm_scan(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_ssm_step(const gdr_ssm_shape* shape, const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* D, const float* dt_bias, float* state, int32_t num_slots,
                        const int32_t* slots, void* y, void* stream) {
  if (gdr_status st = ssm_check(shape, false)) return st;
  if (shape->T != 1) return invalid("a step takes T == 1 (B rows)");
  if (!x || !dt || !A || !B || !C || !state || !y) return invalid("x, dt, A, B, C, state and y must be non-NULL");
  if (num_slots < 1 || (!slots && num_slots < shape->B)) return invalid("num_slots must cover the rows");
  const void* wide[] = {x, B, C, y, state};
  if (!all_aligned(wide, 16)) return invalid("x, B, C, y and the states must be 16-byte aligned");
  const void* f32[] = {A, D, dt_bias, slots};
  if (!all_aligned(f32, 4) || !aligned(dt, esize(shape->dtype))) return invalid("device pointers must be aligned to their elements");
  if ((long)shape->B * shape->H > kMaxThreads / (64 * 4)) return unsupported("too many rows times heads");
  gdr::StepParams p = {};
  p.q = C; p.k = B; p.v = x; p.dt = dt; p.A = A; p.bias = dt_bias; p.skip = D;
  p.state = state; p.slots = slots; p.o = y;
  p.q_stride = shape->c_stride ? shape->c_stride : (long)shape->G * shape->N;
  p.k_stride = shape->b_stride ? shape->b_stride : (long)shape->G * shape->N;
  p.v_stride = shape->x_stride ? shape->x_stride : (long)shape->H * shape->P;
  p.dt_stride = shape->dt_stride ? shape->dt_stride : shape->H;
  p.rows = shape->B; p.Hq = shape->G; p.Hv = shape->H; p.K = shape->N; p.V = shape->P;
  p.num_slots = num_slots;
  p.softplus = shape->dt_softplus;
  return done(gdr::launch_ssm_step(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_rms_norm_fwd(const gdr_norm_shape* shape, const void* x, const void* residual, const void* gate,
                            const void* weight, void* y, float* scales, void* residual_out, void* stream) {
  if (gdr_status st = norm_check(shape)) return st;
  if (!weight || (shape->rows > 0 && (!x || !y || (shape->quant && !scales))))
    return invalid("x, weight, y (and scales with quant) must be non-NULL");
  const void* ptrs[] = {x, residual, gate, weight, residual_out};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !aligned(scales, 4) || (!shape->quant && !aligned(y, esize(shape->dtype))))
    return invalid("device pointers must be aligned to their elements");
  if (shape->rows == 0) return GDR_OK;
  gdr::NormParams p = norm_params(shape);
  p.x = x; p.residual = residual; p.gate = gate; p.weight = weight;
  p.y = y; p.scales = scales; p.h_out = residual_out;
  return done(gdr::launch_norm_fwd(dtype_of(shape->dtype), shape->quant == 1, p, static_cast<hipStream_t>(stream)));
}

size_t gdr_rms_norm_bwd_workspace_size(const gdr_norm_shape* shape) {
  if (norm_check(shape) != GDR_OK) return 0;
  return align_up(((size_t)gdr::norm_bwd_blocks(shape->rows, shape->dim) * shape->dim + 1) * 4);
}

gdr_status gdr_rms_norm_bwd(const gdr_norm_shape* shape, const void* h, const void* gate, const void* weight,
                            const void* dy, const void* d_res, void* dh, void* dw, void* dgate, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (gdr_status st = norm_check(shape)) return st;
  if (!weight || !dw || (shape->rows > 0 && (!h || !dy || !dh || (gate && !dgate))))
    return invalid("h, weight, dy, dh, dw (and dgate with a gate) must be non-NULL");
  const void* ptrs[] = {h, gate, weight, dy, d_res, dh, dw, dgate};
  if (!all_aligned(ptrs, esize(shape->dtype))) return invalid("device pointers must be aligned to their elements");
  if (!workspace || workspace_bytes < gdr_rms_norm_bwd_workspace_size(shape))
    return set_error(GDR_ERR_WORKSPACE, "workspace too small (see gdr_rms_norm_bwd_workspace_size)");
  if (!aligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  gdr::NormParams p = norm_params(shape);
  p.x = h; p.gate = gate; p.weight = weight; p.dy = dy; p.dres = d_res; p.dh = dh; p.dw = dw; p.dgate = dgate;
  p.part = static_cast<float*>(workspace);
  return done(gdr::launch_norm_bwd(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

size_t gdr_linear_scan_fwd_workspace_size(const gdr_linear_scan_shape* shape) {
  if (lin_check(shape, false) != GDR_OK) return 0;
  return align_up(gdr::lin_fwd_bytes(dtype_of(shape->dtype), shape->B * shape->T, shape->D));
}

gdr_status gdr_linear_scan_fwd(const gdr_linear_scan_shape* shape, const void* x, const void* r, const void* i,
                               const float* A, const float* initial_state, const int32_t* cu_seqlens, void* y,
                               float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  if (gdr_status st = lin_check(shape, cu_seqlens != nullptr)) return st;
  if (!A || (shape->T > 0 && (!x || !r || !i || !y))) return invalid("x, r, i, A and y must be non-NULL");
  const void* ptrs[] = {x, r, i, y};
  const void* f32[] = {A, initial_state, final_state, cu_seqlens};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !all_aligned(f32, 4)) return invalid("device pointers must be aligned to their elements");
  if (in_place(y, x) || in_place(y, r) || in_place(y, i) || in_place(final_state, initial_state))
    return invalid("y and final_state must not overlap x, r, i and initial_state");
  if (!workspace || workspace_bytes < gdr_linear_scan_fwd_workspace_size(shape))
    return set_error(GDR_ERR_WORKSPACE, "workspace too small (see gdr_linear_scan_fwd_workspace_size)");
  if (!aligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  gdr::LinParams p = lin_params(shape, x, r, i, A, initial_state, cu_seqlens);
  p.y = y; p.ht = final_state;
  return done(gdr::launch_lin_fwd(dtype_of(shape->dtype), p, workspace, static_cast<hipStream_t>(stream)));
}

size_t gdr_linear_scan_bwd_workspace_size(const gdr_linear_scan_shape* shape) {
  if (lin_check(shape, false) != GDR_OK) return 0;
  return 4 * lin_rows_bytes(shape);
}

gdr_status gdr_linear_scan_bwd(const gdr_linear_scan_shape* shape, const void* x, const void* r, const void* i,
                               const float* A, const float* initial_state, const int32_t* cu_seqlens, const void* dy,
                               const float* dht, void* dx, void* dr, void* di, float* dA, float* dh0, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (gdr_status st = lin_check(shape, cu_seqlens != nullptr)) return st;
  if (!A || !dA || (shape->T > 0 && (!x || !r || !i || !dy || !dx || !dr || !di)))
    return invalid("x, r, i, A, dy, dx, dr, di and dA must be non-NULL");
  const void* ptrs[] = {x, r, i, dy, dx, dr, di};
  const void* f32[] = {A, initial_state, dht, dA, dh0, cu_seqlens};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !all_aligned(f32, 4)) return invalid("device pointers must be aligned to their elements");
  const void* outs[] = {dx, dr, di};
  for (const void* o : outs)
    if (in_place(o, x) || in_place(o, r) || in_place(o, i) || in_place(o, dy)) return invalid("dx, dr and di must not overlap x, r, i and dy");
  if (in_place(dh0, initial_state) || in_place(dh0, dht)) return invalid("dh0 must not overlap initial_state and dht");
  if (!workspace || workspace_bytes < 4 * lin_rows_bytes(shape))
    return set_error(GDR_ERR_WORKSPACE, "workspace too small (see gdr_linear_scan_bwd_workspace_size)");
  if (!aligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  gdr::LinParams p = lin_params(shape, x, r, i, A, initial_state, cu_seqlens);
  p.tiles = gdr::lin_bwd_tiles(shape->B * shape->T);
  p.dy = dy; p.dht = dht; p.dx = dx; p.dr = dr; p.di = di; p.dA = dA; p.dh0 = dh0;
  float** rows[] = {&p.P, &p.S, &p.Q, &p.part};
  for (int k = 0; k < 4; ++k) *rows[k] = reinterpret_cast<float*>(static_cast<char*>(workspace) + k * lin_rows_bytes(shape));
  return done(gdr::launch_lin_bwd(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_linear_scan_step(const gdr_linear_scan_shape* shape, const void* x, const void* r, const void* i,
                                const float* A, float* state, int32_t num_slots, const int32_t* slots, void* y,
                                void* stream) {
  if (gdr_status st = lin_check(shape, false)) return st;
  if (shape->T != 1) return invalid("a step takes T == 1 (B rows)");
  if (!x || !r || !i || !A || !state || !y) return invalid("x, r, i, A, state and y must be non-NULL");
  if (num_slots < 1 || (!slots && num_slots < shape->B)) return invalid("num_slots must cover the rows");
  const void* ptrs[] = {x, r, i, y};
  const void* f32[] = {A, state, slots};
  if (!all_aligned(ptrs, esize(shape->dtype)) || !all_aligned(f32, 4)) return invalid("device pointers must be aligned to their elements");
  if ((long)shape->B * gdr::lin_cols(shape->D) > kMaxThreads / (64 * 4)) return unsupported("too many rows times channels");
  gdr::LinParams p = lin_params(shape, x, r, i, A, nullptr, nullptr);
  p.y = y; p.ht = state; p.slots = slots; p.num_slots = num_slots;
  return done(gdr::launch_lin_step(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_block_norm_fwd(const gdr_block_norm_shape* shape, const void* x, const void* residual, const void* gate,
                              const void* post_weight, const void* pre_weight, const void* scale, void* y, void* h,
                              void* stream) {
  if (gdr_status st = block_norm_check(shape)) return st;
  if (!post_weight || !pre_weight || (shape->rows > 0 && (!x || !residual || !y || !h)))
    return invalid("x, residual, post_weight, pre_weight, y and h must be non-NULL");
  const void* ptrs[] = {x, residual, gate, post_weight, pre_weight, scale, y, h};
  if (!all_aligned(ptrs, esize(shape->dtype))) return invalid("device pointers must be aligned to their elements");
  if (in_place(h, residual) && shape->residual_stride != 0 && shape->residual_stride != shape->dim)
    return invalid("h may take residual's place only where that is dense");
  if (in_place(y, h) || in_place(y, x) || in_place(y, residual) || in_place(y, gate) || in_place(h, x) || in_place(h, gate))
    return invalid("y and h must not overlap x, gate and each other");
  if (shape->rows == 0) return GDR_OK;
  gdr::BlockNormParams p = block_norm_params(shape, x, gate, post_weight, pre_weight, scale);
  p.residual = residual; p.y = y; p.h_out = h;
  return done(gdr::launch_block_norm_fwd(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

size_t gdr_block_norm_bwd_workspace_size(const gdr_block_norm_shape* shape) {
  if (block_norm_check(shape) != GDR_OK) return 0;
  return align_up(((size_t)gdr::block_norm_bwd_blocks(shape->rows, shape->dim) * 3 * shape->dim + 1) * 4);
}

gdr_status gdr_block_norm_bwd(const gdr_block_norm_shape* shape, const void* x, const void* h, const void* gate,
                              const void* post_weight, const void* pre_weight, const void* scale, const void* dy,
                              const void* d_res, void* dx, void* dh, void* dgate, void* dpost, void* dpre,
                              void* dscale, void* workspace, size_t workspace_bytes, void* stream) {
  if (gdr_status st = block_norm_check(shape)) return st;
  if (!post_weight || !pre_weight || !dpost || !dpre || (scale && !dscale) ||
      (shape->rows > 0 && (!x || !h || !dy || !dx || !dh || (gate && !dgate))))
    return invalid("x, h, post_weight, pre_weight, dy, dx, dh, dpost, dpre (dgate with a gate, dscale with a scale) must be non-NULL");
  const void* ptrs[] = {x, h, gate, post_weight, pre_weight, scale, dy, d_res, dx, dh, dgate, dpost, dpre, dscale};
  if (!all_aligned(ptrs, esize(shape->dtype))) return invalid("device pointers must be aligned to their elements");
  const void* outs[] = {dx, dh, dgate};
  const void* ins[] = {x, h, gate, dy, d_res};
  for (const void* o : outs)
    for (const void* in : ins)
      if (in_place(o, in)) return invalid("dx, dh and dgate must not overlap x, h, gate, dy and d_res");
  if (!workspace || workspace_bytes < gdr_block_norm_bwd_workspace_size(shape))
    return set_error(GDR_ERR_WORKSPACE, "workspace too small (see gdr_block_norm_bwd_workspace_size)");
  if (!aligned(workspace, 16)) return invalid("workspace must be 16-byte aligned");
  gdr::BlockNormParams p = block_norm_params(shape, x, gate, post_weight, pre_weight, scale);
  p.h = h; p.dy = dy; p.dres = d_res;
  p.dx = dx; p.dh = dh; p.dgate = dgate; p.dpost = dpost; p.dpre = dpre; p.dscale = dscale;
  p.part = static_cast<float*>(workspace);
  return done(gdr::launch_block_norm_bwd(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_quantize_rows(const gdr_quantize_shape* shape, const void* x, int8_t* q, float* scales, void* stream) {
  if (!shape) return invalid("shape is NULL");
  if (shape->dtype != GDR_BF16 && shape->dtype != GDR_F32) return unsupported("dtype must be GDR_BF16 or GDR_F32");
  if (shape->rows < 0 || shape->dim < 1) return invalid("rows must not be negative, dim positive");
  if (shape->dim > 32768) return unsupported("dim must be at most 32768");
  if (shape->rows > (kMaxThreads - 1024) / row_threads(shape->dim)) return unsupported("too many rows");
  const int pad = (shape->dim + 15) / 16 * 16;
  if ((shape->x_stride != 0 && shape->x_stride < shape->dim) || (shape->q_stride != 0 && shape->q_stride < pad))
    return invalid("a row stride is smaller than its row");
  if (shape->q_stride % 16 != 0) return invalid("q_stride must be a multiple of 16");
  if (shape->rows > 0 && (!x || !q || !scales)) return invalid("x, q and scales must be non-NULL");
  if (!aligned(x, esize(shape->dtype)) || !aligned(q, 16) || !aligned(scales, 4))
    return invalid("x and scales must be aligned to their elements, q to 16 bytes");
  if (shape->rows == 0) return GDR_OK;
  gdr::QuantParams p = {};
  p.rows = shape->rows; p.dim = shape->dim; p.pad = pad; p.x = x; p.q = q; p.scales = scales;
  p.x_stride = shape->x_stride ? shape->x_stride : shape->dim;
  p.q_stride = shape->q_stride ? shape->q_stride : pad;
  return done(gdr::launch_quant_rows(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_matmul_i8(const gdr_matmul_i8_shape* shape, const int8_t* x, const float* x_scales, const int8_t* weight,
                         const float* weight_scales, const float* bias, void* y, void* stream) {
  if (!shape) return invalid("shape is NULL");
  if (shape->dtype != GDR_BF16 && shape->dtype != GDR_F32) return unsupported("dtype must be GDR_BF16 or GDR_F32");
  if (shape->M < 0 || shape->N < 1 || shape->K < 1) return invalid("M must not be negative, N and K positive");
  if (shape->K > (1 << 17) - 1) return unsupported("K must be at most 2^17 - 1");
  // row numbers plus a tile's fit an int, and a tile's rows lie within 2^31 bytes
  if (shape->M > (1 << 30) || shape->N > (1 << 30)) return unsupported("M and N must be at most 2^30");
  const int pad = (shape->K + 15) / 16 * 16;
  const int64_t st[2] = {shape->x_stride, shape->w_stride};
  for (int64_t s : st) {
    if (s != 0 && s < shape->K) return invalid("a row stride is smaller than its row");
    if (s % 16 != 0) return invalid("row strides must be multiples of 16");
    if (s > (1 << 22)) return unsupported("a row stride is over 2^22");
  }
  if (!weight || !weight_scales || (shape->M > 0 && (!x || !x_scales || !y)))
    return invalid("x, x_scales, weight, weight_scales and y must be non-NULL");
  const void* f32[] = {x_scales, weight_scales, bias};
  if (!aligned(x, 16) || !aligned(weight, 16)) return invalid("x and weight must be 16-byte aligned");
  if (!all_aligned(f32, 4) || !aligned(y, esize(shape->dtype))) return invalid("device pointers must be aligned to their elements");
  if ((shape->M / 128 + 1L) * (shape->N / 128 + 1L) > kMaxThreads / 512) return unsupported("too many rows times columns");
  if (shape->M == 0) return GDR_OK;
  gdr::I8Params p = {};
  p.x = x; p.w = weight; p.xs = x_scales; p.ws = weight_scales; p.bias = bias; p.y = y;
  p.x_stride = shape->x_stride ? shape->x_stride : pad;
  p.w_stride = shape->w_stride ? shape->w_stride : pad;
  p.M = shape->M; p.N = shape->N; p.K = shape->K;
  return done(gdr::launch_i8_matmul(dtype_of(shape->dtype), p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
