// fl_rows.cu — entry points of the row kernels (fl_rows.cuh): dropout, dropout + residual +
// LayerNorm, and its backward pass.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "fl_host.h"
#include "fl_rows.cuh"

using namespace fl;
using namespace fl::host;

namespace {

constexpr int64_t kMaxCols = (1LL << 31) - 64;
constexpr int64_t kMaxRows = (1LL << 31) - 1;

fl_status drop_params(const char* who, const fl_dropout_desc* d, DropParams* out) {
  memset(out, 0, sizeof(*out));
  out->scale = 1.0f;
  if (!d) return FL_OK;
  if (!(d->p >= 0.0f && d->p < 1.0f)) return fail(FL_ERR_INVALID_ARG, "%s: the dropout probability must be in [0, 1)", who);
  if (d->reserved != 0) return fail(FL_ERR_INVALID_ARG, "%s: reserved fields must be 0", who);
  if (reinterpret_cast<uintptr_t>(d->offset_dev) % 8)
    return fail(FL_ERR_ALIGNMENT, "%s: offset_dev must be 8-byte aligned", who);
  set_drop_keys(out, d->seed);
  out->offset = d->offset;
  out->offset_dev = d->offset_dev;
  out->threshold = (uint32_t)((double)d->p * 4294967296.0);  // ⌊p·2^32⌋ (p < 1: below 2^32)
  out->scale = (float)(1.0 / (1.0 - (double)d->p));
  out->on = d->p > 0.0f;
  return FL_OK;
}

// One matrix operand of an entry point: checked, its pitch defaulted, and whether each of its
// rows starts on 16 bytes.
struct Operand {
  const char* name;
  const void* p;
  int64_t ld;
  int dt;
};
fl_status check_operand(const char* who, const Operand& o, int64_t N, Mat* m, int* vec) {
  const int es = esize(o.dt);
  const int64_t ld = o.ld == 0 ? N : o.ld;
  if (ld < N) return fail(FL_ERR_INVALID_ARG, "%s: leading dimension of %s < N", who, o.name);
  if (reinterpret_cast<uintptr_t>(o.p) % es) return fail(FL_ERR_ALIGNMENT, "%s: %s is not aligned to its elements", who, o.name);
  m->p = const_cast<void*>(o.p);
  m->ld = ld;
  m->dt = o.dt;
  if (o.p && !(aligned16(o.p) && (ld * es) % 16 == 0)) *vec = 0;
  return FL_OK;
}
fl_status check_param(const char* who, const char* name, const void* p, int dt, int* vec) {
  if (reinterpret_cast<uintptr_t>(p) % esize(dt)) return fail(FL_ERR_ALIGNMENT, "%s: %s is not aligned to its elements", who, name);
  if (p && !aligned16(p)) *vec = 0;
  return FL_OK;
}
fl_status check_shape(const char* who, int64_t M, int64_t N) {
  if (M < 0 || N < 0) return fail(FL_ERR_INVALID_ARG, "%s: negative size", who);
  if (M > kMaxRows || N > kMaxCols) return fail(FL_ERR_INVALID_ARG, "%s: dimension too large", who);
  return FL_OK;
}
fl_status num_sms(int* sms) {
  int dev = 0;
  FL_CUDA(cudaGetDevice(&dev));
  FL_CUDA(cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev));
  return FL_OK;
}

// Kernel of one call: its launch bounds and the threads and vectors that hold a row.
template <typename Args>
struct RowKernel {
  void (*fn)(Args);
  int threads, vecs, block;  // threads 0: the kernel for rows of any length
};
// The types that have kernels of their own: activations in one type, with the residual stream in
// the same type or in fp32.  Everything else runs on the untyped kernels.
enum RowTypes { ROWS_ANY, ROWS_BF16, ROWS_F16, ROWS_BF16_F32, ROWS_F16_F32, ROWS_F32 };
RowTypes row_types(bool vec, int64_t M, int64_t N, int x, int s, int z) {
  // (the typed kernels count blocks of random numbers in 32 bits)
  if (!vec || N % 8 != 0 || M * (N / 4) >= (1LL << 32) || x != z) return ROWS_ANY;
  if (s == x) return x == FL_BF16 ? ROWS_BF16 : x == FL_F16 ? ROWS_F16 : ROWS_F32;
  if (s == FL_F32) return x == FL_BF16 ? ROWS_BF16_F32 : ROWS_F16_F32;
  return ROWS_ANY;
}
template <int T, int V>
RowKernel<DropLnArgs> ln_of(RowTypes r) {
  switch (r) {
    case ROWS_BF16: return {fl_dropout_ln_kernel<T, V, DT_BF16, DT_BF16, DT_BF16>, T, V, ln_block(T)};
    case ROWS_F16: return {fl_dropout_ln_kernel<T, V, DT_F16, DT_F16, DT_F16>, T, V, ln_block(T)};
    case ROWS_BF16_F32: return {fl_dropout_ln_kernel<T, V, DT_BF16, DT_F32, DT_BF16>, T, V, ln_block(T)};
    case ROWS_F16_F32: return {fl_dropout_ln_kernel<T, V, DT_F16, DT_F32, DT_F16>, T, V, ln_block(T)};
    case ROWS_F32: return {fl_dropout_ln_kernel<T, V, DT_F32, DT_F32, DT_F32>, T, V, ln_block(T)};
    default: return {fl_dropout_ln_kernel<T, V, ANY, ANY, ANY>, T, V, ln_block(T)};
  }
}
template <int T, int V>
RowKernel<DropLnBwdArgs> ln_bwd_of(RowTypes r) {
  switch (r) {
    case ROWS_BF16: return {fl_dropout_ln_bwd_kernel<T, V, DT_BF16, DT_BF16, DT_BF16>, T, V, ln_bwd_block(T)};
    case ROWS_F16: return {fl_dropout_ln_bwd_kernel<T, V, DT_F16, DT_F16, DT_F16>, T, V, ln_bwd_block(T)};
    case ROWS_BF16_F32: return {fl_dropout_ln_bwd_kernel<T, V, DT_BF16, DT_F32, DT_BF16>, T, V, ln_bwd_block(T)};
    case ROWS_F16_F32: return {fl_dropout_ln_bwd_kernel<T, V, DT_F16, DT_F32, DT_F16>, T, V, ln_bwd_block(T)};
    case ROWS_F32: return {fl_dropout_ln_bwd_kernel<T, V, DT_F32, DT_F32, DT_F32>, T, V, ln_bwd_block(T)};
    default: return {fl_dropout_ln_bwd_kernel<T, V, ANY, ANY, ANY>, T, V, ln_bwd_block(T)};
  }
}

// Threads and vectors of a row.  Threads beyond the row's end load and store nothing, but they draw (to
// skip that in the forward pass cost full rows 1.5 %), issue the row's sums and hold its barriers, so a
// row wants to fill its threads: two vectors a thread, or three where the row then needs half the threads
// that two would take (768: 32 of them, 96 vectors, no barrier).  A row of three vectors takes longer,
// which shows where an SM walks few of them.
// Three against two, in us (bf16): forward 32768 x 768 40.7 and 50.0, 16384 x 1280 39.2 and 47.4,
// 8192 x 768 13.1 and 14.5, but 2048 x 768 7.0 and 6.2; backward 32768 x 768 48.3 and 64.9, 16384 x 1280
// 51.7 and 65.6, 8192 x 2560 54.8 and 60.3, 4096 x 5120 47.6 and 50.3, 2048 x 768 10.6 and 10.8, but
// 64 x 768 5.3 and 4.8.
RowKernel<DropLnArgs> ln_kernel(int64_t M, int64_t N, int sms, RowTypes r) {
  const bool many = M > 24 * (int64_t)sms;
  if (N <= 512) return ln_of<32, 2>(r);
  if (N <= 768 && many) return ln_of<32, 3>(r);
  if (N <= 1024) return ln_of<64, 2>(r);
  if (N <= 1536 && many) return ln_of<64, 3>(r);
  if (N <= 2048) return ln_of<128, 2>(r);
  if (N <= 16 * 192) return many ? ln_of<128, 3>(r) : ln_of<192, 2>(r);
  if (N <= 4096) return ln_of<256, 2>(r);
  if (N <= 6144) return ln_of<384, 2>(r);
  if (N <= 8192) return ln_of<512, 2>(r);
  if (N <= 12288) return ln_of<768, 2>(r);
  if (N <= 16384) return ln_of<1024, 2>(r);
  return {fl_dropout_ln_long_kernel, 0, 0, 1024};
}
// Backward: four vectors where a CTA of 256 threads then still holds the row.
RowKernel<DropLnBwdArgs> ln_bwd_kernel(int64_t M, int64_t N, int sms, RowTypes r) {
  const bool many = M > 4 * (int64_t)sms;
  if (N <= 512) return ln_bwd_of<32, 2>(r);
  if (N <= 768 && many) return ln_bwd_of<32, 3>(r);
  if (N <= 1024) return ln_bwd_of<64, 2>(r);
  if (N <= 1536 && many) return ln_bwd_of<64, 3>(r);
  if (N <= 2048) return ln_bwd_of<128, 2>(r);
  if (N <= 16 * 192 && many) return ln_bwd_of<128, 3>(r);
  if (N <= 4096) return ln_bwd_of<256, 2>(r);
  if (N <= 6144) return ln_bwd_of<256, 3>(r);
  if (N <= 8192) return ln_bwd_of<256, 4>(r);
  if (N <= 12288) return ln_bwd_of<512, 3>(r);
  if (N <= 16384) return ln_bwd_of<512, 4>(r);
  return {fl_dropout_ln_bwd_long_kernel, 0, 0, 1024};
}

// Launch geometry of the backward pass: CTAs (each leaves one partial row of dγ and one of dβ)
// and the pitch of those rows.  One CTA per SM: a second one would halve the registers of each thread,
// and the loop, which then keeps fewer loads and draws under way, measured slower with it at every width,
// and would leave twice as many partial rows.  One against two, in us: 8192 x 4096 bf16 78.0 (158 registers) and
// 85.0 (124), with an fp32 stream 89.4 and 96.3, in fp32 108.5 and 113.8; 8192 x 2048 44.1 and 51.3; 2048 x 768 9.1
// and 12.1; 32768 x 768 52.4 and 80.1; 4096 x 8192 77.6 and 133.
struct BwdGeom {
  RowKernel<DropLnBwdArgs> k;
  int grid, ws_ld;
  size_t bytes;
};
BwdGeom bwd_geom(int64_t M, int64_t N, int sms, RowTypes r) {
  BwdGeom g;
  g.k = ln_bwd_kernel(M, N, sms, r);
  const int64_t ctas = cdiv(M, g.k.threads == 0 ? 1 : g.k.block / g.k.threads);
  g.grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)sms));
  g.ws_ld = (int)(cdiv(N, 8) * 8);
  // (a partial row for each row or SM, whichever are fewer: no less than the grid, and never less for more
  // rows, so that a workspace for the longest batch serves the shorter ones)
  g.bytes = (size_t)std::max<int64_t>(1, std::min<int64_t>(M, (int64_t)sms)) * 2 * (size_t)g.ws_ld * sizeof(float);
  return g;
}

// Bytes of one slot of the ring of rows ahead.
template <typename Args>
size_t slot_bytes(const RowKernel<Args>& k, std::initializer_list<const Mat*> ops) {
  if (k.threads == 0) return 0;
  size_t words = 0;
  for (const Mat* m : ops) words += row_words(*m, k.vecs * k.threads);
  return 16 * words * (size_t)(k.block / k.threads);
}
// The ring: two slots of `slot` bytes, or one where two do not fit (but at least `least` bytes).  A ring
// that takes a CTA above 48 KB with the kernel's own arrays needs the kernel's opt-in.
template <typename Args>
fl_status ring_of(const RowKernel<Args>& k, size_t slot, size_t least, Args* P, size_t* smem) {
  constexpr size_t kMost = 200 * 1024;  // of the 227 KB of a CTA; the kernels' own arrays take little
  P->ahead = kRowsAhead * slot <= kMost ? kRowsAhead : 1;
  *smem = std::max(P->ahead * slot, least);
  if (*smem > 24 * 1024)
    FL_CUDA(cudaFuncSetAttribute((const void*)k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost));
  return FL_OK;
}

}  // namespace

// ------------------------------------------------------------------ dropout
extern "C" fl_status fl_dropout(const void* x, const void* residual, void* y, int64_t M, int64_t N, int64_t ld_x,
                                int64_t ld_r, int64_t ld_y, int32_t x_dtype, int32_t y_dtype,
                                const fl_dropout_desc* drop, void* stream_) {
  clear_error();
  const char* who = "fl_dropout";
  const bool empty = M == 0 || N == 0;
  if (!empty && (!x || !y)) return fail(FL_ERR_INVALID_ARG, "%s: null x or y", who);
  fl_status st = check_shape(who, M, N);
  if (st) return st;
  if (!is_dtype(x_dtype) || !is_dtype(y_dtype)) return fail(FL_ERR_INVALID_ARG, "%s: unknown dtype", who);
  DropoutArgs P{};
  if ((st = drop_params(who, drop, &P.d))) return st;
  P.vec = 1;
  if ((st = check_operand(who, {"x", x, ld_x, x_dtype}, N, &P.x, &P.vec)) ||
      (st = check_operand(who, {"residual", residual, ld_r, y_dtype}, N, &P.r, &P.vec)) ||
      (st = check_operand(who, {"y", y, ld_y, y_dtype}, N, &P.y, &P.vec)))
    return st;
  if (empty) return FL_OK;
  P.M = M;
  P.N = (int)N;
  P.nvec = (int)cdiv(N, 8);
  int sms = 148;
  if ((st = num_sms(&sms))) return st;
  const RowTypes types = row_types(P.vec, M, N, x_dtype, y_dtype, x_dtype);
  // at most one resident wave
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(cdiv(M * (int64_t)P.nvec, 256),
                                                              (int64_t)sms * dropout_ctas(types != ROWS_ANY)));
  void (*fn)(DropoutArgs) = types == ROWS_BF16       ? fl_dropout_kernel<DT_BF16, DT_BF16>
                            : types == ROWS_F16      ? fl_dropout_kernel<DT_F16, DT_F16>
                            : types == ROWS_BF16_F32 ? fl_dropout_kernel<DT_BF16, DT_F32>
                            : types == ROWS_F16_F32  ? fl_dropout_kernel<DT_F16, DT_F32>
                            : types == ROWS_F32      ? fl_dropout_kernel<DT_F32, DT_F32>
                                                     : fl_dropout_kernel<ANY, ANY>;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t err = launch_pdl_b(fn, dim3((unsigned)grid), 256u, s, P);
  if (err != cudaSuccess) return fail(FL_ERR_CUDA, "%s: kernel launch: %s", who, cudaGetErrorString(err));
  return after_launch(s, who);
}

// ------------------------------------------------------------------ dropout, residual, LayerNorm
extern "C" fl_status fl_dropout_layernorm(const void* x, const void* residual, const void* gamma, const void* beta,
                                          void* sum, void* z, float* mean, float* rstd, int64_t M, int64_t N,
                                          int64_t ld_x, int64_t ld_r, int64_t ld_sum, int64_t ld_z, int32_t x_dtype,
                                          int32_t sum_dtype, int32_t z_dtype, int32_t param_dtype, float eps,
                                          const fl_dropout_desc* drop, void* stream_) {
  clear_error();
  const char* who = "fl_dropout_layernorm";
  const bool empty = M == 0 || N == 0;
  if (!empty && (!x || !z)) return fail(FL_ERR_INVALID_ARG, "%s: null x or z", who);
  if ((mean == nullptr) != (rstd == nullptr)) return fail(FL_ERR_INVALID_ARG, "%s: mean and rstd go together", who);
  fl_status st = check_shape(who, M, N);
  if (st) return st;
  if (!is_dtype(x_dtype) || !is_dtype(sum_dtype) || !is_dtype(z_dtype) || !is_dtype(param_dtype))
    return fail(FL_ERR_INVALID_ARG, "%s: unknown dtype", who);
  if (!(eps >= 0.0f)) return fail(FL_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  DropLnArgs P{};
  if ((st = drop_params(who, drop, &P.d))) return st;
  P.vec = 1;
  if ((st = check_operand(who, {"x", x, ld_x, x_dtype}, N, &P.x, &P.vec)) ||
      (st = check_operand(who, {"residual", residual, ld_r, sum_dtype}, N, &P.r, &P.vec)) ||
      (st = check_operand(who, {"sum", sum, ld_sum, sum_dtype}, N, &P.s, &P.vec)) ||
      (st = check_operand(who, {"z", z, ld_z, z_dtype}, N, &P.z, &P.vec)) ||
      (st = check_param(who, "gamma", gamma, param_dtype, &P.vec)) ||
      (st = check_param(who, "beta", beta, param_dtype, &P.vec)))
    return st;
  if (reinterpret_cast<uintptr_t>(mean) % 4 || reinterpret_cast<uintptr_t>(rstd) % 4)
    return fail(FL_ERR_ALIGNMENT, "%s: mean or rstd is not 4-byte aligned", who);
  if (empty) return FL_OK;
  P.gamma = gamma;
  P.beta = beta;
  P.mean = mean;
  P.rstd = rstd;
  P.M = M;
  P.N = (int)N;
  P.param_dt = param_dtype;
  P.eps = eps;
  int sms = 148, per_sm = 1;
  if ((st = num_sms(&sms))) return st;
  const RowKernel<DropLnArgs> k = ln_kernel(M, N, sms, row_types(P.vec, M, N, x_dtype, sum_dtype, z_dtype));
  const int64_t ctas = cdiv(M, k.threads == 0 ? 1 : k.block / k.threads);
  size_t smem = 0;
  if ((st = ring_of(k, slot_bytes(k, {&P.x, &P.r}), 0, &P, &smem))) return st;
  // one resident wave of CTAs that walk the rows: their rows ahead are then always in flight
  // (few rows need no query, which small calls would pay for)
  if (ctas > sms) FL_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, (const void*)k.fn, k.block, smem));
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)std::max(1, per_sm) * sms);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t err = launch_pdl_smem(k.fn, dim3(grid), (unsigned)k.block, smem, s, P);
  if (err != cudaSuccess) return fail(FL_ERR_CUDA, "%s: kernel launch: %s", who, cudaGetErrorString(err));
  return after_launch(s, who);
}

// ------------------------------------------------------------------ its backward pass
extern "C" fl_status fl_layernorm_grad_workspace_size(int64_t M, int64_t N, size_t* bytes) {
  clear_error();
  const char* who = "fl_layernorm_grad_workspace_size";
  if (!bytes) return fail(FL_ERR_INVALID_ARG, "%s: null pointer", who);
  fl_status st = check_shape(who, M, N);
  if (st) return st;
  int sms = 148;
  if ((st = num_sms(&sms))) return st;
  *bytes = bwd_geom(M, N, sms, ROWS_ANY).bytes;
  return FL_OK;
}

extern "C" fl_status fl_dropout_layernorm_backward(
    const void* dz, const void* dsum, const void* sum, const float* mean, const float* rstd, const void* gamma,
    void* dres, void* dx, float* dgamma, float* dbeta, int64_t M, int64_t N, int64_t ld_dz, int64_t ld_dsum,
    int64_t ld_sum, int64_t ld_dres, int64_t ld_dx, int32_t x_dtype, int32_t sum_dtype, int32_t z_dtype,
    int32_t param_dtype, const fl_dropout_desc* drop, void* workspace, size_t workspace_bytes, void* stream_) {
  clear_error();
  const char* who = "fl_dropout_layernorm_backward";
  const bool empty = M == 0 || N == 0;
  if (!empty && (!dz || !sum || !mean || !rstd))
    return fail(FL_ERR_INVALID_ARG, "%s: null dz, sum, mean or rstd", who);
  if (!empty && !dres && !dx && !dgamma && !dbeta) return fail(FL_ERR_INVALID_ARG, "%s: no output", who);
  fl_status st = check_shape(who, M, N);
  if (st) return st;
  if (!is_dtype(x_dtype) || !is_dtype(sum_dtype) || !is_dtype(z_dtype) || !is_dtype(param_dtype))
    return fail(FL_ERR_INVALID_ARG, "%s: unknown dtype", who);
  DropLnBwdArgs P{};
  if ((st = drop_params(who, drop, &P.d))) return st;
  P.vec = 1;
  if ((st = check_operand(who, {"dz", dz, ld_dz, z_dtype}, N, &P.dz, &P.vec)) ||
      (st = check_operand(who, {"dsum", dsum, ld_dsum, sum_dtype}, N, &P.ds_in, &P.vec)) ||
      (st = check_operand(who, {"sum", sum, ld_sum, sum_dtype}, N, &P.s, &P.vec)) ||
      (st = check_operand(who, {"dres", dres, ld_dres, sum_dtype}, N, &P.dres, &P.vec)) ||
      (st = check_operand(who, {"dx", dx, ld_dx, x_dtype}, N, &P.dx, &P.vec)) ||
      (st = check_param(who, "gamma", gamma, param_dtype, &P.vec)))
    return st;
  for (const void* p : {(const void*)mean, (const void*)rstd, (const void*)dgamma, (const void*)dbeta})
    if (reinterpret_cast<uintptr_t>(p) % 4) return fail(FL_ERR_ALIGNMENT, "%s: an fp32 vector is not 4-byte aligned", who);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (empty) {
    for (float* q : {dgamma, dbeta})
      if (q && N > 0) FL_CUDA(cudaMemsetAsync(q, 0, (size_t)N * sizeof(float), s));
    return FL_OK;
  }
  int sms = 148;
  if ((st = num_sms(&sms))) return st;
  // (the geometry, and so the workspace, does not depend on the types)
  const BwdGeom g = bwd_geom(M, N, sms, row_types(P.vec, M, N, x_dtype, sum_dtype, z_dtype));
  const bool params = dgamma || dbeta;
  if (params && (!workspace || workspace_bytes < g.bytes || !aligned16(workspace)))
    return fail(FL_ERR_INVALID_ARG, "%s: dgamma and dbeta need a 16-byte aligned workspace of %zu bytes "
                "(fl_layernorm_grad_workspace_size)", who, g.bytes);
  P.mean = mean;
  P.rstd = rstd;
  P.gamma = gamma;
  P.ws = params ? reinterpret_cast<float*>(workspace) : nullptr;
  P.M = M;
  P.N = (int)N;
  P.ws_ld = g.ws_ld;
  P.param_dt = param_dtype;
  size_t smem = 0;
  const size_t parts = g.k.threads > 0 && P.ws ? ln_bwd_part_bytes(g.k.threads, g.k.vecs) : 0;
  if ((st = ring_of(g.k, slot_bytes(g.k, {&P.dz, &P.s, &P.ds_in}), parts, &P, &smem))) return st;
  cudaError_t err = launch_pdl_smem(g.k.fn, dim3((unsigned)g.grid), (unsigned)g.k.block, smem, s, P);
  if (err != cudaSuccess) return fail(FL_ERR_CUDA, "%s: kernel launch: %s", who, cudaGetErrorString(err));
  if (params) {
    if ((st = after_launch(s, who))) return st;
    err = launch_pdl_b(fl_ln_wgrad_kernel, dim3((unsigned)cdiv(N, 32), 2u), 1024u, s, (const float*)P.ws, dgamma, dbeta,
                       P.N, P.ws_ld, g.grid);
    if (err != cudaSuccess) return fail(FL_ERR_CUDA, "%s: reduction kernel launch: %s", who, cudaGetErrorString(err));
  }
  return after_launch(s, who);
}
