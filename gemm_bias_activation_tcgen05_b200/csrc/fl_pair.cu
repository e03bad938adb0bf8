// fl_pair.cu — configuration and launch of the gated linear units, their backward and the weight
// gradient (kernels in fl_pair.cuh).
#include <algorithm>
#include <cstring>

#include "fl_host.h"
#include "fl_pair.cuh"
#include "fl_plan.h"

using namespace fl;
using namespace fl::host;

namespace {

using PairFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, KParams);

int epi_of(int kind) {
  switch (kind) {
    case FL_EPI_SWIGLU: return EPI_GLU;
    case FL_EPI_GEGLU_TANH_AUX:
    case FL_EPI_SWIGLU_AUX: return EPI_GLU_AUX;
    case FL_EPI_DGEGLU_TANH:
    case FL_EPI_DSWIGLU: return EPI_DGLU;
    default: return EPI_GRAD;
  }
}
bool is_geglu(int kind) { return kind == FL_EPI_GEGLU_TANH_AUX || kind == FL_EPI_DGEGLU_TANH; }

template <int EPI, int ACT, int OUT>
PairFn by_atoms(int atoms) {
  return atoms == 2 ? &fl_pair_tcgen05<EPI, ACT, OUT, 2> : &fl_pair_tcgen05<EPI, ACT, OUT, 1>;
}
template <int EPI, int ACT>
PairFn by_out(int out, int atoms) {
  return out == FL_BF16 ? by_atoms<EPI, ACT, DT_BF16>(atoms) : by_atoms<EPI, ACT, DT_F16>(atoms);
}
// (128-deep stages only: a run is longer than the K loops that take 64-deep ones)
template <int EPI>
PairFn runs_kernel(int out) {
  return out == FL_F32    ? &fl_pair_tcgen05<EPI, GATE_SWIGLU, DT_F32, 2>
         : out == FL_BF16 ? &fl_pair_tcgen05<EPI, GATE_SWIGLU, DT_BF16, 2>
                          : &fl_pair_tcgen05<EPI, GATE_SWIGLU, DT_F16, 2>;
}
PairFn pair_kernel(int epi, bool geglu, int out, int atoms) {
  switch (epi) {
    case EPI_GLU: return by_out<EPI_GLU, GATE_SWIGLU>(out, atoms);  // (GEGLU_TANH has kernels of its own)
    case EPI_GLU_AUX:
      return geglu ? by_out<EPI_GLU_AUX, GATE_GEGLU_TANH>(out, atoms) : by_out<EPI_GLU_AUX, GATE_SWIGLU>(out, atoms);
    case EPI_DGLU: return geglu ? by_out<EPI_DGLU, GATE_GEGLU_TANH>(out, atoms) : by_out<EPI_DGLU, GATE_SWIGLU>(out, atoms);
    case EPI_GLU_PART: return by_atoms<EPI_GLU_PART, GATE_SWIGLU, DT_F32>(atoms);
    case EPI_DGLU_PART: return by_atoms<EPI_DGLU_PART, GATE_SWIGLU, DT_F32>(atoms);
    case EPI_GRAD_ADD:  // (fp32: 64-deep stages only, see pair_config)
      return out == FL_F32 ? &fl_pair_tcgen05<EPI_GRAD_ADD, GATE_SWIGLU, DT_F32, 1> : by_out<EPI_GRAD_ADD, GATE_SWIGLU>(out, atoms);
    case EPI_RUNS: return runs_kernel<EPI_RUNS>(out);
    case EPI_RUNS_ADD: return runs_kernel<EPI_RUNS_ADD>(out);
    default:
      return out == FL_F32 ? by_atoms<EPI_GRAD, GATE_SWIGLU, DT_F32>(atoms) : by_out<EPI_GRAD, GATE_SWIGLU>(out, atoms);
  }
}
void (*finish_kernel(int kind))(FinishArgs) {
  switch (epi_of(kind)) {
    case EPI_GRAD: return fl_split_finish_kernel<EPI_GRAD, GATE_SWIGLU>;
    case EPI_DGLU:
      return is_geglu(kind) ? fl_split_finish_kernel<EPI_DGLU, GATE_GEGLU_TANH> : fl_split_finish_kernel<EPI_DGLU, GATE_SWIGLU>;
    default:
      return is_geglu(kind) ? fl_split_finish_kernel<EPI_GLU, GATE_GEGLU_TANH> : fl_split_finish_kernel<EPI_GLU, GATE_SWIGLU>;
  }
}
// What the tile kernel itself computes and writes: with K splits, fp32 partial results.  The residual
// of a weight gradient comes and leaves by TMA when the types agree.  Sums longer than the result's type
// allows are taken in runs (pair_run), K splits' too.
int kernel_epi(const fl_plan_s* p) {
  const int epi = epi_of(p->epi.kind);
  const bool split = p->split_k > 1;
  if (epi == EPI_DGLU) return split ? EPI_DGLU_PART : epi;
  if (epi != EPI_GRAD) return split ? EPI_GLU_PART : epi;
  const bool runs = cdiv(cdiv(p->K, kPairBk), p->split_k) * kPairBk > pair_run(p->epi.out_dtype);
  const bool add = !split && p->epi.has_residual && p->epi.residual_dtype == p->epi.out_dtype;
  return runs ? (add ? EPI_RUNS_ADD : EPI_RUNS) : add ? EPI_GRAD_ADD : EPI_GRAD;
}
// Shared memory of the tile kernel: the ring, the epilogue warps' blocks, the barriers.
struct PairLayout {
  uint32_t stage, staging, bar_off, total;
};
PairLayout pair_layout(const fl_plan_s* p) {
  PairLayout L;
  L.stage = (uint32_t)p->k_atoms * (kPairABytes + (uint32_t)(p->mma_n / 2) * 128u);
  L.staging = 8u * pair_warp_staging(p->k_atoms);
  L.bar_off = (uint32_t)p->stages * L.stage + L.staging;
  L.total = L.bar_off + kPairBarBytes + 1024u;  // (the ring starts on the next 1024 bytes)
  return L;
}

// The workspace of a result in K splits: rows of one split (whole 32-row blocks), columns of one
// partial result (whole 32-column blocks) and of a row (GLU: g and u side by side).
int64_t split_rows(const fl_plan_s* p) { return cdiv(p->M, 32) * 32; }
int64_t part_cols(const fl_plan_s* p) { return cdiv(p->N, 32) * 32; }
int64_t ws_ld(const fl_plan_s* p) { return part_cols(p) * (pair_glu(epi_of(p->epi.kind)) ? 2 : 1); }

}  // namespace

fl_status fl::host::pair_check(const char* who, int64_t M, int64_t N, int64_t K, int32_t dtype, const fl_epilogue_desc* e) {
  const bool wgrad = e->kind == FL_EPI_WGRAD;
  const bool need_b_major = wgrad || dglu_kind(e->kind);
  if (dtype == FL_F32) return fail(FL_ERR_UNSUPPORTED, "%s: this kind takes f16/bf16 operands", who);
  if (e->unfused) return fail(FL_ERR_UNSUPPORTED, "%s: this kind has no unfused twin", who);
  if (e->schedule != FL_SCHED_AUTO) return fail(FL_ERR_UNSUPPORTED, "%s: this kind chooses its own schedule", who);
  if ((e->b_major != 0) != need_b_major)
    return fail(FL_ERR_UNSUPPORTED, need_b_major ? "%s: this kind takes W stored [K,N] (b_major 1)"
                                                 : "%s: this kind takes the stacked [2N,K] weight (b_major 0)", who);
  if (!wgrad && e->out_dtype == FL_F32) return fail(FL_ERR_UNSUPPORTED, "%s: this kind writes f16/bf16", who);
  if (!wgrad && (e->has_residual || (e->scale != 0.0f && e->scale != 1.0f)))
    return fail(FL_ERR_UNSUPPORTED, "%s: this kind has no residual and no scale", who);
  if ((glu_aux_kind(e->kind) || dglu_kind(e->kind)) && N % 8 != 0)
    return fail(FL_ERR_ALIGNMENT, "%s: the halves of a [M,2N] buffer start on 16 bytes only when N is a multiple of 8", who);
  (void)M;
  (void)K;
  return FL_OK;
}

// Tile width, K splits, stages and grid, by an estimate of the time of each choice.
//  * A tile is 256 rows by 256 accumulator columns (GLU: 128 gate and 128 up), or by 128 where
//    narrower tiles fill the GPU's pairs better.
//  * Where few tiles would leave most pairs idle while each walks all of K, K is cut into S splits.
fl_status fl::host::pair_config(fl_plan_s* p, bool no_workspace) {
  const int epi = epi_of(p->epi.kind);
  const bool glu = pair_glu(epi);
  const int64_t P = std::max(1, p->num_sms / 2);
  p->swap = false;
  p->small = false;
  if (epi == EPI_GLU && p->M <= small_max_rows()) {
    small_config(p);
    return FL_OK;
  }
  p->pair = true;
  p->k_atoms = 1;
  p->num_kb = (int)cdiv(p->K, kPairBk);
  const double M = (double)p->M, N = (double)p->N, K = (double)p->K, cols = glu ? 2 * N : N;
  double best = 1e300;
  for (int width : {256, 128}) {
    const int64_t tiles = cdiv(p->M, 256) * cdiv(p->N, glu ? width / 2 : width);
    // microseconds of a 64-deep K block, and of what a unit adds outside its K loop.  Measured: a block 0.41
    // 256 wide and 0.26 to 0.34 128 wide; beside its blocks the first round 5, each further one about 1, for
    // which 2.5 a round stands.  The times of one short round come out 1.8 times the estimate, of seven rounds
    // 0.8 times, of long K loops and of K splits 1.0 to 1.2 times.  The epilogue of the backward through the gate
    // (up to 8 us more a round) and the runs of long sums (0.4 us each) are not in it.
    const double block_us = width == 256 ? 0.40 : 0.30, unit_us = 2.5;
    const int most = no_workspace ? 1 : std::min(p->num_kb, 32);
    for (int S = 1; S <= std::max(1, most); ++S) {
      const int64_t units = tiles * S;
      if (units >= (1LL << 24) || (S > 1 && units > 2 * P)) break;  // (the tile raster's range; the workspace's size)
      double us = (double)cdiv(units, P) * ((double)cdiv(p->num_kb, S) * block_us + unit_us);
      // every operand comes from memory once (6 TB/s of the copy's 6.5), by the SMs that are busy
      const double bytes = 2.0 * (M * K + cols * K + (epi == EPI_GRAD ? 2.0 : 3.0) * M * N);
      us = std::max(us, bytes / (6.0e6 * std::min(1.0, (double)units / (double)P)));
      // the partial results are written and read once more (mostly in L2, at about 8 TB/s), by one more launch (3.5)
      if (S > 1) us += 3.5 + (double)S * 8.0 * M * cols / 8e6;
      if (us < best) {
        best = us;
        p->mma_n = width;
        p->split_k = S;
      }
    }
  }
  if (best >= 1e300) return fail(FL_ERR_INVALID_ARG, "fl_plan: dimension too large");
  p->out_tile_n = glu ? p->mma_n / 2 : p->mma_n;
  p->tiles_a = (int)cdiv(p->M, 256);
  p->tiles_b = (int)cdiv(p->N, p->out_tile_n);
  // 128-deep stages where a unit's K loop is long enough to gain from them (see fl_pair.cuh).  From 8
  // blocks on they measured no slower in any kind but the backward through the gate, whose epilogue
  // then has one pair of g, u buffers a warp: about 2.6 us more a 256-wide tile (1.4 a 128-wide one),
  // which shows in the last round, and in every round that is shorter than the epilogue, against 0.03
  // (0.08) us less a block of 64.
  const int kb = p->num_kb / p->split_k;
  if (kernel_epi(p) == EPI_DGLU) {
    const int64_t rounds = cdiv(cdiv(p->M, 256) * cdiv(p->N, p->mma_n), P);
    const bool wide = p->mma_n == 256;
    p->k_atoms = (rounds == 1 || kb >= 20) && (double)rounds * kb * (wide ? 0.03 : 0.08) > (wide ? 2.6 : 1.4) ? 2 : 1;
  } else {
    // (an fp32 residual in short sums needs two 4 KB buffers a warp to come while another leaves: 8192 x 2048
    // of 1024 tokens in one sum 48.5 us so, 72 with one)
    p->k_atoms = kb >= 8 && !(kernel_epi(p) == EPI_GRAD_ADD && p->epi.out_dtype == FL_F32) ? 2 : 1;
  }
  p->num_kb = (int)cdiv(p->K, p->k_atoms * kPairBk);
  p->stages = 0;
  const PairLayout none = pair_layout(p);
  p->stages = (int)std::min<int64_t>(12, std::max<int64_t>(0, (int64_t)p->max_smem - none.total) / none.stage);
  if (p->stages < 2) return fail(FL_ERR_UNSUPPORTED, "fl_plan: shared memory too small");
  p->smem = (int)pair_layout(p).total;
  p->grid = (int)(2 * std::min<int64_t>((int64_t)p->tiles_a * p->tiles_b * p->split_k, P));
  p->kernel = reinterpret_cast<const void*>(
      pair_kernel(kernel_epi(p), is_geglu(p->epi.kind), p->split_k > 1 ? FL_F32 : p->epi.out_dtype, p->k_atoms));
  p->launches = p->split_k > 1 ? 2 : 1;
  return FL_OK;
}

fl_status fl::host::pair_prepare(const fl_plan_s* p) {
  if (p->small) return FL_OK;
  FL_CUDA(cudaFuncSetAttribute(p->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p->max_smem));
  return FL_OK;
}

size_t fl::host::pair_workspace_bytes(const fl_plan_s* p) {
  return p->split_k > 1 ? (size_t)p->split_k * (size_t)split_rows(p) * (size_t)ws_ld(p) * sizeof(float) : 0;
}

fl_status fl::host::pair_execute(fl_plan_s* p, const void* A, const void* W, void* aux, const void* residual, void* out,
                                 cudaStream_t stream) {
  if (p->small) return small_execute(p, A, W, out, stream);
  const fl_epilogue_desc& e = p->epi;
  const int epi = kernel_epi(p);
  const bool split = p->split_k > 1;
  const PairLayout L = pair_layout(p);
  const uint64_t es = 2, eo = (uint64_t)esize(e.out_dtype);
  const uint64_t M = (uint64_t)p->M, N = (uint64_t)p->N, K = (uint64_t)p->K;

  KParams k{};
  k.M = (int)p->M;
  k.N = split ? (int)part_cols(p) : (int)p->N;
  k.K = (int)p->K;
  k.tiles_a = p->tiles_a;
  k.tiles_b = p->tiles_b;
  k.num_kb = p->num_kb;
  k.split_k = p->split_k;
  k.num_stages = p->stages;
  k.mma_n = p->mma_n;
  k.out_tile_n = p->out_tile_n;
  k.b_boxes = p->mma_n / 128;  // 64-column boxes of this CTA's half of an MN-major B
  k.stage_bytes = k.stage_stride = L.stage;
  k.b_atom_bytes = (uint32_t)(p->mma_n / 2) * 128u;
  const uint32_t fmt = p->dtype == FL_BF16 ? 1u : 0u;
  k.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(pair_a_mn(epi) ? 1 : 0) << 15) |
            ((uint32_t)(pair_b_mn(epi) ? 1 : 0) << 16) | ((uint32_t)(p->mma_n >> 3) << 17) | ((256u >> 4) << 24);
  k.tmem_cols = (uint32_t)(2 * p->mma_n);
  k.staging_off = L.bar_off - L.staging;
  k.bar_off = L.bar_off;
  k.residual = split ? nullptr : residual;
  k.ldr = e.ldr;
  k.res_dtype = e.residual_dtype;
  k.out = out;
  k.ldo = e.ldo;
  k.scale = split ? 1.0f : e.scale;
  k.err = p->d_err;
  k.wait_limit_ns = p->wait_limit_ns;
  const int units = p->tiles_a * p->tiles_b * p->split_k, pairs = p->grid / 2;
  k.dp_q = units / pairs;
  k.dp_r = units % pairs;
  k.inv_group = 1.0f / (float)(8 * p->tiles_b);
  k.split_rows = split ? (int)split_rows(p) : 0;

  CUtensorMap mA, mB, mB2, m0, m1, m2, m3;
  for (CUtensorMap* m : {&mA, &mB, &mB2, &m0, &m1, &m2, &m3}) memset(m, 0, sizeof(*m));
  fl_status st = FL_OK;
  if (K > 0) {
    const uint32_t depth = (uint32_t)(p->k_atoms * kPairBk);
    st = pair_a_mn(epi) ? make_map(&mA, A, p->dtype, M, K, (uint64_t)e.lda * es, 64, depth)
                        : make_map(&mA, A, p->dtype, K, M, (uint64_t)e.lda * es, 64, 128);
    if (st) return st;
    if (pair_b_mn(epi)) {
      st = make_map(&mB, W, p->dtype, N, K, (uint64_t)e.ldb * es, 64, depth);
    } else {
      st = make_map(&mB, W, p->dtype, K, N, (uint64_t)e.ldb * es, 64, (uint32_t)p->out_tile_n);
      if (st) return st;
      const char* up = static_cast<const char*>(W) + N * (uint64_t)e.ldb * es;
      st = make_map(&mB2, up, p->dtype, K, N, (uint64_t)e.ldb * es, 64, (uint32_t)p->out_tile_n);
    }
    if (st) return st;
  }
  // the epilogue's tiles: 32 rows x 32 columns
  auto tile = [&](CUtensorMap* m, const void* base, int dt, uint64_t cols, uint64_t rows, uint64_t pitch) {
    return make_map(m, base, dt, cols, rows, pitch, 32, 32, dt != FL_F32);
  };
  if (epi == EPI_DGLU) {
    const char* g = static_cast<const char*>(aux);
    char* dg = static_cast<char*>(out);
    if ((st = tile(&m0, g, e.out_dtype, N, M, 2 * N * eo)) || (st = tile(&m1, g + N * eo, e.out_dtype, N, M, 2 * N * eo)) ||
        (st = tile(&m2, dg, e.out_dtype, N, M, (uint64_t)e.ldo * eo)) ||
        (st = tile(&m3, dg + N * eo, e.out_dtype, N, M, (uint64_t)e.ldo * eo)))
      return st;
    k.n_tma = (int)N;
  } else if (split) {
    k.n_tma = k.N;
    st = tile(&m0, p->d_skws, FL_F32, (uint64_t)ws_ld(p), (uint64_t)p->split_k * (uint64_t)split_rows(p), (uint64_t)ws_ld(p) * 4);
    if (st) return st;
  } else {
    // whole 16-byte granules of a row go out by TMA, the ragged remainder by plain stores
    k.n_tma = (int)(N * eo / 16 * 16 / eo);
    st = tile(&m0, out, e.out_dtype, (uint64_t)std::max<int64_t>(k.n_tma, 16 / (int64_t)eo), M, (uint64_t)e.ldo * eo);
    if (!st && (epi == EPI_GRAD_ADD || epi == EPI_RUNS_ADD)) st = tile(&m1, residual, e.out_dtype, N, M, (uint64_t)e.ldr * eo);
    if (!st && epi == EPI_GLU_AUX) {
      char* g = static_cast<char*>(aux);
      if (!(st = tile(&m1, g, e.out_dtype, N, M, 2 * N * eo))) st = tile(&m2, g + N * eo, e.out_dtype, N, M, 2 * N * eo);
    }
    if (st) return st;
  }

  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p->grid, 1, 1);
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)p->smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t err = cudaLaunchKernelEx(&cfg, reinterpret_cast<PairFn>(const_cast<void*>(p->kernel)), mA, mB, mB2, m0, m1, m2, m3, k);
  if (err != cudaSuccess) return fail(FL_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(err));
  if ((st = after_launch(stream, "pair kernel"))) return st;
  if (!split) return FL_OK;

  FinishArgs r{};
  r.ws = p->d_skws;
  r.split_stride = split_rows(p) * ws_ld(p);
  r.ld_ws = ws_ld(p);
  r.half = part_cols(p);
  r.splits = p->split_k;
  r.residual = residual;
  r.ldr = e.ldr;
  r.res_dtype = e.residual_dtype;
  r.out = out;
  r.ldo = e.ldo;
  r.out_dtype = e.out_dtype;
  r.aux = aux;
  r.M = p->M;
  r.N = (int)p->N;
  r.nvec = (int)cdiv(p->N, 4);
  r.scale = e.scale;
  const int64_t work = p->M * (int64_t)r.nvec;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(cdiv(work, 256), (int64_t)p->num_sms * 8));
  err = launch_pdl_b(finish_kernel(e.kind), dim3(grid), 256u, stream, r);
  if (err != cudaSuccess) return fail(FL_ERR_CUDA, "finishing kernel launch: %s", cudaGetErrorString(err));
  return after_launch(stream, "epilogue after K splits");
}
