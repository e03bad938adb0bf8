// fl_plan.h — the host-side plan of one layer, shared by the translation units that configure
// and launch it.
#pragma once
#include <cuda.h>

#include "fl_gemm.cuh"
#include "fl_host.h"

using fl::KParams;

// Tensor maps and kernel parameters of the last launch of one call site: a
// repeat call with the same operand pointers launches without re-encoding.
struct LaunchCache {
  bool valid = false;
  const void* key[8] = {};
  CUtensorMap tmA, tmB, tmB2, tmOut;
  KParams k;
};

struct fl_plan_s {
  int64_t M, N, K;
  int dtype, compute;
  fl_epilogue_desc epi;
  int act;
  bool has_bias, has_aux;
  int device, num_sms, max_smem;
  // configuration
  bool swap;
  bool pair;  // two CTAs share one 256-row UMMA tile (cluster of 2)
  bool small;  // the gated linear unit of a few rows (fl_small.cuh)
  int k_atoms;  // 128-byte K atoms per pipeline stage
  int mma_n, out_tile_n, split_k, stages, grid, smem;
  int tiles_a, tiles_b, num_kb;
  // stream-K (16-bit CTA pairs): the last sk_tiles tiles are split along K over
  // sk_clusters pairs; no_sk keeps the data-parallel schedule
  bool no_sk;
  int sk_tiles, sk_clusters;
  float* d_skws;  // partial accumulators, sk_ws_bytes()
  int* d_skflags;
  size_t skws_bytes, skflags_bytes;
  const void* kernel;
  int* d_err;
  // unfused twin
  void* d_tmp;
  int64_t tmp_ld;
  size_t tmp_bytes;
  int launches;
  uint64_t wait_limit_ns;
  LaunchCache cache_fused, cache_unfused;
};

namespace fl {
namespace host {

// The kinds of fl_pair.cuh: the gated linear units, their backward and the weight gradient.
inline bool pair_kind(int kind) { return kind >= FL_EPI_SWIGLU && kind <= FL_EPI_WGRAD; }
inline bool dglu_kind(int kind) { return kind == FL_EPI_DGEGLU_TANH || kind == FL_EPI_DSWIGLU; }
inline bool glu_aux_kind(int kind) { return kind == FL_EPI_GEGLU_TANH_AUX || kind == FL_EPI_SWIGLU_AUX; }
// The argument rules of a pair kind (after the rules that every kind shares).
fl_status pair_check(const char* who, int64_t M, int64_t N, int64_t K, int32_t dtype, const fl_epilogue_desc* e);
// Choose tiles, splits, stages, grid and kernel (num_sms and max_smem set); with `no_workspace` no
// K splits.  Host only.
fl_status pair_config(fl_plan_s* p, bool no_workspace);
// Make the chosen kernels launchable on the current device.
fl_status pair_prepare(const fl_plan_s* p);
// fp32 workspace bytes of the chosen configuration (0: none).
size_t pair_workspace_bytes(const fl_plan_s* p);
fl_status pair_execute(fl_plan_s* p, const void* A, const void* W, void* aux, const void* residual, void* out,
                       cudaStream_t stream);

// The gated linear unit of a few rows: most rows it takes, its configuration and its launch.
int small_max_rows();
void small_config(fl_plan_s* p);
fl_status small_execute(const fl_plan_s* p, const void* A, const void* W, void* out, cudaStream_t stream);

}  // namespace host
}  // namespace fl
