// fl_small.cu — launch of the gated linear unit of a few rows (kernel in fl_small.cuh).
#include "fl_host.h"
#include "fl_plan.h"
#include "fl_small.cuh"

using namespace fl;
using namespace fl::host;

namespace {
template <int DT>
void (*by_rows(int64_t M))(SmallArgs) {
  if (M <= 8) return fl_glu_small_kernel<GATE_SWIGLU, DT, 1, 1, 8>;
  return fl_glu_small_kernel<GATE_SWIGLU, DT, 2, 2, 2>;
}
}  // namespace

int fl::host::small_max_rows() { return kSmallMaxRows; }

void fl::host::small_config(fl_plan_s* p) {
  p->small = true;
  p->pair = false;
  p->kernel = reinterpret_cast<const void*>(p->dtype == FL_BF16 ? by_rows<DT_BF16>(p->M) : by_rows<DT_F16>(p->M));
  p->mma_n = p->M <= 8 ? 8 : 16;
  p->out_tile_n = p->M <= 8 ? 8 : 16;
  p->split_k = 1;
  p->stages = 1;
  p->smem = 0;
  p->grid = (int)cdiv(p->N, p->out_tile_n);
  p->launches = 1;
}

fl_status fl::host::small_execute(const fl_plan_s* p, const void* A, const void* W, void* out, cudaStream_t stream) {
  SmallArgs a{};
  a.x = A;
  a.w = W;
  a.out = out;
  a.M = (int)p->M;
  a.N = (int)p->N;
  a.K = (int)p->K;
  a.ldx = p->epi.lda;
  a.ldw = p->epi.ldb;
  a.ldo = p->epi.ldo;
  a.out_dt = p->epi.out_dtype;
  const cudaError_t err = launch_pdl_b(reinterpret_cast<void (*)(SmallArgs)>(const_cast<void*>(p->kernel)),
                                       dim3((unsigned)p->grid), (unsigned)(kSmallWarps * 32), stream, a);
  if (err != cudaSuccess) return fail(FL_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(err));
  return after_launch(stream, "gated linear unit of a few rows");
}
