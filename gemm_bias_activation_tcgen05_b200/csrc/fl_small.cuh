// fl_small.cuh — the gated linear unit of a few rows (serving: one new token of each of up to 16
// sequences): h = act(x·Wgᵀ) ⊙ (x·Wuᵀ), bound by reading the weights once.
//
// Eight output features are a unit: their 8 gate rows and 8 up rows of W are the 16 rows of an
// mma.sync.m16n8k16 operand A, the rows of x its B columns (8 at a time), so that gate and up of a
// feature end in the same lane.  An inner product does not depend on the order of k, so the lanes
// take k in an order of their own: in a step of 32 lane (g, t) holds k = 8t .. 8t + 7 of row g, one
// 16-byte load, whose four words are the k pairs of two products, and the same k of x's row g.
// Weights go from memory to the tensor core through registers: no shared memory, no barrier.
// The products run far below the tensor core's rate (2·M operations a byte), so the legacy warp form
// is enough, and it needs no staging.  The CTA's warps share one unit and take steps of k in turn,
// eight steps (512 bytes of each of 16 rows) at a time, all in flight; their sums meet in shared memory
// in a fixed order.  From 9 rows on x's own loads count: a CTA then takes two units, two steps at a time.
//
// Measured with N 8192, K 4096 bf16 (134 MB of weights, 20.5 us at the copy rate): 1 row 21.2 us
// (6.3 TB/s), 8 rows 23.0, 16 rows 26.6; 32 rows took 44.6, where the pair kernel takes 30.5, so it ends
// at 16.  (1 row with four steps in flight 23-27 us, with four warps a CTA 22.9.)
#pragma once
#include "fl_pair.cuh"

namespace fl {

constexpr int kSmallWarps = 8;
constexpr int kSmallMaxRows = 16;

struct SmallArgs {
  const void *x, *w;
  void* out;
  int M, N, K;
  long long ldx, ldw, ldo;
  int out_dt;
};

// 16 bytes that are read once
__device__ __forceinline__ uint4 ldg_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// elements k .. k + 7 of a row of K, zeros past its end
__device__ __forceinline__ uint4 ldg_tail(const uint16_t* row, int k, int K) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < K ? row[k + 2 * i] : 0u, hi = k + 2 * i + 1 < K ? row[k + 2 * i + 1] : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// d += A·B: A rows 0..7 (a0, a2) and 8..15 (a1, a3), B (b0, b1)
template <int DT>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (DT == DT_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: blocks of 8 rows of x (M ≤ 8·NT); FT: blocks of 8 features a warp (and CTA) owns.
template <int ACT, int DT, int NT, int FT, int U>
__global__ void __launch_bounds__(kSmallWarps * 32, FT == 1 ? 2 : 1) fl_glu_small_kernel(const SmallArgs P) {
  constexpr int W = kSmallWarps;
  __shared__ float part[W][2][8 * FT][8 * NT + 1];  // [warp][gate, up][feature][row of x]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 8 * FT;
  bool n_ok[FT];
  const uint16_t *wg[FT], *wu[FT];
#pragma unroll
  for (int f = 0; f < FT; ++f) {
    n_ok[f] = n0 + 8 * f + g < P.N;
    wg[f] = reinterpret_cast<const uint16_t*>(P.w) + (long long)(n0 + 8 * f + g) * P.ldw;
    wu[f] = wg[f] + (long long)P.N * P.ldw;
  }
  const uint16_t* xr = reinterpret_cast<const uint16_t*>(P.x) + (long long)g * P.ldx;
  float acc[FT][NT][4];
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][j][i] = 0.0f;
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int whole = P.K / (32 * U);  // groups of U whole steps
  for (int s = warp; s < whole; s += W) {
    const int k0 = s * 32 * U + 8 * t;
    uint4 a[U][FT], b[U][FT], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < FT; ++f) {
        a[u][f] = n_ok[f] ? ldg_stream(wg[f] + k0 + 32 * u) : zero;
        b[u][f] = n_ok[f] ? ldg_stream(wu[f] + k0 + 32 * u) : zero;
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        x[u][j] = g + 8 * j < P.M ? *reinterpret_cast<const uint4*>(xr + (long long)(8 * j) * P.ldx + k0 + 32 * u) : zero;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_16816<DT>(acc[f][j], a[u][f].x, b[u][f].x, a[u][f].y, b[u][f].y, x[u][j].x, x[u][j].y);
          mma_16816<DT>(acc[f][j], a[u][f].z, b[u][f].z, a[u][f].w, b[u][f].w, x[u][j].z, x[u][j].w);
        }
  }
  // the last steps, one at a time
#pragma unroll 1
  for (int s = whole * U + warp; 32 * s < P.K; s += W) {
    const int k = 32 * s + 8 * t;
    const bool in = k + 8 <= P.K, some = k < P.K;
    uint4 x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      x[j] = zero;
      if (g + 8 * j < P.M && some) {
        const uint16_t* r = xr + (long long)(8 * j) * P.ldx;
        x[j] = in ? *reinterpret_cast<const uint4*>(r + k) : ldg_tail(r, k, P.K);
      }
    }
#pragma unroll
    for (int f = 0; f < FT; ++f) {
      uint4 a = zero, b = zero;
      if (n_ok[f] && some) {
        a = in ? ldg_stream(wg[f] + k) : ldg_tail(wg[f], k, P.K);
        b = in ? ldg_stream(wu[f] + k) : ldg_tail(wu[f], k, P.K);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_16816<DT>(acc[f][j], a.x, b.x, a.y, b.y, x[j].x, x[j].y);
        mma_16816<DT>(acc[f][j], a.z, b.z, a.w, b.w, x[j].z, x[j].w);
      }
    }
  }
  // lane (g, t): gate and up of feature g and x's rows 8j + 2t, 8j + 2t + 1
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      part[warp][0][8 * f + g][8 * j + 2 * t] = acc[f][j][0];
      part[warp][0][8 * f + g][8 * j + 2 * t + 1] = acc[f][j][1];
      part[warp][1][8 * f + g][8 * j + 2 * t] = acc[f][j][2];
      part[warp][1][8 * f + g][8 * j + 2 * t + 1] = acc[f][j][3];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < 8 * FT * P.M; e += W * 32) {
    const int f = e % (8 * FT), m = e / (8 * FT);
    float vg = 0.0f, vu = 0.0f, slope;
#pragma unroll
    for (int w = 0; w < W; ++w) vg += part[w][0][f][m], vu += part[w][1][f][m];
    const float h = gate_f<ACT>(vg, slope) * vu;
    if (n0 + f < P.N) {
      const long long o = (long long)m * P.ldo + n0 + f;
      if (P.out_dt == DT_BF16) store_elem<DT_BF16>(P.out, o, h);
      else store_elem<DT_F16>(P.out, o, h);
    }
  }
}

}  // namespace fl
