// fl_pair.cuh — the products of a gated feed-forward block, forward and backward, as one
// persistent tcgen05 kernel over CTA pairs (256-row UMMA tiles, 16-bit operands, fp32
// accumulators in tensor memory):
//
//   EPI_GLU      h = act(A·Wgᵀ) ⊙ (A·Wuᵀ)                       W = [Wg; Wu] stacked, K contiguous
//   EPI_GLU_AUX  the same, and g = A·Wgᵀ, u = A·Wuᵀ stored for the backward pass
//   EPI_DGLU     dh = A·W (W stored [K, N]), then dg = dh·u·act'(g), du = dh·act(g) from the
//                stored g, u: dh never leaves the chip (but as the fp32 partial sums of K splits)
//   EPI_GRAD     y = (Aᵀ·W + residual)·scale, A stored [K, M] and W stored [K, N]: the weight
//                gradient, K the tokens.  Both operands are read as they lie, through MN-major UMMA
//                descriptors, so nothing is transposed in memory.
//
// When the tiles would leave most pairs idle, K is cut into splits: the kernel then writes fp32
// partial tiles to a workspace (EPI_GLU_PART, EPI_DGLU_PART; EPI_GRAD itself), and a second, small
// kernel adds them in split order and does the epilogue.
//
// Roles (320 threads, one CTA per SM): warp 0 TMA producer, warp 1 TMEM allocator and (rank 0 of
// the pair) UMMA issuer, warps 2..9 epilogue, two per TMEM lane quarter, each with half of the
// tile's columns in blocks of 32, which come and go by TMA.  Two accumulators, so that a tile's
// epilogue runs under the next tile's products.
//
// Stages are ATOMS x 64 deep in K.  Each hand-over of a stage costs the tensor pipe some 40 clocks, so
// 128-deep stages (64 KB a CTA, three of them) run long K loops faster: weight gradient 8192 x 4096 of
// 4096 tokens 202.6 -> 185.6 us (1.48 PFLOP/s), SwiGLU backward 4096 x 8192 x 4096 224.7 -> 216.1.  They
// leave 4 KB of shared memory for each epilogue warp; 64-deep ones (five or six) leave 8 KB, and with them
// the epilogue, which bounds short K loops, waits less for its blocks: SwiGLU backward 2048 x 2048 of 256
// deep 13.5 us with 128-deep stages, 11.5 with 64-deep ones.
//
// Every wait is bounded; on expiry the kernel records an error code and unwinds.
#pragma once
#include "fl_gemm.cuh"

namespace fl {

enum PairEpi : int {
  EPI_GLU = 0, EPI_GLU_AUX = 1, EPI_DGLU = 2, EPI_GRAD = 3, EPI_GLU_PART = 4, EPI_DGLU_PART = 5,
  EPI_GRAD_ADD = 6, EPI_RUNS = 7, EPI_RUNS_ADD = 8
};
enum GateAct : int { GATE_SWIGLU = 0, GATE_GEGLU_TANH = 1 };

constexpr int kPairThreads = (kEpiWarp0 + 8) * 32;
constexpr int kPairBk = 64;                       // K elements of an atom (128 bytes of a K-major row)
constexpr uint32_t kPairABytes = 128u * 128u;     // A: an atom of this CTA's 128 rows
constexpr uint32_t kPairBox = 64u * 128u;         // an MN-major box of 64 columns x 64 K rows
constexpr int kPairBars = 2 * 12 + 6 + 16;        // at most 12 stages; 16: two per epilogue warp
constexpr uint32_t kPairBarBytes = 8u * (uint32_t)kPairBars;

// bytes of one 32 x 32 block of a type, and of the blocks of one epilogue warp
__host__ __device__ constexpr uint32_t pair_block_bytes(int out) { return out == DT_F32 ? 4096u : 2048u; }
__host__ __device__ constexpr uint32_t pair_warp_staging(int atoms) { return atoms == 1 ? 8192u : 4096u; }
__host__ __device__ constexpr bool pair_a_mn(int epi) {
  return epi == EPI_GRAD || epi == EPI_GRAD_ADD || epi == EPI_RUNS || epi == EPI_RUNS_ADD;
}
__host__ __device__ constexpr bool pair_b_mn(int epi) { return pair_a_mn(epi) || epi == EPI_DGLU || epi == EPI_DGLU_PART; }
__host__ __device__ constexpr bool pair_glu(int epi) { return epi == EPI_GLU || epi == EPI_GLU_AUX || epi == EPI_GLU_PART; }

// The tensor core's accumulators round towards zero, which shrinks a sum by 1e-9 of its norm for each k: an
// fp32 result is off by 4.4e-6 at 4096 tokens, 1.9e-5 at 16384.  So weight gradients of many tokens (EPI_RUNS) are
// taken in runs, each in an accumulator of its own, which the epilogue warps add in fp32 registers, rounded to
// nearest (half of the tile's columns a warp: 128 registers), while the next run is multiplied.  Runs of 896 tokens for fp32
// results: 9e-7 whatever the tokens (f16 operands, whose products have more bits: 1.1e-6).  A run costs 0.4 us a tile: 2048 x 2048 of 4096 tokens 25.6 -> 28 us.
// For 16-bit results the run is as long as leaves the shrinkage near a twentieth of the type's own rounding
// (rms 2.1e-4 f16, 1.7e-3 bf16): 8192 tokens for f16 (8e-6), 65536 for bf16 (7e-5).
__host__ __device__ constexpr int pair_run(int out) { return out == DT_F32 ? 896 : out == DT_F16 ? 8192 : 65536; }

// The gates are x·σ(y): y = x (SWIGLU), or y = 2c(x + 0.044715x³), c = √(2/π), for the tanh GELU,
// because (1 + tanh w)/2 = σ(2w): no cancellation for negative x, so that both keep fp32 precision over
// their whole range.  σ(y) = 1/(1 + e^(-y)) with e^(-y) and the reciprocal on the special-function unit
// (relative errors near 2^-22), saturating to 0 and 1; e^(-y) is 2 to the power of x times a polynomial
// in x² that holds the constants.  Two values at a time: eight epilogue warps are few for the arithmetic
// of a tile, and the packed fp32 instructions halve it.
// act(x), and in `slope` act'(x) = σ + x·σ·(1 − σ)·y'(x).  x is held within ±200 where only σ's ends
// matter: no 0·∞ for the largest values.  A NaN stays one, in act and in act'.
constexpr float kLog2E = 1.4426950408889634f, kTwoC = 2.0f * 0.79788456080286536f;
template <int ACT>
__device__ __forceinline__ float2 gate2(float2 x, float2& slope) {
  const float2 one = make_float2(1.0f, 1.0f), minus = make_float2(-1.0f, -1.0f);
  const float2 xc = make_float2(clamp_nan(x.x, 200.0f), clamp_nan(x.y, 200.0f));
  float2 arg, dy = one;
  if constexpr (ACT == GATE_SWIGLU) {
    arg = mul2(xc, make_float2(-kLog2E, -kLog2E));
  } else {
    constexpr float c3 = -0.044715f * kTwoC * kLog2E, c1 = -kTwoC * kLog2E, d3 = 3.0f * 0.044715f * kTwoC;
    const float2 x2 = mul2(xc, xc);
    arg = mul2(xc, fma2(x2, make_float2(c3, c3), make_float2(c1, c1)));
    dy = fma2(x2, make_float2(d3, d3), make_float2(kTwoC, kTwoC));
  }
  const float2 den = add2(make_float2(ex2_approx(arg.x), ex2_approx(arg.y)), one);
  const float2 s = make_float2(rcp_approx(den.x), rcp_approx(den.y));
  float2 w = mul2(xc, fma2(s, minus, one));
  if constexpr (ACT != GATE_SWIGLU) w = mul2(w, dy);
  slope = mul2(s, add2(w, one));
  return mul2(x, s);
}
template <int ACT>
__device__ __forceinline__ float gate_f(float x, float& slope) {
  float2 sl;
  const float2 a = gate2<ACT>(make_float2(x, x), sl);
  slope = sl.x;
  return a.x;
}

// Item i of a pair: its tile (and K split): units u = pair, pair + pairs, ... of tiles·splits,
// split-major, so that pairs that run together share operand panels in L2.
struct PairItem {
  int ta, tb, split, kb0, kb1;
};
__device__ __forceinline__ bool pair_item(const KParams& p, int cl, int ncl, int i, PairItem& it) {
  if (i >= p.dp_q + (cl < p.dp_r ? 1 : 0)) return false;
  int u = cl + i * ncl;
  it.split = 0;
  it.kb0 = 0;
  it.kb1 = p.num_kb;
  if (p.split_k > 1) {
    const int tiles = p.tiles_a * p.tiles_b;
    it.split = u / tiles;
    u -= it.split * tiles;
    it.kb0 = (int)((long long)p.num_kb * it.split / p.split_k);
    it.kb1 = (int)((long long)p.num_kb * (it.split + 1) / p.split_k);
  }
  tile_coords(u, p, it.ta, it.tb);
  return true;
}

// A block of 32 rows x 32 columns in shared memory as TMA lays it out: lane = row; 16-bit types
// 64 bytes a row with the 64-byte swizzle, fp32 128 bytes a row with the 128-byte swizzle.
__device__ __forceinline__ uint32_t blk16_addr(uint32_t base, int lane, int c) {
  return base + (uint32_t)lane * 64u + (uint32_t)((c ^ ((lane >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t blk32_addr(uint32_t base, int lane, int c) {
  return base + (uint32_t)lane * 128u + (uint32_t)((c ^ (lane & 7)) << 4);
}
__device__ __forceinline__ void st_shared_u4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// this lane's 32 values into a block, in OUT type
template <int OUT>
__device__ __forceinline__ void put_block(uint32_t base, int lane, const float (&v)[32]) {
  if constexpr (OUT == DT_F32) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared_u4(blk32_addr(base, lane, c), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                   __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      st_shared_u4(blk16_addr(base, lane, c), pack2<OUT>(v[8 * c], v[8 * c + 1]), pack2<OUT>(v[8 * c + 2], v[8 * c + 3]),
                   pack2<OUT>(v[8 * c + 4], v[8 * c + 5]), pack2<OUT>(v[8 * c + 6], v[8 * c + 7]));
  }
}
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (DT == DT_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// v += this lane's 32 values of a block
template <int OUT>
__device__ __forceinline__ void add_block(float (&v)[32], uint32_t base, int lane) {
#pragma unroll
  for (int c = 0; c < (OUT == DT_F32 ? 8 : 4); ++c) {
    const uint4 x = ld_shared_u4(OUT == DT_F32 ? blk32_addr(base, lane, c) : blk16_addr(base, lane, c));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (OUT == DT_F32) {
        v[4 * c + e] += __uint_as_float(w[e]);
      } else {
        const float2 f = unpack2<OUT>(w[e]);
        v[8 * c + 2 * e] += f.x, v[8 * c + 2 * e + 1] += f.y;
      }
    }
  }
}
__device__ __forceinline__ float load_dt(const void* p, long long i, int dt) {
  if (dt == DT_F32) return reinterpret_cast<const float*>(p)[i];
  if (dt == DT_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(reinterpret_cast<const __half*>(p)[i]);
}
// v += 32 elements of a row of type dt from column n0 (none past N), by plain (coherent) loads, since the
// output may be the same buffer
__device__ __forceinline__ void add_res32(float (&v)[32], const void* base, long long row_off, int n0, int N, int dt) {
  if (n0 + 32 <= N && dt == DT_F32) {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + row_off + n0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 f = q[i];
      v[4 * i] += f.x, v[4 * i + 1] += f.y, v[4 * i + 2] += f.z, v[4 * i + 3] += f.w;
    }
  } else if (n0 + 32 <= N) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + row_off + n0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = q[i];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = dt == DT_BF16 ? unpack2<DT_BF16>(w[e]) : unpack2<DT_F16>(w[e]);
        v[8 * i + 2 * e] += f.x, v[8 * i + 2 * e + 1] += f.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (n0 + j < N) v[j] += load_dt(base, row_off + n0 + j, dt);
  }
}

// Tensor maps: tmA, tmB operands (GLU: tmB gate rows, tmB2 up rows).  tm0..tm3 the epilogue's:
//   GLU      tm0 h            GLU_AUX  tm0 h, tm1 g, tm2 u
//   DGLU     tm0 g, tm1 u (loads), tm2 dg, tm3 du        GRAD, *_PART  tm0 y (or the workspace),
//            RUNS as GRAD; GRAD_ADD, RUNS_ADD as GRAD, tm1 the residual
// p.M is the number of output rows, p.N its columns; columns from p.n_tma on (a ragged end below 16
// bytes) are stored one by one.  In a workspace p.N is the padded width of one partial result (of g,
// which u follows, for GLU_PART), and p.split_rows ≥ p.M the rows of one split, a multiple of 32.
template <int EPI, int ACT, int OUT, int ATOMS>
__global__ void __launch_bounds__(kPairThreads, 1)
    fl_pair_tcgen05(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tm0,
                    const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                    const __grid_constant__ CUtensorMap tm3, const __grid_constant__ KParams p) {
  constexpr bool GLU = pair_glu(EPI);
  constexpr bool A_MN = pair_a_mn(EPI), B_MN = pair_b_mn(EPI);
  constexpr bool SUMS = EPI == EPI_RUNS || EPI == EPI_RUNS_ADD;
  constexpr int RUN = pair_run(OUT) / (ATOMS * kPairBk);  // stages of a run
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int NS = p.num_stages;
  const uint32_t bars = smem_base + p.bar_off;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (NS + s); };
  auto tfull_bar = [&](int b) { return bars + 8u * (2 * NS + b); };
  auto tempty_bar = [&](int b) { return bars + 8u * (2 * NS + 2 + b); };
  const uint32_t drain_bar = bars + 8u * (2 * NS + 4);
  const uint32_t tmem_slot = bars + 8u * (2 * NS + 5);
  // arrival of what a block of an epilogue warp works on: DGLU g and u, GRAD_ADD and RUNS_ADD the residual
  auto aux_bar = [&](int w, int b) { return bars + 8u * (2 * NS + 6 + 2 * w + b); };

  const uint32_t rank = cluster_ctarank();
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;

  if (warp == 0) {
    const int nbars = 2 * NS + 6 + (EPI == EPI_DGLU || EPI == EPI_GRAD_ADD || EPI == EPI_RUNS_ADD ? 16 : 0);
    for (int i = lane; i < nbars; i += 32) {
      const int j = i - 2 * NS;
      // (j = 5 is the place of the TMEM address; both CTAs' epilogue warps arrive on the two before the drain's)
      if (j != 5) mbar_init(bars + 8u * i, j == 2 || j == 3 ? 16 : 1);
    }
    fence_mbarrier_init();
    if (lane == 0) {
      if (p.num_kb > 0) {  // with K = 0 the operand maps are left unencoded and never used
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        if (GLU) prefetch_tensormap(&tmB2);
      }
      prefetch_tensormap(&tm0);
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, p.tmem_cols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(__cvta_shared_to_generic(tmem_slot));

  if (warp == 0) {
    // ================================================================ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      StageRing rs;
      bool ok = true;
      PairItem itm;
      for (int ii = 0; ok && pair_item(p, cluster_id, num_clusters, ii, itm); ++ii) {
        const int a_row = itm.ta * 256 + (int)rank * 128;
        const int b_row = GLU ? itm.tb * p.out_tile_n : itm.tb * p.mma_n + (int)rank * (p.mma_n / 2);
        const CUtensorMap* mb = (GLU && rank != 0) ? &tmB2 : &tmB;
        for (int kb = itm.kb0; kb < itm.kb1; ++kb, ++it, rs.next((uint32_t)NS)) {
          const int s = (int)rs.s;
          if (!wait_bounded(empty_bar(s), rs.ph ^ 1u, p)) { ok = false; break; }
          const uint32_t sa = smem_base + (uint32_t)s * p.stage_stride;
          const uint32_t sb = sa + ATOMS * kPairABytes;
          const uint32_t fb = mapa_shared(full_bar(s), 0);  // both CTAs' bytes complete on the leader's barrier
          if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2u * p.stage_bytes);
          const int k0 = kb * ATOMS * kPairBk;
          // (MN-major boxes span the stage's depth, K-major ones an atom)
          if constexpr (A_MN) {
            tma_load_2d_pair(sa, &tmA, fb, a_row, k0);
            tma_load_2d_pair(sa + ATOMS * kPairBox, &tmA, fb, a_row + 64, k0);
          } else {
#pragma unroll
            for (int a = 0; a < ATOMS; ++a) tma_load_2d_pair(sa + a * kPairABytes, &tmA, fb, k0 + a * kPairBk, a_row);
          }
          if constexpr (B_MN) {
            for (int i = 0; i < p.b_boxes; ++i)
              tma_load_2d_pair(sb + (uint32_t)i * ATOMS * kPairBox, mb, fb, b_row + 64 * i, k0);
          } else {
#pragma unroll
            for (int a = 0; a < ATOMS; ++a)
              tma_load_2d_pair(sb + (uint32_t)a * p.b_atom_bytes, mb, fb, k0 + a * kPairBk, b_row);
          }
        }
      }
      // Never leave with copies in flight: the leader waits (bounded) for the last fill of every
      // stage; the final cluster barrier keeps the peer resident until then.
      for (uint32_t s = 0; rank == 0 && s < (uint32_t)NS && s < it; ++s) {
        const uint32_t last = it - 1u - ((it - 1u - s) % (uint32_t)NS);
        (void)wait_bounded(full_bar((int)s), (last / (uint32_t)NS) & 1u, p);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================================================================ UMMA issuer (rank 0 for both CTAs)
    if (lane == 0 && rank == 0) {
      const uint64_t da0 = sdesc_sw128(smem_base, A_MN ? ATOMS * kPairBox : 16u, 1024);
      const uint64_t db0 = sdesc_sw128(smem_base + ATOMS * kPairABytes, B_MN ? ATOMS * kPairBox : 16u, 1024);
      const uint64_t stage_step = p.stage_stride >> 4;
      // a UMMA step is 16 deep: 32 bytes along a K-major row of an atom, 16 K rows of 128 bytes in an
      // MN-major box (start-address offsets in 16-byte units)
      constexpr int STEPS = ATOMS * kPairBk / 16;
      uint32_t ao[STEPS], bo[STEPS];
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        ao[k] = A_MN ? k * 128u : (k >> 2) * (kPairABytes >> 4) + (k & 3) * 2u;
        bo[k] = B_MN ? k * 128u : (k >> 2) * (p.b_atom_bytes >> 4) + (k & 3) * 2u;
      }
      const uint32_t idesc = p.idesc;
      uint32_t n = 0;  // accumulators handed over
      StageRing rs;
      bool ok = true, issued = false;
      PairItem itm;
      for (int ii = 0; ok && pair_item(p, cluster_id, num_clusters, ii, itm); ++ii) {
        int kb = itm.kb0;
        do {
          const int first = kb, end = SUMS ? min(itm.kb1, kb + RUN) : itm.kb1;
          const uint32_t buf = n & 1u;
          if (!wait_bounded(tempty_bar(buf), ((n >> 1) & 1u) ^ 1u, p, true)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + buf * (uint32_t)p.mma_n;
          for (; kb < end; ++kb, rs.next((uint32_t)NS)) {
            const int s = (int)rs.s;
            if (!wait_bounded(full_bar(s), rs.ph, p)) { ok = false; break; }
            tc_fence_after();
            const uint64_t da = da0 + (uint64_t)s * stage_step;
            const uint64_t db = db0 + (uint64_t)s * stage_step;
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
              umma_f16_pair(d_tmem, da + ao[k], db + bo[k], idesc, (kb > first || k > 0) ? 1u : 0u);
            umma_commit_pair_both(empty_bar(s));
            issued = true;
          }
          if (!ok) break;
          if (end > first) {
            umma_commit_pair_both(tfull_bar(buf));
          } else {
            mbar_arrive(tfull_bar(buf));
            mbar_arrive_remote(mapa_shared(tfull_bar(buf), 1));
          }
          ++n;
        } while (kb < itm.kb1);
      }
      if (issued) {  // no MMA may still be running when TMEM is released
        umma_commit_pair(drain_bar);
        (void)wait_bounded(drain_bar, 0, p);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int ew = warp - kEpiWarp0;
    const int half_cols = p.out_tile_n >> 1;
    const int c_begin = (ew >> 2) * half_cols;
    const int nblk = half_cols / 32;
    const uint32_t stg = smem_base + p.staging_off + (uint32_t)ew * pair_warp_staging(ATOMS);
    uint32_t local = 0;
    // Blocks leave through SLOTS block buffers in turn: `emit` waits until the store that used the
    // next one has read it, then fills and stores it.
    constexpr int SLOTS = (int)(pair_warp_staging(ATOMS) / pair_block_bytes(OUT));
    uint32_t slot_at = 0;
    auto emit = [&](const CUtensorMap* map, int x, int y, bool inside, int own, const float (&v)[32]) {
      if (lane == 0) bulk_wait_group_read<SLOTS - 1>();
      __syncwarp();
      const uint32_t at = stg + slot_at * pair_block_bytes(OUT);
      put_block<OUT>(at, own, v);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (inside) tma_store_2d(map, at, x, y);
        bulk_commit_group();
      }
      slot_at = slot_at + 1 == (uint32_t)SLOTS ? 0u : slot_at + 1;
    };
    // ragged row end: a TMA store writes whole 16-byte granules
    auto store_ragged = [&](int n0, int m, bool m_ok, const float (&v)[32]) {
      if (n0 + 32 > p.n_tma && n0 < p.N && m_ok) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (n0 + j >= p.n_tma && n0 + j < p.N) store_elem<OUT>(p.out, (long long)m * p.ldo + n0 + j, v[j]);
      }
    };
    uint32_t blk = 0;  // blocks this warp has begun (DGLU: the g, u tiles alternate between two buffers)
    bool ok = true;
    PairItem itm;
    // DGLU: g, u tiles arrive in, and dg, du leave from, GU pairs of buffers in turn; lane 0 sends for
    // those of block b of an item into pair `to`.  GRAD_ADD, the form of GRAD for a residual of the output's
    // type: the same, GU buffers.  (Read by the lanes, a row each, which is 32 lines an
    // instruction, the residual took longer than the products: 8191 x 1999 fp32 of 777 tokens 47.7 us, 33.5 so;
    // 768 x 768 of 256 8.6 and 6.8.)
    // RUNS_ADD takes the whole tile's residual into its sums at the tile's start, during the first run.
    constexpr bool IN_PLACE = EPI == EPI_DGLU || EPI == EPI_GRAD_ADD || EPI == EPI_RUNS_ADD;
    constexpr uint32_t GU_BYTES = EPI == EPI_GRAD_ADD || EPI == EPI_RUNS_ADD ? pair_block_bytes(OUT) : 4096u;
    constexpr uint32_t GU = EPI == EPI_RUNS_ADD || pair_warp_staging(ATOMS) / GU_BYTES < 2u ? 1u : 2u;
    auto fetch_gu = [&](const PairItem& w, int b, uint32_t to) {
      const int n0 = w.tb * p.out_tile_n + c_begin + 32 * b, r0 = w.ta * 256 + (int)rank * 128 + q * 32;
      mbar_arrive_expect_tx(aux_bar(ew, (int)to), GU_BYTES);
      if constexpr (EPI == EPI_DGLU) {
        tma_load_2d(stg + to * 4096u, &tm0, aux_bar(ew, (int)to), n0, r0);
        tma_load_2d(stg + to * 4096u + 2048u, &tm1, aux_bar(ew, (int)to), n0, r0);
      } else {
        tma_load_2d(stg + to * GU_BYTES, &tm1, aux_bar(ew, (int)to), n0, r0);
      }
    };
    uint32_t fetched = 0;  // blocks whose tiles have been sent for
    bool more = pair_item(p, cluster_id, num_clusters, 0, itm);
    if constexpr (IN_PLACE) {
      if (more) {
        if (lane == 0) fetch_gu(itm, 0, 0);
        fetched = 1;  // (the others follow, GU − 1 blocks ahead of their use)
      }
    }
    uint32_t n = 0;  // accumulators taken over
    // this warp's TMEM reads of an accumulator are done: hand its share back to the leader
    auto hand_back = [&](uint32_t buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank != 0) mbar_arrive_remote(mapa_shared(tempty_bar(buf), 0));
        else mbar_arrive(tempty_bar(buf));
      }
    };
    while (more) {
      PairItem nxt;
      bool have_next = false;
      if constexpr (!SUMS) have_next = pair_item(p, cluster_id, num_clusters, (int)local + 1, nxt);
      const bool acc_any = itm.kb1 > itm.kb0;
      const int row0 = itm.ta * 256 + (int)rank * 128 + q * 32;
      const int m = row0 + lane;
      const bool m_ok = m < p.M;
      const int n_tile0 = itm.tb * p.out_tile_n;
      // block b + 1 of the item, or the next item's first, once the other buffer's stores, or this one's,
      // have read it
      auto fetch_next = [&](int b) {
        const bool last = b + 1 == nblk;
        if (!last || have_next) {
          if (lane == 0) {
            bulk_wait_group_read<0>();
            if (last) fetch_gu(nxt, 0, (blk + 1) % GU);
            else fetch_gu(itm, b + 1, (blk + 1) % GU);
          }
          ++fetched;
        }
      };
      // block b of a result y = (v + residual)·scale; false: a wait gave up
      auto grad_block = [&](int b, float (&v)[32]) {
        const int n0 = n_tile0 + c_begin + 32 * b;
        const bool inside = n0 < p.n_tma && (p.split_rows == 0 || row0 < p.split_rows);
        const int row = itm.split * p.split_rows + row0;
        const uint32_t at = stg + (blk % GU) * GU_BYTES;
        int own = lane;  // (hidden from the compiler, which would keep the blocks' addresses in registers)
        if constexpr (SUMS) asm volatile("" : "+r"(own));
        if constexpr (EPI == EPI_GRAD_ADD) {
          if constexpr (GU > 1) fetch_next(b);
          if (!warp_wait_bounded(aux_bar(ew, (int)(blk % GU)), (blk / GU) & 1u, p, lane)) return false;
          add_block<OUT>(v, at, own);
        }
        if ((EPI == EPI_GRAD || EPI == EPI_RUNS) && p.residual != nullptr && m_ok && n0 < p.N)
          add_res32(v, p.residual, (long long)m * p.ldr, n0, p.N, p.res_dtype);
        if (p.scale != 1.0f) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= p.scale;
        }
        store_ragged(n0, m, m_ok, v);
        if constexpr (EPI == EPI_GRAD_ADD) {
          put_block<OUT>(at, own, v);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (inside) tma_store_2d(&tm0, at, n0, row);
            bulk_commit_group();
          }
          if constexpr (GU == 1) fetch_next(b);
        } else {
          emit(&tm0, n0, row, inside, own, v);
        }
        if constexpr (!SUMS) ++blk;
        return true;
      };
      if constexpr (SUMS) {
        float sum[4][32];  // (a tile has two or four blocks a warp)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[b][j] = 0.0f;
        if constexpr (EPI == EPI_RUNS_ADD) {
          static_assert(GU == 1, "one buffer: a block is fetched when the one before it has been read");
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (b >= nblk) break;
            if (!warp_wait_bounded(aux_bar(ew, 0), blk & 1u, p, lane)) { ok = false; break; }
            add_block<OUT>(sum[b], stg, lane);
            __syncwarp();
            ++blk;
            if (b + 1 < nblk) fetch_next(b);
          }
          if (!ok) break;
        }
        int kb = itm.kb0;
        do {
          const uint32_t buf = n & 1u;
          if (!warp_wait_bounded(tfull_bar(buf), (n >> 1) & 1u, p, lane, true)) { ok = false; break; }
          tc_fence_after();
          const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + buf * (uint32_t)p.mma_n + (uint32_t)c_begin;
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            if (b >= 2 * nblk || !acc_any) break;
            uint32_t g[16];
            tmem_ld16(tacc + 16u * b, g);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[b >> 1][16 * (b & 1) + j] += __uint_as_float(g[j]);
          }
          hand_back(buf);
          ++n;
          kb += RUN;
        } while (kb < itm.kb1);
        if (!ok) break;
        have_next = pair_item(p, cluster_id, num_clusters, (int)local + 1, nxt);  // (now, for want of registers)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (b >= nblk) break;
          if (!grad_block(b, sum[b])) { ok = false; break; }
        }
        if (!ok) break;
        if constexpr (EPI == EPI_RUNS_ADD) fetch_next(nblk - 1);
        ++local;
        itm = nxt;
        more = have_next;
        continue;
      }
      const uint32_t buf = n & 1u;
      if (!warp_wait_bounded(tfull_bar(buf), (n >> 1) & 1u, p, lane, true)) { ok = false; break; }
      tc_fence_after();
      const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + buf * (uint32_t)p.mma_n;
#pragma unroll 1
      for (int b = 0; b < nblk; ++b) {
        const int cb = c_begin + 32 * b;
        const int n0 = n_tile0 + cb;
        uint32_t ga[32], gu[32];
        if (acc_any) {
          tmem_ld32(tacc + (uint32_t)cb, ga);
          if constexpr (GLU) tmem_ld32(tacc + (uint32_t)(p.out_tile_n + cb), gu);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ga[j] = gu[j] = 0u;
        }
        if constexpr (EPI == EPI_DGLU) {
          const uint32_t slot = blk % GU;
          const uint32_t sg = stg + slot * 4096u, su = sg + 2048u;
          if constexpr (GU > 1) fetch_next(b);
          if (acc_any) tmem_wait_ld();
          if (!warp_wait_bounded(aux_bar(ew, (int)slot), (blk / GU) & 1u, p, lane)) { ok = false; break; }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t ag = blk16_addr(sg, lane, c), au = blk16_addr(su, lane, c);
            const uint4 g4 = ld_shared_u4(ag), u4 = ld_shared_u4(au);
            const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
            uint32_t dg[4], du[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 g = unpack2<OUT>(gw[e]), u = unpack2<OUT>(uw[e]);
              const float2 dh = make_float2(__uint_as_float(ga[8 * c + 2 * e]), __uint_as_float(ga[8 * c + 2 * e + 1]));
              float2 slope;
              const float2 b2 = mul2(dh, gate2<ACT>(g, slope)), a2 = mul2(mul2(dh, u), slope);
              dg[e] = pack2<OUT>(a2.x, a2.y);
              du[e] = pack2<OUT>(b2.x, b2.y);
            }
            st_shared_u4(ag, dg[0], dg[1], dg[2], dg[3]);
            st_shared_u4(au, du[0], du[1], du[2], du[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (n0 < p.N) {
              tma_store_2d(&tm2, sg, n0, row0);
              tma_store_2d(&tm3, su, n0, row0);
            }
            bulk_commit_group();
          }
          if constexpr (GU == 1) fetch_next(b);
          ++blk;
        } else {
          if (acc_any) tmem_wait_ld();
          float v[32];
          if constexpr (pair_a_mn(EPI) || EPI == EPI_DGLU_PART) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(ga[j]);
            if (!grad_block(b, v)) { ok = false; break; }
          } else {
            const bool inside = n0 < p.n_tma && (p.split_rows == 0 || row0 < p.split_rows);
            const int row = itm.split * p.split_rows + row0;
            if constexpr (EPI == EPI_GLU_AUX || EPI == EPI_GLU_PART) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(ga[j]);
              emit(EPI == EPI_GLU_AUX ? &tm1 : &tm0, n0, row, inside, lane, v);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(gu[j]);
              if constexpr (EPI == EPI_GLU_AUX) emit(&tm2, n0, row, inside, lane, v);
              else emit(&tm0, p.N + n0, row, inside, lane, v);
            }
            if constexpr (EPI == EPI_GLU || EPI == EPI_GLU_AUX) {
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                float2 slope;
                const float2 g = make_float2(__uint_as_float(ga[j]), __uint_as_float(ga[j + 1]));
                const float2 h = mul2(gate2<ACT>(g, slope), make_float2(__uint_as_float(gu[j]), __uint_as_float(gu[j + 1])));
                v[j] = h.x;
                v[j + 1] = h.y;
              }
              if constexpr (EPI == EPI_GLU) store_ragged(n0, m, m_ok, v);
              emit(&tm0, n0, row, inside, lane, v);
            }
          }
        }
      }
      if (!ok) break;
      hand_back(buf);
      ++n;
      ++local;
      itm = nxt;
      more = have_next;
    }
    if constexpr (IN_PLACE) {
      // after a wait that gave up: no tile may still be on its way when the CTA leaves
      for (uint32_t f = blk; f < fetched; ++f) (void)warp_wait_bounded(aux_bar(ew, (int)(f % GU)), (f / GU) & 1u, p, lane);
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  // ================================================================ teardown
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, p.tmem_cols);
  }
}

// ---------------------------------------------------------------- after K splits
// Σ_s ws[s] of four columns, in split order; the loads of eight splits are in flight together.
__device__ __forceinline__ float4 sum_splits(const float* w, long long split_stride, int splits) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < splits; s0 += 8) {
    float4 t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      t[k] = s0 + k < splits ? __ldcg(reinterpret_cast<const float4*>(w + (long long)(s0 + k) * split_stride))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) a.x += t[k].x, a.y += t[k].y, a.z += t[k].z, a.w += t[k].w;
  }
  return a;
}
// four columns at element i (a multiple of four of a row that starts on 16 bytes), cnt of them inside
__device__ __forceinline__ void load4_dt(float (&v)[4], const void* p, long long i, int dt, int cnt) {
  if (cnt == 4 && dt == DT_F32) {
    const float4 q = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else if (cnt == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + i);
    const float2 a = dt == DT_BF16 ? unpack2<DT_BF16>(q.x) : unpack2<DT_F16>(q.x);
    const float2 b = dt == DT_BF16 ? unpack2<DT_BF16>(q.y) : unpack2<DT_F16>(q.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < cnt ? load_dt(p, i + j, dt) : 0.0f;
  }
}
__device__ __forceinline__ void store4_dt(void* p, long long i, int dt, int cnt, const float (&v)[4]) {
  if (cnt == 4 && dt == DT_F32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (cnt == 4) {
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) =
        dt == DT_BF16 ? make_uint2(pack2<DT_BF16>(v[0], v[1]), pack2<DT_BF16>(v[2], v[3]))
                      : make_uint2(pack2<DT_F16>(v[0], v[1]), pack2<DT_F16>(v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= cnt) break;
      if (dt == DT_F32) store_elem<DT_F32>(p, i + j, v[j]);
      else if (dt == DT_BF16) store_elem<DT_BF16>(p, i + j, v[j]);
      else store_elem<DT_F16>(p, i + j, v[j]);
    }
  }
}

struct FinishArgs {
  const float* ws;
  long long split_stride, ld_ws, half;  // half: column of u in a row of the workspace
  int splits;
  const void* residual;  // GRAD
  long long ldr;
  int res_dtype;
  void* out;
  long long ldo;
  int out_dtype;
  void* aux;  // [M, 2N] of out_dtype: written by GLU_AUX, read by DGLU
  long long M;
  int N, nvec;
  float scale;
};

// The epilogue of a result in K splits; a thread takes four columns of a row.
//   GRAD  y = (Σ + residual)·scale     GLU  h = act(Σg)·Σu, and g, u to aux when it is given
//   DGLU  out = [Σ·u·act'(g), Σ·act(g)] with g, u from aux (out may be aux's own buffer)
template <int EPI, int ACT>
__global__ void __launch_bounds__(256) fl_split_finish_kernel(const FinishArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const long long total = P.M * P.nvec;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const long long m = i / P.nvec;
    const int n0 = 4 * (int)(i - m * P.nvec);
    const int cnt = min(4, P.N - n0);
    const float* w = P.ws + m * P.ld_ws + n0;
    const float4 a = sum_splits(w, P.split_stride, P.splits);
    float v[4] = {a.x, a.y, a.z, a.w};
    if constexpr (EPI == EPI_GRAD) {
      if (P.residual != nullptr) {
        float r[4];
        load4_dt(r, P.residual, m * P.ldr + n0, P.res_dtype, cnt);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= P.scale;
      store4_dt(P.out, m * P.ldo + n0, P.out_dtype, cnt, v);
    } else if constexpr (EPI == EPI_GLU) {
      const float4 b = sum_splits(w + P.half, P.split_stride, P.splits);
      const float u[4] = {b.x, b.y, b.z, b.w};
      if (P.aux != nullptr) {
        store4_dt(P.aux, m * 2 * P.N + n0, P.out_dtype, cnt, v);
        store4_dt(P.aux, m * 2 * P.N + P.N + n0, P.out_dtype, cnt, u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float slope;
        v[j] = gate_f<ACT>(v[j], slope) * u[j];
      }
      store4_dt(P.out, m * P.ldo + n0, P.out_dtype, cnt, v);
    } else {
      float g[4], u[4], dg[4];
      load4_dt(g, P.aux, m * 2 * P.N + n0, P.out_dtype, cnt);
      load4_dt(u, P.aux, m * 2 * P.N + P.N + n0, P.out_dtype, cnt);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float slope;
        const float act = gate_f<ACT>(g[j], slope);
        dg[j] = v[j] * u[j] * slope;
        v[j] *= act;
      }
      store4_dt(P.out, m * P.ldo + n0, P.out_dtype, cnt, dg);
      store4_dt(P.out, m * P.ldo + P.N + n0, P.out_dtype, cnt, v);
    }
  }
}

}  // namespace fl
