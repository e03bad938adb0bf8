// fl_rows.cuh — HBM-bound row kernels of a sublayer's end, in training:
//
//   * fl_dropout_kernel:      y = residual + D(x)
//   * fl_dropout_ln_kernel:   s = residual + D(x), z = (s − μ)·rstd·γ + β, with s, μ and rstd kept
//   * fl_dropout_ln_bwd_kernel, fl_ln_wgrad_kernel: the gradients of s, x, γ and β
//
// D(x)[m,n] = x[m,n]/(1 − p) where the element is kept, else 0.  The decision is a function of
// the element's place alone, so the backward pass draws it again and no mask is stored.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fl_gemm.cuh"

namespace fl {

// ---------------------------------------------------------------- random numbers
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011): four 32-bit words from a 128-bit counter and a 64-bit key in ten rounds.  The
// counter is (block, offset), the key the seed; block = m·⌈N/4⌉ + n/4 and word n mod 4 belong to
// element (m, n), so that the numbers depend on the logical shape only, never on pitches,
// alignment or the launch.
struct DropParams {
  uint32_t k0, k1;             // key: the seed's halves
  uint64_t offset;             // upper counter half
  const uint64_t* offset_dev;  // added to offset when not null (read on the device)
  uint32_t threshold;          // dropped where the word is below ⌊p·2^32⌋
  float scale;                 // 1/(1 − p)
  int on;                      // 0: p = 0, nothing is drawn
};

__device__ __forceinline__ uint4 philox4x32_10(uint64_t block, uint64_t offset, uint32_t k0, uint32_t k1) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// v[i] = D(v)[i] for the eight elements of blocks `block` and `block` + 1
__device__ __forceinline__ void drop8(float (&v)[8], uint64_t block, uint64_t offset, const DropParams& d) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 r = philox4x32_10(block + h, offset, d.k0, d.k1);
    v[4 * h + 0] = r.x >= d.threshold ? v[4 * h + 0] * d.scale : 0.0f;
    v[4 * h + 1] = r.y >= d.threshold ? v[4 * h + 1] * d.scale : 0.0f;
    v[4 * h + 2] = r.z >= d.threshold ? v[4 * h + 2] * d.scale : 0.0f;
    v[4 * h + 3] = r.w >= d.threshold ? v[4 * h + 3] * d.scale : 0.0f;
  }
}

__device__ __forceinline__ uint64_t drop_offset(const DropParams& d) {
  return d.on && d.offset_dev != nullptr ? d.offset + *d.offset_dev : d.offset;
}

// ---------------------------------------------------------------- eight elements of a row
// A matrix operand: null, or [M, ld] of dtype dt.  All accesses are plain (coherent) loads and
// stores, because an output may be an input's own buffer.
struct Mat {
  void* p;
  long long ld;
  int dt;
};

struct Raw8 {
  uint4 a, b;  // 16-bit types: a; fp32: a and b
};

__device__ __forceinline__ Raw8 load_raw8(const Mat& t, long long row, int c0) {
  Raw8 r;
  if (t.dt == DT_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(t.p) + row * t.ld + c0);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(t.p) + row * t.ld + c0);
    r.b = make_uint4(0u, 0u, 0u, 0u);
  }
  return r;
}
__device__ __forceinline__ void widen8(float (&v)[8], const Raw8& r, int dt) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (dt == DT_F32) {
    const uint32_t x[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]), v[4 + i] = __uint_as_float(x[i]);
  } else if (dt == DT_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ float load1(const void* p, long long i, int dt) {
  if (dt == DT_F32) return reinterpret_cast<const float*>(p)[i];
  const uint16_t h = reinterpret_cast<const uint16_t*>(p)[i];
  return dt == DT_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}
__device__ __forceinline__ void store1(void* p, long long i, int dt, float v) {
  if (dt == DT_F32) reinterpret_cast<float*>(p)[i] = v;
  else if (dt == DT_BF16) reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}
// elements c0 .. c0 + cnt − 1 of a row one by one, zeros after them
__device__ __forceinline__ void load_some8(float (&v)[8], const Mat& t, long long row, int c0, int cnt) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < cnt ? load1(t.p, row * t.ld + c0 + i, t.dt) : 0.0f;
}
__device__ __forceinline__ void store8(const Mat& t, long long row, int c0, int cnt, bool vec, const float (&v)[8]) {
  if (vec) {
    if (t.dt == DT_F32) {
      float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(t.p) + row * t.ld + c0);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint4 q;
      if (t.dt == DT_BF16) {
        q = make_uint4(pack2<DT_BF16>(v[0], v[1]), pack2<DT_BF16>(v[2], v[3]), pack2<DT_BF16>(v[4], v[5]),
                       pack2<DT_BF16>(v[6], v[7]));
      } else {
        q = make_uint4(pack2<DT_F16>(v[0], v[1]), pack2<DT_F16>(v[2], v[3]), pack2<DT_F16>(v[4], v[5]),
                       pack2<DT_F16>(v[6], v[7]));
      }
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(t.p) + row * t.ld + c0) = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) store1(t.p, row * t.ld + c0 + i, t.dt, v[i]);
  }
}
// eight parameters of type dt from c0; `dflt` for a null pointer
__device__ __forceinline__ void load_param8(float (&v)[8], const void* p, int dt, int c0, int cnt, bool vec, float dflt) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = dflt;
  } else {
    const Mat t{const_cast<void*>(p), 0, dt};
    if (vec) widen8(v, load_raw8(t, 0, c0), dt);
    else load_some8(v, t, 0, c0, cnt);
  }
}

// ---------------------------------------------------------------- dropout
struct DropoutArgs {
  Mat x, r, y;  // r.p null: no residual
  long long M;
  int N, nvec, vec;  // nvec = ⌈N/8⌉ vectors a row; vec: every row of every operand is 16-byte aligned
  DropParams d;
};

// Thread i of the grid takes vectors i, i + threads, ... of the M·nvec (row, vector) pairs; row
// and vector advance by the stride's quotient and remainder, so that one division runs per
// thread.  Two vectors a trip: both vectors' loads are in flight before the first use.
__global__ void __launch_bounds__(256) fl_dropout_kernel(const DropoutArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long i0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long srow = stride / P.nvec;
  const int svec = (int)(stride - srow * P.nvec);
  long long row = i0 / P.nvec;
  int v = (int)(i0 - row * P.nvec);
  const uint64_t offset = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  while (row < P.M) {
    long long rows[2];
    int c0[2], cnt[2];
    bool live[2], vec[2];
    Raw8 rx[2], rr[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      rows[u] = row;
      live[u] = row < P.M;
      c0[u] = 8 * v;
      cnt[u] = min(8, P.N - c0[u]);
      vec[u] = P.vec && cnt[u] == 8;
      if (live[u] && vec[u]) {
        rx[u] = load_raw8(P.x, row, c0[u]);
        if (P.r.p != nullptr) rr[u] = load_raw8(P.r, row, c0[u]);
      }
      row += srow;
      v += svec;
      if (v >= P.nvec) v -= P.nvec, ++row;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (!live[u]) continue;
      float x[8];
      if (vec[u]) widen8(x, rx[u], P.x.dt);
      else load_some8(x, P.x, rows[u], c0[u], cnt[u]);
      if (P.d.on) drop8(x, (uint64_t)(rows[u] * groups + (c0[u] >> 2)), offset, P.d);
      if (P.r.p != nullptr) {
        float r[8];
        if (vec[u]) widen8(r, rr[u], P.r.dt);
        else load_some8(r, P.r, rows[u], c0[u], cnt[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += r[i];
      }
      store8(P.y, rows[u], c0[u], cnt[u], vec[u], x);
    }
  }
}

// ---------------------------------------------------------------- sums over a row's threads
// Sum of (a, b) over the T threads that share a row, the same in every thread: a butterfly in
// each warp, then the warps' sums in warp order.  `red` holds two sets of T/32 pairs, used in
// turn (`flip`), so that one barrier a call is enough: a warp writes a set again only after the
// next call's barrier, which every reader of the set has passed its reads before.
template <int T>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* red, int& flip, int group) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    float2* set = red + flip * W;
    flip ^= 1;
    const int w = (threadIdx.x % T) >> 5;
    if ((threadIdx.x & 31) == 0) set[w] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(T) : "memory");
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 q = set[i];
      a += q.x;
      b += q.y;
    }
  }
  return make_float2(a, b);
}

// ---------------------------------------------------------------- rows ahead in shared memory
// A thread copies its own vectors of a row into its own slots of shared memory (cp.async, one
// group a row) `ahead` rows before it needs them, and reads back only those, so that no barrier
// stands between the copy and its use, and the bytes in flight cost no registers.  One ring slot
// holds, for each operand, V·BLOCK 16-byte pieces (16-bit types) or two such planes (fp32).  The
// ring has two slots, or one where two do not fit (fp32 rows of more than 8192 elements).
constexpr int kRowsAhead = 2;
__device__ __forceinline__ void wait_row(int ahead) {
  if (ahead == kRowsAhead) cp_async_wait<kRowsAhead - 1>();
  else cp_async_wait<0>();
}
__host__ __device__ __forceinline__ uint32_t plane_bytes(int v, int block) { return (uint32_t)v * (uint32_t)block * 16u; }
__host__ __device__ __forceinline__ uint32_t operand_bytes(const Mat& t, int v, int block) {
  return t.p == nullptr ? 0u : plane_bytes(v, block) * (t.dt == DT_F32 ? 2u : 1u);
}
template <int V, int BLOCK>
__device__ __forceinline__ void stage_vec(uint32_t dst, const Mat& t, long long row, int c0, int k) {
  const char* src = reinterpret_cast<const char*>(t.p) + (row * t.ld + c0) * (t.dt == DT_F32 ? 4 : 2);
  const uint32_t a = dst + (uint32_t)(k * BLOCK + threadIdx.x) * 16u;
  cp_async_16(a, src, 16u);
  if (t.dt == DT_F32) cp_async_16(a + plane_bytes(V, BLOCK), src + 16, 16u);
}
template <int V, int BLOCK>
__device__ __forceinline__ void unstage_vec(float (&v)[8], uint32_t src, int dt, int k) {
  const uint32_t a = src + (uint32_t)(k * BLOCK + threadIdx.x) * 16u;
  const float4 q = ld_shared_f4(a);
  Raw8 r;
  r.a = make_uint4(__float_as_uint(q.x), __float_as_uint(q.y), __float_as_uint(q.z), __float_as_uint(q.w));
  r.b = make_uint4(0u, 0u, 0u, 0u);
  if (dt == DT_F32) {
    const float4 w = ld_shared_f4(a + plane_bytes(V, BLOCK));
    r.b = make_uint4(__float_as_uint(w.x), __float_as_uint(w.y), __float_as_uint(w.z), __float_as_uint(w.w));
  }
  widen8(v, r, dt);
}

// ---------------------------------------------------------------- dropout, residual, LayerNorm
struct DropLnArgs {
  Mat x, r, s, z;  // r, s may be null
  const void *gamma, *beta;
  float *mean, *rstd;  // [M], both or neither
  long long M;
  int N, param_dt, vec;  // vec: every operand and parameter is 16-byte aligned in every row
  int ahead;             // slots of the ring
  float eps;
  DropParams d;
};

// T threads hold a row, V vectors of eight each (N ≤ 8·V·T): the row is read once, stays in
// registers through the mean, Σ(s − μ)² and the normalisation, and every output is written once.
// A CTA holds max(1, 128/T) rows at a time and walks the rows a grid apart.
template <int T, int V>
__global__ void __launch_bounds__(T < 128 ? 128 : T) fl_dropout_ln_kernel(const DropLnArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr int BLOCK = T < 128 ? 128 : T;
  constexpr int R = BLOCK / T;
  extern __shared__ __align__(16) uint8_t ring_s[];
  __shared__ float2 red_s[R][2 * (T / 32)];
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  int flip = 0;
  const uint64_t offset = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N;
  const long long m0 = (long long)blockIdx.x * R + group, step = (long long)gridDim.x * R;
  const uint32_t ring = smem_u32(ring_s);
  const uint32_t xb = operand_bytes(P.x, V, BLOCK), slot_bytes = xb + operand_bytes(P.r, V, BLOCK);
  auto prefetch = [&](long long m, uint32_t slot) {
    if (m < P.M && P.vec) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c0 = 8 * (k * T + t);
        if (c0 + 8 <= P.N) {
          stage_vec<V, BLOCK>(slot, P.x, m, c0, k);
          if (P.r.p != nullptr) stage_vec<V, BLOCK>(slot + xb, P.r, m, c0, k);
        }
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < P.ahead; ++i) prefetch(m0 + i * step, ring + i * slot_bytes);
  int at = 0;
  for (long long m = m0; m < P.M; m += step) {
    const uint32_t slot = ring + at * slot_bytes;
    float s[V][8];
    float sum = 0.0f;
    wait_row(P.ahead);  // this row's copies have landed
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * T + t);
      const int cnt = max(0, min(8, P.N - c0));
      const bool vec = P.vec && cnt == 8;
      if (vec) unstage_vec<V, BLOCK>(s[k], slot, P.x.dt, k);
      else load_some8(s[k], P.x, m, c0, cnt);
      if (cnt == 0) continue;
      if (P.d.on) drop8(s[k], (uint64_t)(m * groups + (c0 >> 2)), offset, P.d);
      if (P.r.p != nullptr) {
        float r[8];
        if (vec) unstage_vec<V, BLOCK>(r, slot + xb, P.r.dt, k);
        else load_some8(r, P.r, m, c0, cnt);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[k][i] += r[i];
      }
      if (P.s.p != nullptr) store8(P.s, m, c0, cnt, vec, s[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += i < cnt ? s[k][i] : 0.0f;
    }
    prefetch(m + P.ahead * step, slot);  // (the slot's values are in registers)
    at = at + 1 == P.ahead ? 0 : at + 1;
    const float mean = row_sum<T>(sum, 0.0f, red_s[group], flip, group).x / n_f;
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int cnt = P.N - 8 * (k * T + t);
#pragma unroll
      for (int i = 0; i < 8; ++i) q += i < cnt ? (s[k][i] - mean) * (s[k][i] - mean) : 0.0f;
    }
    const float var = row_sum<T>(q, 0.0f, red_s[group], flip, group).x / n_f;
    const float rstd = 1.0f / sqrtf(var + P.eps);
    if (t == 0 && P.mean != nullptr) P.mean[m] = mean, P.rstd[m] = rstd;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * T + t);
      const int cnt = min(8, P.N - c0);
      if (cnt <= 0) continue;
      const bool vec = P.vec && cnt == 8;
      float g[8], b[8];
      load_param8(g, P.gamma, P.param_dt, c0, cnt, vec, 1.0f);
      load_param8(b, P.beta, P.param_dt, c0, cnt, vec, 0.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = (s[k][i] - mean) * rstd * g[i] + b[i];
      store8(P.z, m, c0, cnt, vec, g);
    }
  }
  cp_async_wait<0>();  // no copy is in flight when the CTA leaves
}

// Rows longer than 16·1024 elements: a CTA of 1024 threads walks the row once for each of the
// three steps and forms s again from x, the residual and the drawn numbers each time.  s and z are
// written in the last walk, so that they may be the inputs' own buffers.
__global__ void __launch_bounds__(1024) fl_dropout_ln_long_kernel(const DropLnArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  __shared__ float2 red[2 * 32];
  int flip = 0;
  const uint64_t offset = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N;
  for (long long m = blockIdx.x; m < P.M; m += gridDim.x) {
    auto value = [&](int c0, int cnt, bool vec, float (&s)[8]) {
      if (vec) widen8(s, load_raw8(P.x, m, c0), P.x.dt);
      else load_some8(s, P.x, m, c0, cnt);
      if (P.d.on) drop8(s, (uint64_t)(m * groups + (c0 >> 2)), offset, P.d);
      if (P.r.p != nullptr) {
        float r[8];
        if (vec) widen8(r, load_raw8(P.r, m, c0), P.r.dt);
        else load_some8(r, P.r, m, c0, cnt);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += r[i];
      }
    };
    float mean = 0.0f, rstd = 0.0f;
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      float acc = 0.0f;
      for (long long c = 8LL * threadIdx.x; c < P.N; c += 8 * 1024) {
        const int c0 = (int)c, cnt = min(8, P.N - c0);
        const bool vec = P.vec && cnt == 8;
        float s[8];
        value(c0, cnt, vec, s);
        if (step < 2) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float d = s[i] - mean;
            acc += i < cnt ? (step == 0 ? s[i] : d * d) : 0.0f;
          }
        } else {
          float g[8], b[8];
          load_param8(g, P.gamma, P.param_dt, c0, cnt, vec, 1.0f);
          load_param8(b, P.beta, P.param_dt, c0, cnt, vec, 0.0f);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = (s[i] - mean) * rstd * g[i] + b[i];
          if (P.s.p != nullptr) store8(P.s, m, c0, cnt, vec, s);
          store8(P.z, m, c0, cnt, vec, g);
        }
      }
      if (step == 0) mean = row_sum<1024>(acc, 0.0f, red, flip, 0).x / n_f;
      if (step == 1) rstd = 1.0f / sqrtf(row_sum<1024>(acc, 0.0f, red, flip, 0).x / n_f + P.eps);
    }
    if (threadIdx.x == 0 && P.mean != nullptr) P.mean[m] = mean, P.rstd[m] = rstd;
  }
}

// ---------------------------------------------------------------- its backward pass
struct DropLnBwdArgs {
  Mat dz, ds_in, s, dres, dx;  // ds_in, dres, dx may be null
  const float *mean, *rstd;
  const void* gamma;
  float* ws;  // [gridDim.x][2][ws_ld] fp32 column partial sums of dγ and dβ, or null
  long long M;
  int N, ws_ld, param_dt, vec, ahead;
  DropParams d;
};

// With u = (s − μ)·rstd and g = dz·γ:  ds = rstd·(g − mean(g) − u·mean(g·u)) + ds_in,
// dx = D(ds), dγ = Σ_m dz·u, dβ = Σ_m dz.  T threads share a row, V vectors each, staged two rows
// ahead in shared memory and read from there twice (for the sums, then for the gradients), so that
// registers hold little beside the dγ, dβ sums of the thread's columns, which it keeps over all its
// rows.  A CTA of 512 (or T) threads holds R rows at a time; at the end its row groups add their
// sums in turn in shared memory and store one partial row each of dγ and dβ, which
// fl_ln_wgrad_kernel adds in a fixed order.
template <int T, int V>
__global__ void __launch_bounds__(T < 512 ? 512 : T, T < 1024 ? 2 : 1) fl_dropout_ln_bwd_kernel(const DropLnBwdArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr int BLOCK = T < 512 ? 512 : T;
  constexpr int R = BLOCK / T;
  extern __shared__ __align__(16) uint8_t ring_s[];
  __shared__ float2 red_s[R][2 * (T / 32)];
  __shared__ float part_s[R > 1 ? 16 * V * T : 1];
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  int flip = 0;
  const uint64_t offset = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N;
  const long long m0 = (long long)blockIdx.x * R + group, step = (long long)gridDim.x * R;
  const uint32_t ring = smem_u32(ring_s);
  const uint32_t zb = operand_bytes(P.dz, V, BLOCK), sb = operand_bytes(P.s, V, BLOCK);
  const uint32_t slot_bytes = zb + sb + operand_bytes(P.ds_in, V, BLOCK);
  float pg[V][8], pb[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) pg[k][i] = pb[k][i] = 0.0f;
  auto prefetch = [&](long long m, uint32_t slot) {
    if (m < P.M && P.vec) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int c0 = 8 * (k * T + t);
        if (c0 + 8 <= P.N) {
          stage_vec<V, BLOCK>(slot, P.dz, m, c0, k);
          stage_vec<V, BLOCK>(slot + zb, P.s, m, c0, k);
          if (P.ds_in.p != nullptr) stage_vec<V, BLOCK>(slot + zb + sb, P.ds_in, m, c0, k);
        }
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < P.ahead; ++i) prefetch(m0 + i * step, ring + i * slot_bytes);
  int at = 0;
  for (long long m = m0; m < P.M; m += step) {
    const uint32_t slot = ring + at * slot_bytes;
    const float mean = P.mean[m], rstd = P.rstd[m];
    // dz and u = (s − μ)·rstd of vector k (zeros past N)
    auto values = [&](int k, int c0, int cnt, bool vec, float (&dz)[8], float (&u)[8]) {
      if (vec) {
        unstage_vec<V, BLOCK>(dz, slot, P.dz.dt, k);
        unstage_vec<V, BLOCK>(u, slot + zb, P.s.dt, k);
      } else {
        load_some8(dz, P.dz, m, c0, cnt);
        load_some8(u, P.s, m, c0, cnt);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = i < cnt ? (u[i] - mean) * rstd : 0.0f;
    };
    wait_row(P.ahead);
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * T + t);
      const int cnt = min(8, P.N - c0);
      if (cnt <= 0) continue;
      const bool vec = P.vec && cnt == 8;
      float dz[8], u[8], gam[8];
      load_param8(gam, P.gamma, P.param_dt, c0, cnt, vec, 1.0f);
      values(k, c0, cnt, vec, dz, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pg[k][i] = fmaf(dz[i], u[i], pg[k][i]);
        pb[k][i] += dz[i];
        const float g = dz[i] * gam[i];
        a += i < cnt ? g : 0.0f;
        b = fmaf(g, u[i], b);
      }
    }
    const float2 ab = row_sum<T>(a, b, red_s[group], flip, group);
    const float ma = ab.x / n_f, mb = ab.y / n_f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * T + t);
      const int cnt = min(8, P.N - c0);
      if (cnt <= 0) continue;
      const bool vec = P.vec && cnt == 8;
      float dz[8], u[8], gam[8];
      load_param8(gam, P.gamma, P.param_dt, c0, cnt, vec, 1.0f);
      values(k, c0, cnt, vec, dz, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) dz[i] = rstd * (dz[i] * gam[i] - ma - u[i] * mb);
      if (P.ds_in.p != nullptr) {
        if (vec) unstage_vec<V, BLOCK>(u, slot + zb + sb, P.ds_in.dt, k);
        else load_some8(u, P.ds_in, m, c0, cnt);
#pragma unroll
        for (int i = 0; i < 8; ++i) dz[i] += u[i];
      }
      if (P.dres.p != nullptr) store8(P.dres, m, c0, cnt, vec, dz);
      if (P.dx.p != nullptr) {
        if (P.d.on) drop8(dz, (uint64_t)(m * groups + (c0 >> 2)), offset, P.d);
        store8(P.dx, m, c0, cnt, vec, dz);
      }
    }
    prefetch(m + P.ahead * step, slot);
    at = at + 1 == P.ahead ? 0 : at + 1;
  }
  cp_async_wait<0>();
  if (P.ws == nullptr) return;
  float* out = P.ws + (long long)blockIdx.x * 2 * P.ws_ld;
  if constexpr (R > 1) {
    constexpr int W = 8 * V * T;
    for (int g = 0; g < R; ++g) {
      if (group == g) {
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = (i * V + k) * T + t;  // (a warp's lanes side by side: no bank conflicts)
            if (g > 0) pg[k][i] += part_s[c], pb[k][i] += part_s[W + c];
            part_s[c] = pg[k][i];
            part_s[W + c] = pb[k][i];
          }
      }
      __syncthreads();
    }
  }
  if (group == R - 1) {  // (the last group's registers hold the sums of all)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * T + t);
      if (c0 >= P.N) continue;
      float4* q = reinterpret_cast<float4*>(out + c0);
      q[0] = make_float4(pg[k][0], pg[k][1], pg[k][2], pg[k][3]);
      q[1] = make_float4(pg[k][4], pg[k][5], pg[k][6], pg[k][7]);
      q = reinterpret_cast<float4*>(out + P.ws_ld + c0);
      q[0] = make_float4(pb[k][0], pb[k][1], pb[k][2], pb[k][3]);
      q[1] = make_float4(pb[k][4], pb[k][5], pb[k][6], pb[k][7]);
    }
  }
}

// Rows longer than 16·1024 elements: a CTA of 1024 threads walks each of its rows twice (sums,
// then gradients) and adds to its partial rows of dγ and dβ in the workspace, each column always
// by the same thread.
__global__ void __launch_bounds__(1024) fl_dropout_ln_bwd_long_kernel(const DropLnBwdArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  __shared__ float2 red[2 * 32];
  int flip = 0;
  const uint64_t offset = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N;
  float* out = P.ws == nullptr ? nullptr : P.ws + (long long)blockIdx.x * 2 * P.ws_ld;
  for (long long m = blockIdx.x; m < P.M; m += gridDim.x) {
    const float mean = P.mean[m], rstd = P.rstd[m];
    const bool first = m == blockIdx.x;
    float ma = 0.0f, mb = 0.0f;
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
      float a = 0.0f, b = 0.0f;
      for (long long c = 8LL * threadIdx.x; c < P.N; c += 8 * 1024) {
        const int c0 = (int)c, cnt = min(8, P.N - c0);
        const bool vec = P.vec && cnt == 8;
        float dz[8], u[8], gam[8];
        if (vec) {
          widen8(dz, load_raw8(P.dz, m, c0), P.dz.dt);
          widen8(u, load_raw8(P.s, m, c0), P.s.dt);
        } else {
          load_some8(dz, P.dz, m, c0, cnt);
          load_some8(u, P.s, m, c0, cnt);
        }
        load_param8(gam, P.gamma, P.param_dt, c0, cnt, vec, 1.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = i < cnt ? (u[i] - mean) * rstd : 0.0f;
        if (step == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (out != nullptr && i < cnt) {
              float* pg = out + c0 + i;
              float* pb = out + P.ws_ld + c0 + i;
              *pg = first ? dz[i] * u[i] : fmaf(dz[i], u[i], *pg);
              *pb = first ? dz[i] : *pb + dz[i];
            }
            const float g = dz[i] * gam[i];
            a += i < cnt ? g : 0.0f;
            b = fmaf(g, u[i], b);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) dz[i] = rstd * (dz[i] * gam[i] - ma - u[i] * mb);
          if (P.ds_in.p != nullptr) {
            float in[8];
            if (vec) widen8(in, load_raw8(P.ds_in, m, c0), P.ds_in.dt);
            else load_some8(in, P.ds_in, m, c0, cnt);
#pragma unroll
            for (int i = 0; i < 8; ++i) dz[i] += in[i];
          }
          if (P.dres.p != nullptr) store8(P.dres, m, c0, cnt, vec, dz);
          if (P.dx.p != nullptr) {
            if (P.d.on) drop8(dz, (uint64_t)(m * groups + (c0 >> 2)), offset, P.d);
            store8(P.dx, m, c0, cnt, vec, dz);
          }
        }
      }
      if (step == 0) {
        const float2 ab = row_sum<1024>(a, b, red, flip, 0);
        ma = ab.x / n_f;
        mb = ab.y / n_f;
      }
    }
  }
}

// dγ[c] (blockIdx.y 0) or dβ[c] (1) = Σ over the `rows` partial rows of the workspace, in a
// fixed order: thread (g, l) of a CTA of 32 x 32 adds rows g, g + 32, ... of column l, then the 32
// group sums are added in group order.
__global__ void __launch_bounds__(1024) fl_ln_wgrad_kernel(const float* __restrict__ ws, float* dgamma, float* dbeta,
                                                           int N, int ws_ld, int rows) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  float* out = blockIdx.y == 0 ? dgamma : dbeta;
  const int g = threadIdx.x >> 5, l = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + l;
  __shared__ float red[32][33];
  float s = 0.0f;
  if (c < N && out != nullptr) {
    const float* p = ws + (long long)blockIdx.y * ws_ld + c;
    for (int b0 = g; b0 < rows; b0 += 32 * 8) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int b = b0 + 32 * k;
        t[k] = b < rows ? __ldcg(p + (long long)b * 2 * ws_ld) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += t[k];
    }
  }
  red[g][l] = s;
  __syncthreads();
  if (g == 0 && c < N && out != nullptr) {
    float r = red[0][l];
#pragma unroll
    for (int k = 1; k < 32; ++k) r += red[k][l];
    out[c] = r;
  }
}

}  // namespace fl
