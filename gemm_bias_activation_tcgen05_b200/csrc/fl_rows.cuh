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
//
// A round is two 32 x 32 -> 64 multiplications and two three-way exclusive ors: the round keys come
// from the host, so that they are constant-bank operands, and what the first round makes of the
// offset is the same for every element.  The multiplications (four cycles each of one of the SM's
// pipes) are what bounds these kernels after the memory: that pipe was active for 73 % of the time
// of an 8192 x 4096 bf16 dropout with residual (42 us).
struct DropParams {
  uint32_t k0[10], k1[10];     // the rounds' keys, from the seed's halves
  uint64_t offset;             // upper counter half
  const uint64_t* offset_dev;  // added to offset when not null (read on the device)
  uint32_t threshold;          // dropped where the word is below ⌊p·2^32⌋
  float scale;                 // 1/(1 − p)
  int on;                      // 0: p = 0, nothing is drawn
};
inline void set_drop_keys(DropParams* d, uint64_t seed) {
  for (uint32_t r = 0; r < 10; ++r) {
    d->k0[r] = (uint32_t)seed + r * 0x9E3779B9u;
    d->k1[r] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
  }
}

// What a thread keeps of the offset and the keys: everything that the first two rounds make of
// them alone, for blocks below 2^32 (so that 18 multiplications remain of 20).
struct DropOffset {
  uint32_t w0, w1, w2;      // round 1: shares of the new words 0, 1 and 2
  uint32_t v0, v2, v3;      // round 2: shares of the new words 0, 2 and 3
};
__host__ __device__ __forceinline__ DropOffset drop_offset(const DropParams& d) {
  uint64_t off = d.offset;
  if (d.on && d.offset_dev != nullptr) off += *d.offset_dev;
  const uint64_t b = (uint64_t)(uint32_t)off * 0xCD9E8D57u;
  DropOffset o;
  o.w0 = (uint32_t)(b >> 32) ^ d.k0[0];
  o.w1 = (uint32_t)b;
  o.w2 = (uint32_t)(off >> 32) ^ d.k1[0];
  const uint64_t a = (uint64_t)o.w0 * 0xD2511F53u;
  o.v0 = o.w1 ^ d.k0[1];
  o.v2 = (uint32_t)(a >> 32) ^ d.k1[1];
  o.v3 = (uint32_t)a;
  return o;
}

// BIG: blocks may reach 2^32 (matrices of 2^34 elements and more, which run on the untyped kernels)
template <bool BIG>
__host__ __device__ __forceinline__ uint4 philox4x32_10(uint64_t block, const DropOffset& o, const DropParams& d) {
  const uint64_t first = (uint64_t)(uint32_t)block * 0xD2511F53u;
  const uint32_t f2 = (uint32_t)(first >> 32) ^ o.w2, f3 = (uint32_t)first;
  const uint64_t second = (uint64_t)f2 * 0xCD9E8D57u;
  uint32_t c0 = (uint32_t)(second >> 32) ^ o.v0, c1 = (uint32_t)second, c2 = o.v2 ^ f3, c3 = o.v3;
  if (BIG) {
    const uint64_t a = (uint64_t)(o.w0 ^ (uint32_t)(block >> 32)) * 0xD2511F53u;
    c2 = (uint32_t)(a >> 32) ^ f3 ^ d.k1[1];
    c3 = (uint32_t)a;
  }
#pragma unroll
  for (int r = 2; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ d.k0[r];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ d.k1[r];
    c3 = (uint32_t)a;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The random numbers of the eight elements of blocks `block` and `block` + 1.  Drawn while the
// elements themselves are still on their way from memory.
struct Draw8 {
  uint4 a, b;
};
template <bool BIG>
__device__ __forceinline__ Draw8 draw8(uint64_t block, const DropOffset& o, const DropParams& d) {
  return {philox4x32_10<BIG>(block, o, d), philox4x32_10<BIG>(block + 1, o, d)};
}
// r[i] += D(v)[i].  A dropped element adds nothing at all (not 0·v, which would keep a NaN); a kept
// one is one fused product and sum.
__device__ __forceinline__ void add_dropped8(float (&r)[8], const float (&v)[8], const Draw8& w, const DropParams& d) {
  const uint32_t x[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (x[i] >= d.threshold) r[i] = fmaf(v[i], d.scale, r[i]);
}
// v = D(v)
__device__ __forceinline__ void drop8(float (&v)[8], const Draw8& w, const DropParams& d) {
  const uint32_t x[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i] >= d.threshold ? v[i] * d.scale : 0.0f;
}

// ---------------------------------------------------------------- eight elements of a row
// A matrix operand: null, or [M, ld] of dtype dt.  All accesses are plain (coherent) loads and
// stores, because an output may be an input's own buffer.
struct Mat {
  void* p;
  long long ld;
  int dt;
};
// The kernels come in two forms.  The typed ones know their operands' types (template arguments
// ≥ 0) and run on rows of whole 16-byte vectors that start on 16 bytes; the others take the types from
// the operands, accept rows that start anywhere, and check every vector.  The checks and type branches
// cost about a third of the instructions, which bound these kernels: 8192 x 4096 bf16 with a residual,
// dropout 53.7 us untyped, with LayerNorm 86.5, its backward 133, against 42.6, 60.5 and 103 typed (in
// their first forms).
constexpr int ANY = -1;
template <int DT>
__device__ __forceinline__ int dt_of(const Mat& t) {
  if constexpr (DT >= 0) return DT;
  else return t.dt;
}

struct Raw8 {
  uint4 a, b;  // 16-bit types: a; fp32: a and b
};

__device__ __forceinline__ Raw8 load_raw8(const Mat& t, long long row, int c0, int dt) {
  Raw8 r;
  if (dt == DT_F32) {
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
    // (a byte permutation, not a shift, which would go to the multiplications' pipe)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(__byte_perm(w[i], 0u, 0x1044));
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
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
// elements c0 .. c0 + cnt − 1 of a row one by one, zeros after them
__device__ __forceinline__ void load_some8(float (&v)[8], const Mat& t, long long row, int c0, int cnt) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < cnt ? load1(t.p, row * t.ld + c0 + i, t.dt) : 0.0f;
}
// Eight elements that start `skew` bytes into the words w (three 16-byte words; 16-bit types need two).
__device__ __forceinline__ Raw8 unskew(uint32_t (&w)[12], int skew) {
  if (skew & 8) {
#pragma unroll
    for (int j = 0; j < 10; ++j) w[j] = w[j + 2];
  }
  if (skew & 4) {
#pragma unroll
    for (int j = 0; j < 9; ++j) w[j] = w[j + 1];
  }
  if (skew & 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
  }
  return {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}
// Elements c0 .. c0 + 7 of a row that starts anywhere, zeros from element cnt on: the 16-byte words
// that hold them where these lie inside the operand (M rows of N), else one by one.
__device__ __forceinline__ void gather8(float (&v)[8], const Mat& t, long long row, long long M, int N, int c0, int cnt) {
  const int es = t.dt == DT_F32 ? 4 : 2;
  const char* base = reinterpret_cast<const char*>(t.p);
  const char* at = base + (row * t.ld + c0) * es;
  const int skew = (int)(reinterpret_cast<uintptr_t>(at) & 15u);
  const int words = es / 2 + (skew != 0);
  const char* from = at - skew;
  if (cnt < 8 || from < base || from + 16 * words > base + ((M - 1) * t.ld + N) * es) {
    load_some8(v, t, row, c0, cnt);
    return;
  }
  uint32_t w[12];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const uint4 q = j < words ? reinterpret_cast<const uint4*>(from)[j] : make_uint4(0u, 0u, 0u, 0u);
    w[4 * j] = q.x, w[4 * j + 1] = q.y, w[4 * j + 2] = q.z, w[4 * j + 3] = q.w;
  }
  widen8(v, unskew(w, skew), t.dt);
}
// v into elements c0 .. c0 + cnt − 1.  vec: all eight, on 16 bytes.  Otherwise eight elements that
// start anywhere go out as words where they can (16-bit types: a first half, three words and a last
// half where the address is odd in words), fewer one by one.
__device__ __forceinline__ void store8(const Mat& t, long long row, int c0, int cnt, bool vec, const float (&v)[8], int dt) {
  const long long i0 = row * t.ld + c0;
  if (dt == DT_F32) {
    float* q = reinterpret_cast<float*>(t.p) + i0;
    if (vec) {
      reinterpret_cast<float4*>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) q[i] = v[i];
    }
    return;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = dt == DT_BF16 ? pack2<DT_BF16>(v[2 * j], v[2 * j + 1]) : pack2<DT_F16>(v[2 * j], v[2 * j + 1]);
  uint16_t* q = reinterpret_cast<uint16_t*>(t.p) + i0;
  if (vec) {
    *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (cnt == 8) {
    if ((reinterpret_cast<uintptr_t>(q) & 2u) == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(q)[j] = w[j];
    } else {
      q[0] = (uint16_t)w[0];
#pragma unroll
      for (int j = 0; j < 3; ++j) *reinterpret_cast<uint32_t*>(q + 1 + 2 * j) = __funnelshift_r(w[j], w[j + 1], 16);
      q[7] = (uint16_t)(w[3] >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
// eight parameters of type dt from c0; `dflt` for a null pointer
__device__ __forceinline__ void load_param8(float (&v)[8], const void* p, int dt, int c0, int cnt, bool vec, float dflt) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = dflt;
  } else {
    const Mat t{const_cast<void*>(p), 0, dt};
    if (vec) widen8(v, load_raw8(t, 0, c0, dt), dt);
    else gather8(v, t, 0, 1, c0 + cnt, c0, cnt);
  }
}

__device__ __forceinline__ float2 pair_of(const float (&v)[8], int j) { return make_float2(v[2 * j], v[2 * j + 1]); }
__device__ __forceinline__ void put_pair(float (&v)[8], int j, float2 q) { v[2 * j] = q.x, v[2 * j + 1] = q.y; }

// ---------------------------------------------------------------- dropout
struct DropoutArgs {
  Mat x, r, y;  // r.p null: no residual
  long long M;
  int N, nvec, vec;  // nvec = ⌈N/8⌉ vectors a row; vec: every row of every operand is 16-byte aligned
  DropParams d;
};

// Thread i of the grid takes vectors i, i + threads, ... of the M·nvec (row, vector) pairs; row
// and vector advance by the stride's quotient and remainder, so that one division runs per
// thread.  The random numbers are drawn while the vectors are on their way.  One vector a trip and
// all the warps an SM holds: 8192 x 4096 bf16 with a residual takes 37.4 us (5.4 TB/s; without the
// drawing, p = 0, 30.4 us, the copy rate), two vectors and half the warps 42.4, and with two
// vectors six CTAs 38.5.
// (The untyped form needs more registers than eight CTAs leave it.)
__host__ __device__ constexpr int dropout_ctas(bool typed) { return typed ? 8 : 4; }
template <int XT, int YT>
__global__ void __launch_bounds__(256, dropout_ctas(XT >= 0)) fl_dropout_kernel(const DropoutArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr bool TYPED = XT >= 0;
  const int xt = dt_of<XT>(P.x), yt = dt_of<YT>(P.y);
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long i0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long srow = stride / P.nvec;
  const int svec = (int)(stride - srow * P.nvec);
  long long row = i0 / P.nvec;
  int v = (int)(i0 - row * P.nvec);
  const DropOffset off = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const bool has_r = P.r.p != nullptr;
  while (row < P.M) {
    const int c0 = 8 * v;
    const int cnt = TYPED ? 8 : min(8, P.N - c0);
    const bool vec = TYPED || (P.vec && cnt == 8);
    Raw8 rx, rr;
    if (vec) {
      rx = load_raw8(P.x, row, c0, xt);
      if (has_r) rr = load_raw8(P.r, row, c0, yt);
    }
    Draw8 w;
    if (P.d.on) w = draw8<!TYPED>((uint64_t)(row * groups + (c0 >> 2)), off, P.d);
    float x[8], r[8];
    if (vec) widen8(x, rx, xt);
    else gather8(x, P.x, row, P.M, P.N, c0, cnt);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0.0f;
    if (has_r) {
      if (vec) widen8(r, rr, yt);
      else gather8(r, P.r, row, P.M, P.N, c0, cnt);
    }
    if (P.d.on) {
      add_dropped8(r, x, w, P.d);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] += x[i];
    }
    store8(P.y, row, c0, cnt, vec, r, yt);
    row += srow;
    v += svec;
    if (v >= P.nvec) v -= P.nvec, ++row;
  }
}

// ---------------------------------------------------------------- sums over a row's threads
// Sums of one or two values over the threads that share a row, the same in every thread: a
// butterfly in each warp, then the warps' sums in warp order.  `red` holds two sets of T/32 pairs,
// used in turn (`flip`), so that one barrier a call is enough: a warp writes a set again only after the
// next call's barrier, which every reader of the set has passed its reads before.
__device__ __forceinline__ void row_barrier(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
}
template <int T>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red, int& flip, int group, int t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    float2* set = red + flip * W;
    flip ^= 1;
    if ((t & 31) == 0) set[t >> 5] = v;
    row_barrier(group, T);
    v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float4 q = *reinterpret_cast<const float4*>(set + i);
      v = add2(v, make_float2(q.x, q.y));
      v = add2(v, make_float2(q.z, q.w));
    }
  }
  return v;
}
template <int T>
__device__ __forceinline__ float row_sum(float v, float2* red2, int& flip, int group, int t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    float* set = reinterpret_cast<float*>(red2 + flip * W);
    flip ^= 1;
    if ((t & 31) == 0) set[t >> 5] = v;
    row_barrier(group, T);
    float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      a = add2(a, *reinterpret_cast<const float2*>(set + i));
    }
    v = a.x + a.y;
  }
  return v;
}

// a/n for a row length n, with inv = 1/n: one step of Newton's iteration on the rounded product
// (five instructions, against a dozen for a division).  The step has no answer for an infinite sum,
// whose mean is the infinity itself.
__device__ __forceinline__ float div_n(float a, float n, float inv) {
  const float q = a * inv;
  return isinf(q) ? q : fmaf(fmaf(-q, n, a), inv, q);
}

// ---------------------------------------------------------------- rows ahead in shared memory
// The 16-byte words of a row are copied to shared memory (cp.async, one group a row) `ahead` rows
// before they are needed, so that the bytes in flight cost no registers.  The ring has two slots, or
// one where two do not fit.  A slot holds for each operand and row group `row_words` words.
//  * Typed: a thread copies its own vectors and reads back only those: no barrier stands between the
//    copy and its use.
//  * Untyped: the row may start anywhere.  The words that cover it are copied, the row's threads meet
//    at a barrier, and a thread puts its eight elements together from the words they lie in.
constexpr int kRowsAhead = 2;
__device__ __forceinline__ void wait_row(int ahead) {
  if (ahead == kRowsAhead) cp_async_wait<kRowsAhead - 1>();
  else cp_async_wait<0>();
}
// words of a row of `vectors` vectors of eight; two more for one that starts anywhere
__host__ __device__ __forceinline__ uint32_t row_words(const Mat& t, int vectors) {
  return t.p == nullptr ? 0u : (uint32_t)vectors * (t.dt == DT_F32 ? 2u : 1u) + 2u;
}

// Typed: vector vi of a row to its place from `dst`; an fp32 vector's second half lies `vectors` words
// behind its first.  The two halves share 32-byte sectors, so they go through the L1 cache: past it
// each sector is fetched twice (LayerNorm of 4096 x 4096 fp32 with a residual: 71.0 us so, 46.7 with the
// cache).  A line may outlive its data there when y is x's own buffer, but a row is read by its own
// threads alone, before they write it.
__device__ __forceinline__ void stage_vec(uint32_t dst, const Mat& t, long long row, int vi, int vectors, int dt) {
  const char* src = reinterpret_cast<const char*>(t.p) + (row * t.ld + 8 * vi) * (dt == DT_F32 ? 4 : 2);
  const uint32_t a = dst + (uint32_t)vi * 16u;
  if (dt == DT_F32) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(a), "l"(src) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(a + (uint32_t)vectors * 16u), "l"(src + 16) : "memory");
  } else {
    cp_async_16(a, src, 16u);
  }
}
__device__ __forceinline__ uint4 ld_shared_w4(uint32_t a) {
  const float4 q = ld_shared_f4(a);
  return make_uint4(__float_as_uint(q.x), __float_as_uint(q.y), __float_as_uint(q.z), __float_as_uint(q.w));
}
__device__ __forceinline__ void unstage_vec(float (&v)[8], uint32_t src, int vi, int vectors, int dt) {
  const uint32_t a = src + (uint32_t)vi * 16u;
  Raw8 r;
  r.a = ld_shared_w4(a);
  r.b = make_uint4(0u, 0u, 0u, 0u);
  if (dt == DT_F32) r.b = ld_shared_w4(a + (uint32_t)vectors * 16u);
  widen8(v, r, dt);
}

// Untyped: this thread's share (words t, t + threads, ...) of the words that cover row `row`.  A word
// that reaches outside the operand (its first row may start, its last row end, inside a word) is put
// together element by element.
__device__ __forceinline__ void stage_row(uint32_t dst, const Mat& t, long long row, long long M, int N, int tid, int threads) {
  const int es = t.dt == DT_F32 ? 4 : 2;
  const char* base = reinterpret_cast<const char*>(t.p);
  const char* begin = base + row * t.ld * es;
  const char* end = begin + (long long)N * es;
  const char* last = base + ((M - 1) * t.ld + N) * es;  // the operand's end
  const int skew = (int)(reinterpret_cast<uintptr_t>(begin) & 15u);
  const char* from = begin - skew;
  const int words = (int)((skew + (long long)N * es + 15) >> 4);
  for (int j = tid; j < words; j += threads) {
    const char* src = from + 16LL * j;
    const uint32_t to = dst + (uint32_t)j * 16u;
    if (src >= base && src + 16 <= last) {
      cp_async_16(to, src, 16u);
    } else {
      for (int e = 0; e < 16; e += es) {
        if (src + e < begin || src + e >= end) continue;
        if (es == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + e), "r"(*reinterpret_cast<const uint32_t*>(src + e)) : "memory");
        else asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + e), "h"(*reinterpret_cast<const uint16_t*>(src + e)) : "memory");
      }
    }
  }
}
// eight elements from element 8·vi of a staged row, zeros from element cnt on
__device__ __forceinline__ void unstage_row(float (&v)[8], uint32_t src, const Mat& t, long long row, int vi, int cnt) {
  const int es = t.dt == DT_F32 ? 4 : 2;
  const int skew = (int)((reinterpret_cast<uintptr_t>(t.p) + (unsigned long long)(row * t.ld * es)) & 15u);
  const uint32_t a = src + (uint32_t)vi * (8u * (uint32_t)es);
  uint32_t w[12];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    // (the word behind the vector only where the row is skewed; 16-bit types have no third word)
    if (j == 0 || (j == 1 && (es == 4 || skew != 0)) || (j == 2 && es == 4 && skew != 0)) q = ld_shared_w4(a + 16u * j);
    w[4 * j] = q.x, w[4 * j + 1] = q.y, w[4 * j + 2] = q.z, w[4 * j + 3] = q.w;
  }
  widen8(v, unskew(w, skew), t.dt);
  if (cnt < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cnt ? v[i] : 0.0f;
  }
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
// A CTA holds max(1, 128/T) rows at a time and walks the rows a grid apart; γ and β stay in registers
// (32 of them) but for 768 and 1024 threads, which have 80 and 64 each and read them from the cache at each
// row: kept in registers they made the 768-thread kernels spill (4096 x 10240 f16 with an fp32 stream 127.8 us
// against 113.8, 4096 x 12288 bf16 105.7 against 104.0, 64 rows of it 7.0 against 5.7).  Three vectors need 150 to 168 registers: three CTAs of 128
// threads an SM (with four, 128 registers spilled: 16384 x 1536 with an fp32 stream 66.6 us against 50.2).
__host__ __device__ constexpr int ln_block(int t) { return t < 128 ? 128 : t; }
template <int T, int V, int XT, int ST, int ZT>
__global__ void __launch_bounds__(ln_block(T), V == 3 ? 3 : T <= 128 ? 4 : T == 192 ? 2 : 1)
    fl_dropout_ln_kernel(const DropLnArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr bool TYPED = XT >= 0, HOIST = T < 768;
  constexpr int R = ln_block(T) / T;
  static_assert(R <= 15, "a row group has a named barrier of its own, 1 to 15");
  extern __shared__ __align__(16) uint8_t ring_s[];
  __shared__ __align__(16) float2 red_s[R][2 * (T / 32)];
  const int xt = dt_of<XT>(P.x), st = ST >= 0 ? ST : (P.r.p != nullptr ? P.r.dt : P.s.dt), zt = dt_of<ZT>(P.z);
  constexpr int threads = T, vectors = V * T;  // of a row
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  int flip = 0;
  const DropOffset off = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N, inv_n = 1.0f / n_f;
  const long long m0 = (long long)blockIdx.x * R + group, step = (long long)gridDim.x * R;
  const uint32_t xw = row_words(P.x, vectors), rw = row_words(P.r, vectors);
  const uint32_t slot_bytes = 16u * R * (xw + rw);
  const uint32_t ring = smem_u32(ring_s), xo = 16u * group * xw, ro = 16u * (R * xw + group * rw);
  const bool has_r = P.r.p != nullptr;
  // elements of vector k inside the row (typed: 8 or none)
  auto count = [&](int k) {
    const int left = P.N - 8 * (k * threads + t);
    return TYPED ? (left > 0 ? 8 : 0) : max(0, min(8, left));
  };
  auto prefetch = [&](long long m, uint32_t slot) {
    if (m < P.M) {
      if constexpr (TYPED) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (count(k) == 0) continue;
          stage_vec(slot + xo, P.x, m, k * threads + t, vectors, xt);
          if (has_r) stage_vec(slot + ro, P.r, m, k * threads + t, vectors, st);
        }
      } else {
        stage_row(slot + xo, P.x, m, P.M, P.N, t, threads);
        if (has_r) stage_row(slot + ro, P.r, m, P.M, P.N, t, threads);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < P.ahead; ++i) prefetch(m0 + i * step, ring + i * slot_bytes);
  float gam[HOIST ? V : 1][8], bet[HOIST ? V : 1][8];
  auto params = [&](int k, float (&g)[8], float (&b)[8]) {
    const int c0 = 8 * (k * threads + t), cnt = count(k);
    const bool vec = TYPED || (P.vec && cnt == 8);
    load_param8(g, P.gamma, P.param_dt, c0, cnt, vec, 1.0f);
    load_param8(b, P.beta, P.param_dt, c0, cnt, vec, 0.0f);
  };
  if constexpr (HOIST) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (count(k) > 0) params(k, gam[k], bet[k]);
  }
  int at = 0;
  for (long long m = m0; m < P.M; m += step) {
    const uint32_t slot = ring + at * slot_bytes;
    float s[V][8];
    float2 sum2 = make_float2(0.0f, 0.0f);
    Draw8 w[V];
    if (P.d.on) {
#pragma unroll
      for (int k = 0; k < V; ++k) w[k] = draw8<!TYPED>((uint64_t)(m * groups + 2 * (k * threads + t)), off, P.d);
    }
    wait_row(P.ahead);  // this thread's copies of the row have landed
    if constexpr (!TYPED) row_barrier(group, threads);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int vi = k * threads + t, cnt = count(k);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[k][i] = 0.0f;
      if (cnt == 0) continue;
      float x[8];
      if constexpr (TYPED) unstage_vec(x, slot + xo, vi, vectors, xt);
      else unstage_row(x, slot + xo, P.x, m, vi, cnt);
      if (has_r) {
        if constexpr (TYPED) unstage_vec(s[k], slot + ro, vi, vectors, st);
        else unstage_row(s[k], slot + ro, P.r, m, vi, cnt);
      }
      if (P.d.on) {
        add_dropped8(s[k], x, w[k], P.d);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) put_pair(s[k], j, add2(pair_of(s[k], j), pair_of(x, j)));
      }
      if (P.s.p != nullptr) store8(P.s, m, 8 * vi, cnt, TYPED || (P.vec && cnt == 8), s[k], st);
      // (elements past the row are zeros, and zeros they stay)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum2 = add2(sum2, pair_of(s[k], j));
    }
    if constexpr (TYPED) prefetch(m + P.ahead * step, slot);  // (the slot's values are in registers)
    const float mean = div_n(row_sum<T>(sum2.x + sum2.y, red_s[group], flip, group, t), n_f, inv_n);
    if constexpr (!TYPED) {
      // every thread's values are in registers (T = 32: the butterfly above joined the warp)
      prefetch(m + P.ahead * step, slot);
    }
    at = at + 1 == P.ahead ? 0 : at + 1;
    float2 q2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int cnt = count(k);
      if (cnt == 0) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 d = add2(pair_of(s[k], j), make_float2(-mean, -mean));
        if (!TYPED) d = make_float2(2 * j < cnt ? d.x : 0.0f, 2 * j + 1 < cnt ? d.y : 0.0f);
        put_pair(s[k], j, d);  // from here on s − μ
        q2 = fma2(d, d, q2);
      }
    }
    const float var = div_n(row_sum<T>(q2.x + q2.y, red_s[group], flip, group, t), n_f, inv_n);
    const float rstd = 1.0f / sqrtf(var + P.eps);
    if (t == 0 && P.mean != nullptr) P.mean[m] = mean, P.rstd[m] = rstd;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * threads + t), cnt = count(k);
      if (cnt == 0) continue;
      float g[8], b[8];
      if constexpr (!HOIST) params(k, g, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = mul2(pair_of(s[k], j), make_float2(rstd, rstd));
        put_pair(s[k], j, HOIST ? fma2(u, pair_of(gam[HOIST ? k : 0], j), pair_of(bet[HOIST ? k : 0], j))
                                : fma2(u, pair_of(g, j), pair_of(b, j)));
      }
      store8(P.z, m, c0, cnt, TYPED || (P.vec && cnt == 8), s[k], zt);
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
  __shared__ __align__(16) float2 red[2 * 32];
  int flip = 0;
  const DropOffset off = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N, inv_n = 1.0f / n_f;
  for (long long m = blockIdx.x; m < P.M; m += gridDim.x) {
    auto value = [&](int c0, int cnt, bool vec, float (&s)[8]) {
      float x[8];
      if (vec) widen8(x, load_raw8(P.x, m, c0, P.x.dt), P.x.dt);
      else gather8(x, P.x, m, P.M, P.N, c0, cnt);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.0f;
      if (P.r.p != nullptr) {
        if (vec) widen8(s, load_raw8(P.r, m, c0, P.r.dt), P.r.dt);
        else gather8(s, P.r, m, P.M, P.N, c0, cnt);
      }
      if (P.d.on) {
        add_dropped8(s, x, draw8<true>((uint64_t)(m * groups + (c0 >> 2)), off, P.d), P.d);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += x[i];
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
          if (P.s.p != nullptr) store8(P.s, m, c0, cnt, vec, s, P.s.dt);
          store8(P.z, m, c0, cnt, vec, g, P.z.dt);
        }
      }
      if (step == 0) mean = div_n(row_sum<1024>(acc, red, flip, 0, threadIdx.x), n_f, inv_n);
      if (step == 1) rstd = 1.0f / sqrtf(div_n(row_sum<1024>(acc, red, flip, 0, threadIdx.x), n_f, inv_n) + P.eps);
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
// dx = D(ds), dγ = Σ_m dz·u, dβ = Σ_m dz.  T threads share a row, V vectors each, staged rows
// ahead in shared memory; registers hold the row's g and u, γ, and the dγ, dβ sums of the thread's
// columns over all its rows (512 threads, which have half the registers, read the row from shared
// memory twice instead, for the sums and for the gradients).  A CTA of 256 (or T) threads holds R rows at
// a time; at the end its row groups' sums are added in shared memory and stored as one partial row each
// of dγ and dβ, which fl_ln_wgrad_kernel adds in a fixed order.
__host__ __device__ constexpr int ln_bwd_block(int t) { return 256 % t == 0 ? 256 : t; }
// bytes of the row groups' column sums at the end
__host__ __device__ constexpr size_t ln_bwd_part_bytes(int t, int v) {
  return ln_bwd_block(t) > t ? (size_t)(ln_bwd_block(t) / t) * 16u * (size_t)v * (size_t)t * sizeof(float) : 0;
}
template <int T, int V, int XT, int ST, int ZT>
__global__ void __launch_bounds__(ln_bwd_block(T), 1) fl_dropout_ln_bwd_kernel(const DropLnBwdArgs P) {
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  constexpr bool TYPED = XT >= 0;
  constexpr int BLOCK = ln_bwd_block(T);
  constexpr int R = BLOCK / T;
  static_assert(R <= 15, "a row group has a named barrier of its own, 1 to 15");
  constexpr bool KEEP = T <= 256;  // the row's values and γ stay in registers
  constexpr int VK = KEEP ? V : 1;
  extern __shared__ __align__(16) uint8_t ring_s[];
  __shared__ __align__(16) float2 red_s[R][2 * (T / 32)];
  const int xt = dt_of<XT>(P.dx), st = dt_of<ST>(P.s), zt = dt_of<ZT>(P.dz);
  constexpr int threads = T, vectors = V * T;  // of a row
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  int flip = 0;
  const DropOffset off = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N, inv_n = 1.0f / n_f;
  const long long m0 = (long long)blockIdx.x * R + group, step = (long long)gridDim.x * R;
  const uint32_t zw = row_words(P.dz, vectors), sw = row_words(P.s, vectors), iw = row_words(P.ds_in, vectors);
  const uint32_t slot_bytes = 16u * R * (zw + sw + iw);
  const uint32_t ring = smem_u32(ring_s);
  const uint32_t zo = 16u * group * zw, so = 16u * (R * zw + group * sw), io = 16u * (R * (zw + sw) + group * iw);
  const bool has_in = P.ds_in.p != nullptr;
  auto count = [&](int k) {
    const int left = P.N - 8 * (k * threads + t);
    return TYPED ? (left > 0 ? 8 : 0) : max(0, min(8, left));
  };
  auto prefetch = [&](long long m, uint32_t slot) {
    if (m < P.M) {
      if constexpr (TYPED) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (count(k) == 0) continue;
          stage_vec(slot + zo, P.dz, m, k * threads + t, vectors, zt);
          stage_vec(slot + so, P.s, m, k * threads + t, vectors, st);
          if (has_in) stage_vec(slot + io, P.ds_in, m, k * threads + t, vectors, st);
        }
      } else {
        stage_row(slot + zo, P.dz, m, P.M, P.N, t, threads);
        stage_row(slot + so, P.s, m, P.M, P.N, t, threads);
        if (has_in) stage_row(slot + io, P.ds_in, m, P.M, P.N, t, threads);
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < P.ahead; ++i) prefetch(m0 + i * step, ring + i * slot_bytes);
  float pg[V][8], pb[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) pg[k][i] = pb[k][i] = 0.0f;
  auto param = [&](int k, float (&g)[8]) {
    const int cnt = count(k);
    load_param8(g, P.gamma, P.param_dt, 8 * (k * threads + t), cnt, TYPED || (P.vec && cnt == 8), 1.0f);
  };
  float gam[VK][8];
  if constexpr (KEEP) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (count(k) > 0) param(k, gam[k]);
  }
  int at = 0;
  float next_mean = 0.0f, next_rstd = 0.0f;  // read a row ahead
  if (m0 < P.M) next_mean = P.mean[m0], next_rstd = P.rstd[m0];
  for (long long m = m0; m < P.M; m += step) {
    const uint32_t slot = ring + at * slot_bytes;
    const float mean = next_mean, rstd = next_rstd;
    if (m + step < P.M) next_mean = P.mean[m + step], next_rstd = P.rstd[m + step];
    // dz and u = (s − μ)·rstd of vector k (zeros past N)
    auto values = [&](int k, int cnt, float (&dz)[8], float (&u)[8]) {
      const int vi = k * threads + t;
      if constexpr (TYPED) {
        unstage_vec(dz, slot + zo, vi, vectors, zt);
        unstage_vec(u, slot + so, vi, vectors, st);
      } else {
        unstage_row(dz, slot + zo, P.dz, m, vi, cnt);
        unstage_row(u, slot + so, P.s, m, vi, cnt);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 q = mul2(add2(pair_of(u, j), make_float2(-mean, -mean)), make_float2(rstd, rstd));
        if (!TYPED) q = make_float2(2 * j < cnt ? q.x : 0.0f, 2 * j + 1 < cnt ? q.y : 0.0f);
        put_pair(u, j, q);
      }
    };
    wait_row(P.ahead);
    if constexpr (!TYPED) row_barrier(group, threads);
    float2 a2 = make_float2(0.0f, 0.0f), b2 = a2;
    float g[VK][8], u[VK][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int cnt = count(k);
      if (cnt == 0) continue;
      const int kk = KEEP ? k : 0;
      values(k, cnt, g[kk], u[kk]);
      if constexpr (!KEEP) param(k, gam[kk]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 z = pair_of(g[kk], j), w = pair_of(u[kk], j);
        put_pair(pg[k], j, fma2(z, w, pair_of(pg[k], j)));
        put_pair(pb[k], j, add2(z, pair_of(pb[k], j)));
        float2 q = mul2(z, pair_of(gam[kk], j));
        put_pair(g[kk], j, q);
        a2 = add2(a2, q);
        b2 = fma2(q, w, b2);
      }
    }
    const float2 ab = row_sum2<T>(make_float2(a2.x + a2.y, b2.x + b2.y), red_s[group], flip, group, t);
    const float ma = div_n(ab.x, n_f, inv_n), mb = div_n(ab.y, n_f, inv_n);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int vi = k * threads + t, c0 = 8 * vi, cnt = count(k);
      if (cnt == 0) continue;
      const bool vec = TYPED || (P.vec && cnt == 8);
      const int kk = KEEP ? k : 0;
      if constexpr (!KEEP) {
        values(k, cnt, g[0], u[0]);
        param(k, gam[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) put_pair(g[0], j, mul2(pair_of(g[0], j), pair_of(gam[0], j)));
      }
      float in[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) in[i] = 0.0f;
      if (has_in) {
        if constexpr (TYPED) unstage_vec(in, slot + io, vi, vectors, st);
        else unstage_row(in, slot + io, P.ds_in, m, vi, cnt);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 q = fma2(pair_of(u[kk], j), make_float2(-mb, -mb), add2(pair_of(g[kk], j), make_float2(-ma, -ma)));
        put_pair(in, j, fma2(q, make_float2(rstd, rstd), pair_of(in, j)));
      }
      if (P.dres.p != nullptr) store8(P.dres, m, c0, cnt, vec, in, st);
      if (P.dx.p != nullptr) {
        if (P.d.on) drop8(in, draw8<!TYPED>((uint64_t)(m * groups + (c0 >> 2)), off, P.d), P.d);
        store8(P.dx, m, c0, cnt, vec, in, xt);
      }
    }
    if constexpr (!TYPED) row_barrier(group, threads);  // every thread has read the slot
    prefetch(m + P.ahead * step, slot);
    at = at + 1 == P.ahead ? 0 : at + 1;
  }
  cp_async_wait<0>();
  if (P.ws == nullptr) return;
  float* out = P.ws + (long long)blockIdx.x * 2 * P.ws_ld;
  if constexpr (R > 1) {
    // every group's sums side by side in the ring's memory, then each thread adds the R sums of its
    // share of the columns in group order
    constexpr int W = 8 * V * T;
    float* part_s = reinterpret_cast<float*>(ring_s);
    __syncthreads();  // the ring is free
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (i * V + k) * T + t;  // (a warp's lanes side by side: no bank conflicts)
        part_s[group * 2 * W + c] = pg[k][i];
        part_s[group * 2 * W + W + c] = pb[k][i];
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2 * W / BLOCK; ++q) {
      const int e = q * BLOCK + (int)threadIdx.x;
      float v = part_s[e];
#pragma unroll
      for (int gr = 1; gr < R; ++gr) v += part_s[gr * 2 * W + e];
      const int j = e % W;
      const int c = 8 * (j / T % V * T + j % T) + j / (V * T);
      if (c < P.N) out[e / W * P.ws_ld + c] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c0 = 8 * (k * threads + t);
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
  __shared__ __align__(16) float2 red[2 * 32];
  int flip = 0;
  const DropOffset off = drop_offset(P.d);
  const long long groups = (P.N + 3) / 4;
  const float n_f = (float)P.N, inv_n = 1.0f / n_f;
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
          widen8(dz, load_raw8(P.dz, m, c0, P.dz.dt), P.dz.dt);
          widen8(u, load_raw8(P.s, m, c0, P.s.dt), P.s.dt);
        } else {
          gather8(dz, P.dz, m, P.M, P.N, c0, cnt);
          gather8(u, P.s, m, P.M, P.N, c0, cnt);
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
            if (vec) widen8(in, load_raw8(P.ds_in, m, c0, P.ds_in.dt), P.ds_in.dt);
            else gather8(in, P.ds_in, m, P.M, P.N, c0, cnt);
#pragma unroll
            for (int i = 0; i < 8; ++i) dz[i] += in[i];
          }
          if (P.dres.p != nullptr) store8(P.dres, m, c0, cnt, vec, dz, P.dres.dt);
          if (P.dx.p != nullptr) {
            if (P.d.on) drop8(dz, draw8<true>((uint64_t)(m * groups + (c0 >> 2)), off, P.d), P.d);
            store8(P.dx, m, c0, cnt, vec, dz, P.dx.dt);
          }
        }
      }
      if (step == 0) {
        const float2 ab = row_sum2<1024>(make_float2(a, b), red, flip, 0, threadIdx.x);
        ma = div_n(ab.x, n_f, inv_n);
        mb = div_n(ab.y, n_f, inv_n);
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
