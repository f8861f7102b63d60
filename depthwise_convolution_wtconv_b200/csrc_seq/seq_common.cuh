// Shared pieces of the sequence kernels: I/O types, rows of an activation,
// the gate functions and the fixed-order sum of per-block partials.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "wtconv_seq.h"

namespace wtseq {

template <typename IO> __device__ __forceinline__ float to_f(IO v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
// One rounding to nearest even, of outputs only: off by at most 2^-8 of the value.
template <typename IO> __device__ __forceinline__ IO from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Rows of an activation, strides in elements (64-bit: a cache may hold more
// than 2^31 elements).
template <typename IO> struct Rows {
  IO* p;
  long long sb, st;
  __device__ __forceinline__ IO* at(int b, long long t) const { return p + b * sb + t * st; }
};

// Rows of one token have no token stride: what the caller holds there may be
// anything, and kernels that copy whole tiles form the addresses of the tokens
// that are not there too (a copy of no bytes still wants an aligned one).
template <typename IO> inline Rows<IO> rows_of(const wtconv_rows* r, int T) {
  if (!r) return Rows<IO>{nullptr, 0, 0};
  return Rows<IO>{static_cast<IO*>(r->data), r->batch_stride, T > 1 ? r->token_stride : 0};
}

// V consecutive channels in accesses of up to 16 bytes, which they are aligned
// to, and as fp32 values.
template <typename IO, int V> struct alignas(sizeof(IO) * V <= 16 ? sizeof(IO) * V : 16) Pack { IO v[V]; };

template <typename IO, int V> __device__ __forceinline__ void load_pack(const IO* p, float (&f)[V]) {
  constexpr int W = sizeof(IO) * V <= 16 ? V : 16 / sizeof(IO);
#pragma unroll
  for (int k = 0; k < V; k += W) {
    const Pack<IO, W> r = *reinterpret_cast<const Pack<IO, W>*>(p + k);
#pragma unroll
    for (int i = 0; i < W; ++i) f[k + i] = to_f<IO>(r.v[i]);
  }
}
// V channels as they lie in memory, to be had in flight and converted later.
// Read-only loads: for inputs, which no output may overlap, so that loads may
// pass the stores of earlier tokens.
template <typename IO, int V> struct Raw {
  static constexpr int W = sizeof(IO) * V <= 16 ? V : 16 / sizeof(IO);
  Pack<IO, W> r[V / W];
  __device__ __forceinline__ void load(const IO* p) {
#pragma unroll
    for (int k = 0; k < V / W; ++k) {
      if constexpr (sizeof(Pack<IO, W>) == 16)
        *reinterpret_cast<uint4*>(&r[k]) = __ldg(reinterpret_cast<const uint4*>(p + k * W));
      else if constexpr (sizeof(Pack<IO, W>) == 8)
        *reinterpret_cast<uint2*>(&r[k]) = __ldg(reinterpret_cast<const uint2*>(p + k * W));
      else if constexpr (W == 2)
        *reinterpret_cast<unsigned*>(&r[k]) = __ldg(reinterpret_cast<const unsigned*>(p + k * W));
      else
        r[k].v[0] = __ldg(p + k * W);
    }
  }
  __device__ __forceinline__ void floats(float (&f)[V]) const {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = to_f<IO>(r[k / W].v[k % W]);
  }
};
template <typename IO, int V> __device__ __forceinline__ void store_pack(IO* p, const float (&f)[V]) {
  constexpr int W = sizeof(IO) * V <= 16 ? V : 16 / sizeof(IO);
#pragma unroll
  for (int k = 0; k < V; k += W) {
    Pack<IO, W> r;
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i] = from_f<IO>(f[k + i]);
    *reinterpret_cast<Pack<IO, W>*>(p + k) = r;
  }
}

__device__ __forceinline__ int row_length(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = __ldg(lengths + b);
  return n < 0 ? 0 : (n < T ? n : T);
}

// 2^v and 1/v with results (and arguments) below 2^-126 flushed to zero:
// relative errors below 2^-22 and 2^-23.  The forms that keep such values cost
// three more instructions each.
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// 1 / (1 + exp(-v)): the exponential overflows to infinity for v < -88, and
// the quotient is then the zero that it should be.
__device__ __forceinline__ float sigmoid(float v) { return rcp_approx(1.f + exp2_approx(v * -LOG2E)); }

// d silu(v) / dv, given sigmoid(v)
__device__ __forceinline__ float dsilu(float v, float sg) { return sg * (1.f + v * (1.f - sg)); }

// Two fp32 values in a register pair and the operations on both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 twice(float v) { return pair(v, v); }
__device__ __forceinline__ void unpair(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 1 / (1 + exp(-v)) of a pair
__device__ __forceinline__ f32x2 sigmoid2(f32x2 v) {
  float a, b;
  unpair(mul2(v, twice(-LOG2E)), a, b);
  unpair(add2(pair(exp2_approx(a), exp2_approx(b)), twice(1.f)), a, b);
  return pair(rcp_approx(a), rcp_approx(b));
}

// d silu(v) / dv = s + v s (1 - s), s = sigmoid(v), of a pair
__device__ __forceinline__ f32x2 dsilu2(f32x2 v, f32x2 s) {
  return fma2(mul2(v, s), fma2(s, twice(-1.f), twice(1.f)), s);
}

// The V channels of a thread, as fp32 pairs where V is even: every operation
// below is on a pair (or, for V = 1, on one value and a zero beside it).
template <int V> struct Vals {
  static constexpr int P = (V + 1) / 2;
  f32x2 p[P];
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = pair(f[2 * i], 2 * i + 1 < V ? f[2 * i + 1 < V ? 2 * i + 1 : 0] : 0.f);
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float lo, hi;
      unpair(p[i], lo, hi);
      f[2 * i] = lo;
      if (2 * i + 1 < V) f[2 * i + 1 < V ? 2 * i + 1 : 0] = hi;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = 0;
  }
};

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) <= 1.
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3, is s times a polynomial in
// s^2 (degree 4, interpolated at the Chebyshev nodes of [0, 1/9]: off by less
// than 1e-8).  The logarithm of the rounded sum 1 + e would lose the small e,
// and with them the step sizes near 1e-3 that a scan lives on.  NaN stays NaN
// (fmaxf gives 0 then, but the exponential is NaN).
__device__ __forceinline__ float softplus(float v) {
  const float e = exp2_approx(fabsf(v) * -LOG2E);
  const float s = e * rcp_approx(2.f + e), q = s * s;
  float r = fmaf(0.28157778f, q, 0.27965158f);
  r = fmaf(r, q, 0.40024595f);
  r = fmaf(r, q, 0.66666322f);
  r = fmaf(r, q, 2.f);
  return fmaf(r, s, fmaxf(v, 0.f));
}

// out[i] = sum over p of part[p * stride + i] in a fixed order: a block holds
// 32 outputs x SLICES slices of p, each summed in order, the slices joined in
// order.
template <int SLICES, typename Target>
__device__ __forceinline__ void sum_block(const float* __restrict__ part, long long P, long long stride, long long n, long long block,
                                          const Target& target) {
  __shared__ float s[SLICES][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const long long i = block * 32 + x;
  float v = 0.f;
  if (i < n) {
    const long long per = (P + SLICES - 1) / SLICES, p1 = (y + 1) * per < P ? (y + 1) * per : P;
#pragma unroll 8
    for (long long p = y * per; p < p1; ++p) v += __ldg(part + p * stride + i);
  }
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && i < n) {
#pragma unroll
    for (int k = 1; k < SLICES; ++k) v += s[k][x];
    target.put(i, v);
  }
}

template <int SLICES, typename Target>
__global__ void __launch_bounds__(SLICES * 32)
    sum_partials(const float* __restrict__ part, long long P, long long stride, long long n, Target target) {
  sum_block<SLICES>(part, P, stride, n, blockIdx.x, target);
}

// Many parts of few outputs are a chain of loads per thread: 32 slices then
// (2368 parts of 744 sums, a norm's gradients of 6276 rows of 248 channels in
// bf16: the call takes 47 us with 8 slices, 28 us with 32; 8x2048x512 fp32: 96
// and 87 us).
template <typename Target>
inline void launch_sum(const float* part, long long P, long long stride, long long n, Target t, cudaStream_t st) {
  const unsigned blocks = (unsigned)((n + 31) / 32);
  if (P >= 256)
    sum_partials<32, Target><<<blocks, 1024, 0, st>>>(part, P, stride, n, t);
  else
    sum_partials<8, Target><<<blocks, 256, 0, st>>>(part, P, stride, n, t);
}

}  // namespace wtseq
