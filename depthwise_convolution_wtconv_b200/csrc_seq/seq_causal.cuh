// Causal depthwise convolution over tokens: forward, gradients, one token.
//
// Each thread owns V neighbouring channels and walks a strip of tokens with
// the last k-1 inputs, the taps and the sums in registers, so every input is
// read once but for the k-1 tokens before a strip.
#pragma once

#include "seq_common.cuh"

namespace wtseq {

constexpr int CAUSAL_STRIP = 32;   // tokens of a forward thread
constexpr int CAUSAL_GSTRIP = 32;  // tokens of a gradient thread
constexpr int CAUSAL_GY = 8;       // strips of a gradient block

template <typename IO> struct CausalArgs {
  Rows<IO> x, y, dy, dx;
  const float *w, *bias;
  const IO* state;  // [B][k-1][C], or null: zeros
  IO* state_out;
  const IO* dstate_out;
  IO* dstate;
  const int* lengths;
  float* part;  // [groups][C][K+1]
  int B, T, C, silu, strips;
};

// Input at token t (t < 0: of the state before the pass).
template <typename IO, int K, int V>
__device__ __forceinline__ void causal_input(const CausalArgs<IO>& a, int b, long long t, int c, float (&f)[V]) {
  if (t >= 0) {
    load_pack<IO, V>(a.x.at(b, t) + c, f);
  } else if (a.state) {
    load_pack<IO, V>(a.state + ((long long)b * (K - 1) + (K - 1 + t)) * a.C + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
  }
}

template <typename IO, int K, int V>
__device__ __forceinline__ void causal_taps(const CausalArgs<IO>& a, int c, float (&w)[K][V], float (&bias)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = a.bias ? __ldg(a.bias + c + i) : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = __ldg(a.w + (long long)(c + i) * K + j);
  }
}

template <typename IO, int K, int V> __global__ void __launch_bounds__(128) causal_forward_kernel(CausalArgs<IO> a) {
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  const int groups = a.C / V;
  const int c = (int)(id % groups) * V;
  const long long r = id / groups;
  const int b = (int)(r / a.strips);
  if (b >= a.B) return;
  const int t0 = (int)(r % a.strips) * CAUSAL_STRIP;
  const int t1 = min(t0 + CAUSAL_STRIP, a.T), len = row_length(a.lengths, b, a.T);
  float w[K][V], bias[V], win[K][V];
  causal_taps<IO, K, V>(a, c, w, bias);
  const int stop = min(t1, len);
  if (t0 < len) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) causal_input<IO, K, V>(a, b, (long long)t0 - (K - 1) + j, c, win[j]);
  }
  // the state after the pass, by the threads of the first strip, which alone
  // read the one before it (the two may be the same memory)
  if (t0 == 0 && a.state_out && K > 1) {
    float s[K][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) causal_input<IO, K, V>(a, b, (long long)len - (K - 1) + j, c, s[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_pack<IO, V>(a.state_out + ((long long)b * (K - 1) + j) * a.C + c, s[j]);
  }
#pragma unroll 4
  for (int t = t0; t < stop; ++t) {
    load_pack<IO, V>(a.x.at(b, t) + c, win[K - 1]);
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float p = bias[i];
#pragma unroll
      for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
      o[i] = a.silu ? p * sigmoid(p) : p;
    }
    store_pack<IO, V>(a.y.at(b, t) + c, o);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
  }
  const float zero[V] = {};
  for (int t = max(t0, stop); t < t1; ++t) store_pack<IO, V>(a.y.at(b, t) + c, zero);
}

// Gradients.  At token t: g = dy silu'(p); the gradient of the input at
// t - (k-1) is then complete: sum_j w[j] g[t-j], plus that of the state after
// the pass where that state holds the input.  A strip [t0, t1) walks the
// tokens t0 .. t1+k-2 and sums dw and dbias over its own tokens only.  Block:
// 32 threads along the channels, 8 strips; the strips' sums are joined in
// order and go to the workspace.
template <typename IO, int K, int V> __global__ void __launch_bounds__(256) causal_backward_kernel(CausalArgs<IO> a) {
  __shared__ float sums[CAUSAL_GY][32 * V];
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int cblocks = (a.C / V + 31) / 32;
  const int cb = blockIdx.x % cblocks;
  const long long r = blockIdx.x / cblocks;
  const int b = (int)(r / a.strips);
  const long long t0 = (r % a.strips * CAUSAL_GY + y) * CAUSAL_GSTRIP;
  const int c = (cb * 32 + lane) * V;
  const int len = row_length(a.lengths, b, a.T);
  float dw[K][V] = {}, db[V] = {};
  if (c < a.C && t0 < a.T) {
    const long long t1 = min(t0 + CAUSAL_GSTRIP, (long long)a.T);
    float w[K][V], bias[V], win[K][V] = {}, g[K][V] = {};
    causal_taps<IO, K, V>(a, c, w, bias);
    if (t0 < len) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) causal_input<IO, K, V>(a, b, t0 - (K - 1) + j, c, win[j]);
    }
#pragma unroll 2
    for (long long t = t0; t < t1 + K - 1; ++t) {
      if (t < len) {
        float d[V];
        load_pack<IO, V>(a.x.at(b, t) + c, win[K - 1]);
        load_pack<IO, V>(a.dy.at(b, t) + c, d);
        const bool mine = t < t1;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (a.silu) {
            float p = bias[i];
#pragma unroll
            for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
            d[i] *= dsilu(p, sigmoid(p));
          }
          g[K - 1][i] = d[i];
          if (mine) {
            db[i] += d[i];
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][i] = fmaf(d[i], win[j][i], dw[j][i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) g[K - 1][i] = 0.f;
      }
      const long long s = t - (K - 1);  // the input whose gradient is complete
      if (s >= t0 || (t0 == 0 && K > 1)) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j) v = fmaf(w[j][i], g[K - 1 - j][i], v);
          o[i] = v;
        }
        if (a.dstate_out && t >= len && t < (long long)len + K - 1) {
          float d[V];
          load_pack<IO, V>(a.dstate_out + ((long long)b * (K - 1) + (t - len)) * a.C + c, d);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += d[i];
        }
        if (s >= 0)
          store_pack<IO, V>(a.dx.at(b, s) + c, o);
        else if (a.dstate)
          store_pack<IO, V>(a.dstate + ((long long)b * (K - 1) + (s + K - 1)) * a.C + c, o);
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          win[j][i] = win[j + 1][i];
          g[j][i] = g[j + 1][i];
        }
    }
  }
  // part[r][c][0..K-1] = dw, [K] = dbias
#pragma unroll
  for (int q = 0; q <= K; ++q) {
#pragma unroll
    for (int i = 0; i < V; ++i) sums[y][lane * V + i] = q < K ? dw[q][i] : db[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
      float v = sums[0][i];
#pragma unroll
      for (int k = 1; k < CAUSAL_GY; ++k) v += sums[k][i];
      const int cc = cb * 32 * V + i;
      if (cc < a.C) a.part[(r * a.C + cc) * (K + 1) + q] = v;
    }
    __syncthreads();
  }
}

// Where the sums of (c, q) go: q < K the taps, q = K the bias.
struct CausalSums {
  float *dw, *dbias;
  int K;
  __device__ __forceinline__ void put(long long i, float v) const {
    const long long c = i / (K + 1);
    const int q = (int)(i % (K + 1));
    if (q < K)
      dw[c * K + q] = v;
    else if (dbias)
      dbias[c] = v;
  }
};

// One token of every row: k-1 states and x read, y and the moved state written.
template <typename IO, int K, int V>
__global__ void __launch_bounds__(128) causal_step_kernel(CausalArgs<IO> a, const int* __restrict__ active) {
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  const int groups = a.C / V;
  const int c = (int)(id % groups) * V, b = (int)(id / groups);
  if (b >= a.B) return;
  float o[V] = {};
  if (!active || __ldg(active + b)) {
    float w[K][V], bias[V], win[K][V];
    IO* s = a.state_out + (long long)b * (K - 1) * a.C + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_pack<IO, V>(s + (long long)j * a.C, win[j]);
    load_pack<IO, V>(a.x.at(b, 0) + c, win[K - 1]);
    causal_taps<IO, K, V>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_pack<IO, V>(s + (long long)j * a.C, win[j + 1]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float p = bias[i];
#pragma unroll
      for (int j = 0; j < K; ++j) p = fmaf(w[j][i], win[j][i], p);
      o[i] = a.silu ? p * sigmoid(p) : p;
    }
  }
  store_pack<IO, V>(a.y.at(b, 0) + c, o);
}

}  // namespace wtseq
