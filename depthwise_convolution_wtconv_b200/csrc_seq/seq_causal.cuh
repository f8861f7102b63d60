// Causal depthwise convolution over tokens: forward, gradients, one token.
//
// Each thread owns V neighbouring channels and walks a strip of tokens with
// the last k-1 inputs, the taps and the sums in registers, so every input is
// read once but for the k-1 tokens before a strip.  Memory is the floor: 41 us
// for 4x4096x4096 bf16, k = 4, which takes 59 us (4.5 TB/s), the exponential
// and the quotient of silu being the next bound (30 us of their unit).  Four
// channels a thread: eight leave fewer warps than hide the loads (67 us).
// The gradients of 8x2048x2048 bf16 take 63 us (3.2 TB/s, floor 31): taps,
// two windows and the sums fill 126 registers a thread.
#pragma once

#include "seq_common.cuh"

namespace wtseq {

constexpr int CAUSAL_GY = 8;  // strips of a gradient block
// Tokens that the loops take in one piece, and whose loads are in flight: a
// multiple of the taps, so that the window of the last K inputs goes round in
// its registers and nothing is moved.  Forward at least 8, which keeps enough
// bytes in flight; the gradients load two inputs and have fewer registers left.
__host__ __device__ constexpr int causal_unroll(int K, int least) { return (least + K - 1) / K * K; }

template <typename IO> struct CausalArgs {
  Rows<IO> x, y, dy, dx;
  const float *w, *bias;
  const IO* state;  // [B][k-1][C], or null: zeros
  IO* state_out;
  const IO* dstate_out;
  IO* dstate;
  const int* lengths;
  float* part;  // [groups][C][K+1]
  int B, T, C, silu;
  int strip, strips;  // tokens of a thread; strips (gradients: blocks of strips) of a row
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
__device__ __forceinline__ void causal_taps(const CausalArgs<IO>& a, int c, Vals<V> (&w)[K], Vals<V>& bias) {
  float f[K][V], g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = a.bias ? __ldg(a.bias + c + i) : 0.f;
  bias.set(g);
  const float* p = a.w + (long long)c * K;  // V * K values in a row, 16-byte aligned where V is a multiple of 4
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int q = 0; q < V * K / 4; ++q) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(p) + q);
      const float e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[(q * 4 + i) % K][(q * 4 + i) / K] = e[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V * K; ++i) f[i % K][i / K] = __ldg(p + i);
  }
#pragma unroll
  for (int j = 0; j < K; ++j) w[j].set(f[j]);
}

// sum_j w[j] win[(first + j) % K] + v, win a ring
template <int K, int V>
__device__ __forceinline__ Vals<V> causal_sum(const Vals<V> (&w)[K], const Vals<V> (&win)[K], int first, Vals<V> v) {
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int i = 0; i < Vals<V>::P; ++i) v.p[i] = fma2(w[j].p[i], win[(first + j) % K].p[i], v.p[i]);
  return v;
}
template <typename IO, int K, int V> __global__ void __launch_bounds__(128) causal_forward_kernel(CausalArgs<IO> a) {
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  const int groups = a.C / V;
  const int c = (int)(id % groups) * V;
  const long long r = id / groups;
  const int b = (int)(r / a.strips);
  if (b >= a.B) return;
  const int t0 = (int)(r % a.strips) * a.strip;
  const int t1 = min(t0 + a.strip, a.T), len = row_length(a.lengths, b, a.T);
  const int stop = min(t1, len);
  constexpr int U = causal_unroll(K, 8);
  const IO* in = a.x.at(b, t0) + c;  // of the next load: U tokens ahead of the work
  IO* out = a.y.at(b, t0) + c;
  const int xs = (int)a.x.st, ys = (int)a.y.st;
  Raw<IO, V> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i, in += xs)
    if (t0 + i < stop) raw[i].load(in);
  Vals<V> w[K], bias, win[K];
  causal_taps<IO, K, V>(a, c, w, bias);
  if (t0 < len) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float f[V];
      causal_input<IO, K, V>(a, b, (long long)t0 - (K - 1) + j, c, f);
      win[j].set(f);
    }
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
  for (int t = t0; t < stop; t += U) {
#pragma unroll
    for (int i = 0; i < U; ++i, in += xs, out += ys) {
      if (t + i >= stop) break;
      float f[V];
      raw[i].floats(f);
      if (t + U + i < stop) raw[i].load(in);
      win[(i + K - 1) % K].set(f);
      Vals<V> p = causal_sum<K, V>(w, win, i % K, bias);
      if (a.silu) {
#pragma unroll
        for (int v = 0; v < Vals<V>::P; ++v) p.p[v] = mul2(p.p[v], sigmoid2(p.p[v]));
      }
      p.get(f);
      store_pack<IO, V>(out, f);
    }
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
  constexpr int P = Vals<V>::P;
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int cblocks = (a.C / V + 31) / 32;
  const int cb = blockIdx.x % cblocks;
  const long long r = blockIdx.x / cblocks;
  const int b = (int)(r / a.strips);
  const long long first = (r % a.strips * CAUSAL_GY + y) * a.strip;
  const int c = (cb * 32 + lane) * V;
  const int len = row_length(a.lengths, b, a.T);
  Vals<V> dw[K], db;
#pragma unroll
  for (int j = 0; j < K; ++j) dw[j].zero();
  db.zero();
  if (c < a.C && first < a.T) {
    const int t0 = (int)first, t1 = (int)min(first + a.strip, (long long)a.T), stop = min(t1, len);
    constexpr int U = causal_unroll(K, 4);
    const int xs = (int)a.x.st, gs = (int)a.dy.st, os = (int)a.dx.st;
    const IO *in = a.x.at(b, t0) + c, *in_g = a.dy.at(b, t0) + c;  // of the next load
    IO* out = a.dx.at(b, (long long)t0 - (K - 1)) + c;              // of the input that is complete
    Raw<IO, V> rx[U], rg[U];
#pragma unroll
    for (int i = 0; i < U; ++i, in += xs, in_g += gs)
      if (t0 + i < stop) rx[i].load(in), rg[i].load(in_g);
    Vals<V> w[K], bias, win[K], g[K];  // rings: token t0 + i is win[(i + K - 1) % K] and g[K - 1 - i % K]
    causal_taps<IO, K, V>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < K; ++j) g[j].zero(), win[j].zero();
    if (t0 < len) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        float f[V];
        causal_input<IO, K, V>(a, b, (long long)t0 - (K - 1) + j, c, f);
        win[j].set(f);
      }
    }
    // g of token t0 + i from its x and dy
    auto gate = [&](int i, const float (&x)[V], const float (&dy)[V]) {
      win[(i + K - 1) % K].set(x);
      Vals<V>& d = g[K - 1 - i % K];
      d.set(dy);
      if (a.silu) {
        const Vals<V> p = causal_sum<K, V>(w, win, i % K, bias);
#pragma unroll
        for (int v = 0; v < P; ++v) d.p[v] = mul2(d.p[v], dsilu2(p.p[v], sigmoid2(p.p[v])));
      }
    };
    // the gradient of the input at t0 + i - (K - 1): sum_j w[j] g of token t0 + i - j
    auto complete = [&](int i) {
      Vals<V> v;
      v.zero();
      return causal_sum<K, V>(w, g, K - 1 - i % K, v);
    };
    const bool top = t0 == 0 && a.dstate;
    for (int t = t0; t < stop; t += U) {
#pragma unroll
      for (int i = 0; i < U; ++i, in += xs, in_g += gs, out += os) {
        if (t + i >= stop) break;
        float x[V], dy[V];
        rx[i].floats(x), rg[i].floats(dy);
        if (t + U + i < stop) rx[i].load(in), rg[i].load(in_g);
        gate(i, x, dy);
#pragma unroll
        for (int v = 0; v < P; ++v) {
          const f32x2 d = g[K - 1 - i % K].p[v];
          db.p[v] = add2(db.p[v], d);
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j].p[v] = fma2(d, win[(i + j) % K].p[v], dw[j].p[v]);
        }
        float f[V];
        complete(i).get(f);
        if (t + i - t0 >= K - 1)
          store_pack<IO, V>(out, f);
        else if (top)
          store_pack<IO, V>(a.dstate + ((long long)b * (K - 1) + t + i) * a.C + c, f);
      }
    }
    // the tokens of the next strip that this one's inputs reach, and those behind the length
    const long long t2 = (long long)t1 + K - 1;
    const int from = max(t0, stop), phase = (from - t0) % K;
    for (long long t = from - phase; t < t2; t += K) {
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if (t + i < from || t + i >= t2) continue;
        if (t + i < len) {
          float x[V], dy[V];
          load_pack<IO, V>(a.x.at(b, t + i) + c, x), load_pack<IO, V>(a.dy.at(b, t + i) + c, dy);
          gate(i, x, dy);
        } else {
          g[K - 1 - i].zero();
        }
        const long long s = t + i - (K - 1);
        if (s < t0 && !top) continue;
        float f[V];
        complete(i).get(f);
        if (a.dstate_out && t + i >= len && t + i < (long long)len + K - 1) {
          float d[V];
          load_pack<IO, V>(a.dstate_out + ((long long)b * (K - 1) + (t + i - len)) * a.C + c, d);
#pragma unroll
          for (int v = 0; v < V; ++v) f[v] += d[v];
        }
        if (s >= t0)
          store_pack<IO, V>(a.dx.at(b, s) + c, f);
        else
          store_pack<IO, V>(a.dstate + ((long long)b * (K - 1) + (s + K - 1)) * a.C + c, f);
      }
    }
  }
  // part[r][c][0..K-1] = dw, [K] = dbias
#pragma unroll
  for (int q = 0; q <= K; ++q) {
    float f[V];
    if (q < K)
      dw[q < K ? q : 0].get(f);
    else
      db.get(f);
#pragma unroll
    for (int i = 0; i < V; ++i) sums[y][lane * V + i] = f[i];
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
    Vals<V> w[K], bias, u[K];
    float win[K][V];
    IO* s = a.state_out + (long long)b * (K - 1) * a.C + c;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_pack<IO, V>(s + (long long)j * a.C, win[j]);
    load_pack<IO, V>(a.x.at(b, 0) + c, win[K - 1]);
    causal_taps<IO, K, V>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_pack<IO, V>(s + (long long)j * a.C, win[j + 1]);
#pragma unroll
    for (int j = 0; j < K; ++j) u[j].set(win[j]);
    Vals<V> p = causal_sum<K, V>(w, u, 0, bias);
    if (a.silu) {
#pragma unroll
      for (int i = 0; i < Vals<V>::P; ++i) p.p[i] = mul2(p.p[i], sigmoid2(p.p[i]));
    }
    p.get(o);
  }
  store_pack<IO, V>(a.y.at(b, 0) + c, o);
}

}  // namespace wtseq
