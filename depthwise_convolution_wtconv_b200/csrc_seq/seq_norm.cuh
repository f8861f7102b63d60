// Norms before and after a block with its gate and residual scale.
//
// A block of threads holds one row at a time in registers: NV chunks of V
// neighbouring channels a thread, each input read once and each output
// written once.  The gradients keep the sums over the rows for their channels
// in registers while the block goes through its rows.
#pragma once

#include "seq_common.cuh"

namespace wtseq {

template <typename IO, typename RES> struct NormArgs {
  Rows<IO> x, gate, y, dy, dx, dgate;
  Rows<RES> res, res_out, dres_out, dres;
  const float *w, *scale, *w_res;
  const int* lengths;
  float* part;  // [blocks][3][C]: dw, dscale, dw_res
  int B, T, C;
  float eps;
};

// Sum over the block, for all of its threads; `s` holds a float per warp and
// is not used again before a barrier.
__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
  for (int w = 0; w < warps; ++w) r += s[w];
  return r;
}

// One row's u and v: u = x silu(gate), n1 = 1 / sqrt(mean(u^2) + eps) (1
// without w), v = u n1 w.
template <typename IO, typename RES, int V, int NV>
__device__ __forceinline__ void norm_u(const NormArgs<IO, RES>& a, int b, int t, float (&u)[NV][V]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c >= a.C) {
#pragma unroll
      for (int k = 0; k < V; ++k) u[i][k] = 0.f;
      continue;
    }
    load_pack<IO, V>(a.x.at(b, t) + c, u[i]);
    if (a.gate.p) {
      float g[V];
      load_pack<IO, V>(a.gate.at(b, t) + c, g);
#pragma unroll
      for (int k = 0; k < V; ++k) u[i][k] *= g[k] * sigmoid(g[k]);
    }
  }
}

template <int V, int NV> __device__ __forceinline__ float squares(const float (&u)[NV][V]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) s = fmaf(u[i][k], u[i][k], s);
  return s;
}

template <int V> __device__ __forceinline__ void load_param(const float* p, int c, float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = __ldg(p + c + k);
}

template <typename IO, typename RES, int V, int NV>
__global__ void __launch_bounds__(V * NV <= 8 ? 256 : 512) norm_forward_kernel(NormArgs<IO, RES> a) {
  __shared__ float s1[32], s2[32];
  const int b = (int)(blockIdx.x / a.T), t = (int)(blockIdx.x % a.T);
  const float zero[V] = {};
  if (t >= row_length(a.lengths, b, a.T)) {
    for (int c = threadIdx.x * V; c < a.C; c += blockDim.x * V) {
      if (a.y.p) store_pack<IO, V>(a.y.at(b, t) + c, zero);
      if (a.res_out.p) store_pack<RES, V>(a.res_out.at(b, t) + c, zero);
    }
    return;
  }
  float u[NV][V];
  norm_u<IO, RES, V, NV>(a, b, t, u);
  if (a.w) {
    const float n1 = rsqrtf(block_sum(squares<V, NV>(u), s1) / a.C + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V;
      if (c >= a.C) continue;
      float w[V];
      load_param<V>(a.w, c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) u[i][k] *= n1 * w[k];
    }
  }
  float n2 = 1.f;
  if (a.res.p) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V;
      if (c >= a.C) continue;
      float r[V], sc[V];
      load_pack<RES, V>(a.res.at(b, t) + c, r);
#pragma unroll
      for (int k = 0; k < V; ++k) sc[k] = 1.f;
      if (a.scale) load_param<V>(a.scale, c, sc);
#pragma unroll
      for (int k = 0; k < V; ++k) u[i][k] = fmaf(sc[k], u[i][k], r[k]);
      store_pack<RES, V>(a.res_out.at(b, t) + c, u[i]);
    }
    if (!a.w_res) return;
    n2 = rsqrtf(block_sum(squares<V, NV>(u), s2) / a.C + a.eps);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c >= a.C) continue;
    if (a.w_res) {
      float w[V];
      load_param<V>(a.w_res, c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) u[i][k] *= n2 * w[k];
    }
    store_pack<IO, V>(a.y.at(b, t) + c, u[i]);
  }
}

// Gradients.  With t = dy w_res:
//   dr = dres_out + n2 t - r n2^3 mean(r t)      dw_res = sum dy r n2
//   dres = dr   dscale = sum dr v   q = dr scale (or dy, without res)
//   dw = sum q u n1   du = n1 q w - u n1^3 mean(u q w)
//   dx = du silu(gate)   dgate = du x silu'(gate)
template <typename IO, typename RES, int V, int NV>
__global__ void __launch_bounds__(V * NV <= 8 ? 256 : 512) norm_backward_kernel(NormArgs<IO, RES> a) {
  __shared__ float s[4][32];
  float aw[NV][V] = {}, as[NV][V] = {}, ar[NV][V] = {};
  const long long rows = (long long)a.B * a.T;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const int b = (int)(row / a.T), t = (int)(row % a.T);
    if (t >= row_length(a.lengths, b, a.T)) {
      const float zero[V] = {};
      for (int c = threadIdx.x * V; c < a.C; c += blockDim.x * V) {
        store_pack<IO, V>(a.dx.at(b, t) + c, zero);
        if (a.gate.p) store_pack<IO, V>(a.dgate.at(b, t) + c, zero);
        if (a.res.p) store_pack<RES, V>(a.dres.at(b, t) + c, zero);
      }
      continue;
    }
    float u[NV][V], q[NV][V], n1 = 1.f;
    norm_u<IO, RES, V, NV>(a, b, t, u);
    if (a.w) n1 = rsqrtf(block_sum(squares<V, NV>(u), s[0]) / a.C + a.eps);
    if (a.res.p) {
      float r[NV][V], n2 = 1.f, m = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= a.C) {
#pragma unroll
          for (int k = 0; k < V; ++k) r[i][k] = 0.f;
          continue;
        }
        float sc[V], w[V];
#pragma unroll
        for (int k = 0; k < V; ++k) sc[k] = w[k] = 1.f;
        load_pack<RES, V>(a.res.at(b, t) + c, r[i]);
        if (a.scale) load_param<V>(a.scale, c, sc);
        if (a.w) load_param<V>(a.w, c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) r[i][k] = fmaf(sc[k], u[i][k] * n1 * w[k], r[i][k]);
      }
      if (a.w_res) {
        n2 = rsqrtf(block_sum(squares<V, NV>(r), s[1]) / a.C + a.eps);
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * blockDim.x + threadIdx.x) * V;
          if (c >= a.C) continue;
          float w[V];
          load_pack<IO, V>(a.dy.at(b, t) + c, q[i]);
          load_param<V>(a.w_res, c, w);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            ar[i][k] = fmaf(q[i][k], r[i][k] * n2, ar[i][k]);
            q[i][k] *= w[k];
            d = fmaf(r[i][k], q[i][k], d);
          }
        }
        m = block_sum(d, s[2]) / a.C * n2 * n2 * n2;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= a.C) continue;
        float g[V] = {}, sc[V], w[V];
        if (a.dres_out.p) load_pack<RES, V>(a.dres_out.at(b, t) + c, g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          sc[k] = w[k] = 1.f;
          if (a.w_res) g[k] += n2 * q[i][k] - r[i][k] * m;
        }
        store_pack<RES, V>(a.dres.at(b, t) + c, g);
        if (a.scale) load_param<V>(a.scale, c, sc);
        if (a.w) load_param<V>(a.w, c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          as[i][k] = fmaf(g[k], u[i][k] * n1 * w[k], as[i][k]);
          q[i][k] = g[k] * sc[k];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c < a.C) load_pack<IO, V>(a.dy.at(b, t) + c, q[i]);
      }
    }
    if (a.w) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * V;
        if (c >= a.C) continue;
        float w[V];
        load_param<V>(a.w, c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          aw[i][k] = fmaf(q[i][k], u[i][k] * n1, aw[i][k]);
          q[i][k] *= w[k];
          d = fmaf(u[i][k], q[i][k], d);
        }
      }
      const float m = block_sum(d, s[3]) / a.C * n1 * n1 * n1;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) q[i][k] = n1 * q[i][k] - u[i][k] * m;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V;
      if (c >= a.C) continue;
      if (a.gate.p) {
        float x[V], g[V], dg[V];
        load_pack<IO, V>(a.x.at(b, t) + c, x);
        load_pack<IO, V>(a.gate.at(b, t) + c, g);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float sg = sigmoid(g[k]);
          dg[k] = q[i][k] * x[k] * dsilu(g[k], sg);
          q[i][k] *= g[k] * sg;
        }
        store_pack<IO, V>(a.dgate.at(b, t) + c, dg);
      }
      store_pack<IO, V>(a.dx.at(b, t) + c, q[i]);
    }
    __syncthreads();  // the next row's sums reuse s
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c >= a.C) continue;
    float* p = a.part + (long long)blockIdx.x * 3 * a.C + c;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      p[k] = aw[i][k];
      p[a.C + k] = as[i][k];
      p[2 * a.C + k] = ar[i][k];
    }
  }
}

struct NormSums {  // sums over the rows, [3][C], to the gradients that are wanted
  float *dw, *dscale, *dw_res;
  int C;
  __device__ __forceinline__ void put(long long i, float v) const {
    float* const to = i < C ? dw : (i < 2 * (long long)C ? dscale : dw_res);
    if (to) to[i % C] = v;
  }
};

}  // namespace wtseq
