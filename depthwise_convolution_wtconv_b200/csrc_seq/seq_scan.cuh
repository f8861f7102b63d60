// Selective state space scan: forward, gradients, one token.
//
// A block owns 32 channels (a lane each) of one batch row and SCAN_W warps
// that share out the N states; tokens go by in tiles of SCAN_T.  Per tile:
//   A  the warps share out the tokens and turn dt and x into delta and
//      delta x in shared memory, once for all states; b and c go there too;
//   B  each warp runs the recurrence of its states over the tile with delta
//      and the sums over its states in registers (state by state, so that the
//      sums over the states need no exchange between lanes);
//   C  the warps share out the tokens again, join the warps' sums and apply
//      d x and the gate.
// Tokens behind a row's length get delta = 0, x = 0: they leave h as it is.
#pragma once

#include "seq_common.cuh"

namespace wtseq {

constexpr int SCAN_T = 16;        // tokens of a tile
constexpr int SCAN_W = 4;         // warps of a block
constexpr int SCAN_R = SCAN_T / SCAN_W;  // tokens of a warp in A and C
constexpr int SCAN_LD = SCAN_T + 4;      // floats between states in the b, c tiles
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <typename IO> struct ScanArgs {
  Rows<IO> x, dt, z, b, c, y, dy, dx, ddt, dz;
  const float *a, *d, *dt_bias, *state;
  float* state_out;
  const float* dstate_out;
  float* dstate;
  const int* lengths;
  float* ckpt;               // [B][tiles][N][C] states before each tile
  float *part_b, *part_c;    // [C blocks][B][T][N]
  float *part_a;             // [B][C][N]
  float *part_d, *part_bias; // [B][C]
  int B, T, C, N, G, softplus;
  int blocks;  // blocks of 32 channels in a group
  int tiles;
};

// 2^v; relative error below 2^-22 (flushes results below 2^-126 to zero)
__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float step_size(float v, int use_softplus) { return use_softplus ? softplus(v) : v; }

// b or c of the tile's tokens as [n][t] floats, zero behind the length.
template <typename IO>
__device__ __forceinline__ void scan_load_bc(const Rows<IO>& r, int b, int g, int t0, int len, int N, float* s) {
  for (int i = threadIdx.x; i < SCAN_T * N; i += SCAN_W * 32) {
    const int t = i / N, n = i - t * N;
    s[n * SCAN_LD + t] = t0 + t < len ? to_f<IO>(r.at(b, t0 + t)[(long long)g * N + n]) : 0.f;
  }
}

// Forward pass; with CKPT, the states before each tile instead of y.
template <typename IO, bool CKPT> __global__ void __launch_bounds__(SCAN_W * 32) scan_forward_kernel(ScanArgs<IO> p) {
  extern __shared__ float smem[];
  const int N = p.N, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* sd = smem;                        // [T][32] delta
  float* sx = sd + SCAN_T * 32;            // [T][32] delta x
  float* sy = sx + SCAN_T * 32;            // [W][T][32] sums over a warp's states
  float* sb = sy + (CKPT ? 0 : SCAN_W * SCAN_T * 32);  // [N][LD]
  float* sc = sb + N * SCAN_LD;
  float* sa = sc + N * SCAN_LD;            // [N][32] a log2(e)
  float* sh = sa + N * 32;                 // [N][32] h
  const int per = p.C / p.G;
  const int blk = blockIdx.x % (p.blocks * p.G), b = blockIdx.x / (p.blocks * p.G);
  const int g = blk / p.blocks, off = (blk % p.blocks) * 32 + lane;
  const bool on = off < per;
  const int c = g * per + (on ? off : 0);
  const int len = row_length(p.lengths, b, p.T);
  const float bias = p.dt_bias ? __ldg(p.dt_bias + c) : 0.f, dskip = p.d ? __ldg(p.d + c) : 0.f;
  for (int n = warp; n < N; n += SCAN_W) {
    sa[n * 32 + lane] = __ldg(p.a + (long long)c * N + n) * LOG2E;
    sh[n * 32 + lane] = p.state ? p.state[((long long)b * p.C + c) * N + n] : 0.f;
  }
  for (int t0 = 0; t0 < len; t0 += SCAN_T) {
    float xr[SCAN_R], zr[SCAN_R];
#pragma unroll
    for (int i = 0; i < SCAN_R; ++i) {
      const int t = warp * SCAN_R + i;
      float delta = 0.f;
      xr[i] = zr[i] = 0.f;
      if (on && t0 + t < len) {
        xr[i] = to_f<IO>(p.x.at(b, t0 + t)[c]);
        if (!CKPT && p.z.p) zr[i] = to_f<IO>(p.z.at(b, t0 + t)[c]);
        delta = step_size(to_f<IO>(p.dt.at(b, t0 + t)[c]) + bias, p.softplus);
      }
      sd[t * 32 + lane] = delta;
      sx[t * 32 + lane] = delta * xr[i];
    }
    scan_load_bc<IO>(p.b, b, g, t0, len, N, sb);
    if (!CKPT) scan_load_bc<IO>(p.c, b, g, t0, len, N, sc);
    __syncthreads();
    float de[SCAN_T], dx[SCAN_T], y[SCAN_T];
#pragma unroll
    for (int t = 0; t < SCAN_T; ++t) {
      de[t] = sd[t * 32 + lane];
      dx[t] = sx[t * 32 + lane];
      y[t] = 0.f;
    }
    for (int n = warp; n < N; n += SCAN_W) {
      const float a = sa[n * 32 + lane];
      float h = sh[n * 32 + lane];
      if (CKPT && on) p.ckpt[(((long long)b * p.tiles + t0 / SCAN_T) * N + n) * p.C + c] = h;
#pragma unroll
      for (int t = 0; t < SCAN_T; ++t) {
        h = fmaf(exp2_approx(de[t] * a), h, dx[t] * sb[n * SCAN_LD + t]);
        if (!CKPT) y[t] = fmaf(sc[n * SCAN_LD + t], h, y[t]);
      }
      sh[n * 32 + lane] = h;
    }
    if (!CKPT) {
#pragma unroll
      for (int t = 0; t < SCAN_T; ++t) sy[(warp * SCAN_T + t) * 32 + lane] = y[t];
    }
    __syncthreads();
    if (!CKPT) {
#pragma unroll
      for (int i = 0; i < SCAN_R; ++i) {
        const int t = warp * SCAN_R + i;
        if (!on || t0 + t >= len) continue;
        float v = dskip * xr[i];
#pragma unroll
        for (int w = 0; w < SCAN_W; ++w) v += sy[(w * SCAN_T + t) * 32 + lane];
        if (p.z.p) v *= zr[i] * sigmoid(zr[i]);
        p.y.at(b, t0 + t)[c] = from_f<IO>(v);
      }
    }
  }
  if constexpr (!CKPT) {
    if (!on) return;
    for (int t = len + warp; t < p.T; t += SCAN_W) p.y.at(b, t)[c] = from_f<IO>(0.f);
    if (p.state_out)
      for (int n = warp; n < N; n += SCAN_W) p.state_out[((long long)b * p.C + c) * N + n] = sh[n * 32 + lane];
  }
}

// v[i] summed over the 32 lanes, for 32 values at once: lane l returns the
// sum of v[l].  Each turn halves the values and the lanes that they lie on.
__device__ __forceinline__ float transpose_sum(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// Gradients, tiles last to first, from the states before each tile.  With
// dp = dy silu(z), e_t = c_t dp_t + a_{t+1} e_{t+1} (the gradient of h_t) and
// k_t = a_t h_{t-1} (what is kept of the state):
//   dc = sum_c dp h   db = sum_c e delta x   da = sum e k delta
//   ddelta = sum_n e (a k + b x)   dx = d dp + delta sum_n e b
template <typename IO> __global__ void __launch_bounds__(SCAN_W * 32) scan_backward_kernel(ScanArgs<IO> p) {
  extern __shared__ float smem[];
  const int N = p.N, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* sd = smem;                       // [T][32] delta
  float* sx = sd + SCAN_T * 32;           // [T][32] delta x
  float* sg = sx + SCAN_T * 32;           // [T][32] dp
  float* sy = sg + SCAN_T * 32;           // [3][W][T][32]: y, sum e a k, sum e b
  float* sb = sy + 3 * SCAN_W * SCAN_T * 32;
  float* sc = sb + N * SCAN_LD;
  float* sa = sc + N * SCAN_LD;           // [N][32] a log2(e)
  float* se = sa + N * 32;                // [N][32] e from the tile behind, decayed
  float* sda = se + N * 32;               // [N][32] da
  const int per = p.C / p.G;
  const int blk = blockIdx.x % (p.blocks * p.G), b = blockIdx.x / (p.blocks * p.G);
  const int g = blk / p.blocks, off = (blk % p.blocks) * 32 + lane;
  const bool on = off < per;
  const int c = g * per + (on ? off : 0);
  const int len = row_length(p.lengths, b, p.T);
  const float bias = p.dt_bias ? __ldg(p.dt_bias + c) : 0.f, dskip = p.d ? __ldg(p.d + c) : 0.f;
  float acc_d = 0.f, acc_bias = 0.f;
  for (int n = warp; n < N; n += SCAN_W) {
    sa[n * 32 + lane] = __ldg(p.a + (long long)c * N + n) * LOG2E;
    se[n * 32 + lane] = on && p.dstate_out ? p.dstate_out[((long long)b * p.C + c) * N + n] : 0.f;
    sda[n * 32 + lane] = 0.f;
  }
  // [C blocks of the group][B][T][N] partial sums over this block's channels
  const long long part0 = (((long long)(blk % p.blocks) * p.G + g) * p.B + b) * p.T;
  for (int tile = (len + SCAN_T - 1) / SCAN_T - 1; tile >= 0; --tile) {
    const int t0 = tile * SCAN_T;
    float xr[SCAN_R], zr[SCAN_R], vr[SCAN_R], gr[SCAN_R];
#pragma unroll
    for (int i = 0; i < SCAN_R; ++i) {
      const int t = warp * SCAN_R + i;
      float delta = 0.f, dp = 0.f;
      xr[i] = zr[i] = vr[i] = gr[i] = 0.f;
      if (on && t0 + t < len) {
        xr[i] = to_f<IO>(p.x.at(b, t0 + t)[c]);
        vr[i] = to_f<IO>(p.dt.at(b, t0 + t)[c]) + bias;
        gr[i] = dp = to_f<IO>(p.dy.at(b, t0 + t)[c]);
        if (p.z.p) {
          zr[i] = to_f<IO>(p.z.at(b, t0 + t)[c]);
          dp *= zr[i] * sigmoid(zr[i]);
        }
        delta = step_size(vr[i], p.softplus);
      }
      sd[t * 32 + lane] = delta;
      sx[t * 32 + lane] = delta * xr[i];
      sg[t * 32 + lane] = dp;
    }
    scan_load_bc<IO>(p.b, b, g, t0, len, N, sb);
    scan_load_bc<IO>(p.c, b, g, t0, len, N, sc);
    __syncthreads();
    float y[SCAN_T] = {}, ek[SCAN_T] = {}, eb[SCAN_T] = {};
    for (int n = warp; n < N; n += SCAN_W) {
      const float a = sa[n * 32 + lane];
      float h = on ? p.ckpt[(((long long)b * p.tiles + tile) * N + n) * p.C + c] : 0.f;
      float av[SCAN_T], kv[SCAN_T], v[32];
#pragma unroll
      for (int t = 0; t < SCAN_T; ++t) {
        av[t] = exp2_approx(sd[t * 32 + lane] * a);
        kv[t] = av[t] * h;
        h = fmaf(sx[t * 32 + lane], sb[n * SCAN_LD + t], kv[t]);
        y[t] = fmaf(sc[n * SCAN_LD + t], h, y[t]);
        v[16 + t] = sg[t * 32 + lane] * h;
      }
      float e = se[n * 32 + lane], da = 0.f;
#pragma unroll
      for (int t = SCAN_T - 1; t >= 0; --t) {
        e = fmaf(sc[n * SCAN_LD + t], sg[t * 32 + lane], e);
        v[t] = e * sx[t * 32 + lane];
        const float q = e * kv[t];
        ek[t] = fmaf(a, q, ek[t]);
        da = fmaf(sd[t * 32 + lane], q, da);
        eb[t] = fmaf(e, sb[n * SCAN_LD + t], eb[t]);
        e *= av[t];
      }
      se[n * 32 + lane] = e;
      sda[n * 32 + lane] += da;
      const float sum = transpose_sum(v);
      const int t = lane & 15;
      if (t0 + t < len) (lane < 16 ? p.part_b : p.part_c)[(part0 + t0 + t) * N + n] = sum;
    }
#pragma unroll
    for (int t = 0; t < SCAN_T; ++t) {
      sy[(warp * SCAN_T + t) * 32 + lane] = y[t];
      sy[((SCAN_W + warp) * SCAN_T + t) * 32 + lane] = ek[t];
      sy[((2 * SCAN_W + warp) * SCAN_T + t) * 32 + lane] = eb[t];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SCAN_R; ++i) {
      const int t = warp * SCAN_R + i;
      if (!on || t0 + t >= len) continue;
      float yv = dskip * xr[i], ekv = 0.f, ebv = 0.f;
#pragma unroll
      for (int w = 0; w < SCAN_W; ++w) {
        yv += sy[(w * SCAN_T + t) * 32 + lane];
        ekv += sy[((SCAN_W + w) * SCAN_T + t) * 32 + lane];
        ebv += sy[((2 * SCAN_W + w) * SCAN_T + t) * 32 + lane];
      }
      const float dp = sg[t * 32 + lane], delta = sd[t * 32 + lane];
      if (p.z.p) {
        const float s = sigmoid(zr[i]);
        p.dz.at(b, t0 + t)[c] = from_f<IO>(gr[i] * yv * dsilu(zr[i], s));
      }
      p.dx.at(b, t0 + t)[c] = from_f<IO>(fmaf(dskip, dp, delta * ebv));
      float dv = fmaf(xr[i], ebv, LN2 * ekv);
      if (p.softplus) dv *= sigmoid(vr[i]);
      p.ddt.at(b, t0 + t)[c] = from_f<IO>(dv);
      acc_d = fmaf(dp, xr[i], acc_d);
      acc_bias += dv;
    }
    __syncthreads();
  }
  // rows behind the length
  for (int t = len + warp; t < p.T; t += SCAN_W) {
    if (on) {
      p.dx.at(b, t)[c] = from_f<IO>(0.f);
      p.ddt.at(b, t)[c] = from_f<IO>(0.f);
      if (p.z.p) p.dz.at(b, t)[c] = from_f<IO>(0.f);
    }
    for (int n = lane; n < N; n += 32) p.part_b[(part0 + t) * N + n] = p.part_c[(part0 + t) * N + n] = 0.f;
  }
  for (int n = warp; n < N; n += SCAN_W) {
    if (!on) continue;
    p.part_a[((long long)b * p.C + c) * N + n] = sda[n * 32 + lane];
    if (p.dstate) p.dstate[((long long)b * p.C + c) * N + n] = se[n * 32 + lane];
  }
  sy[warp * 32 + lane] = acc_d;
  sy[(SCAN_W + warp) * 32 + lane] = acc_bias;
  __syncthreads();
  if (warp < 2 && on) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < SCAN_W; ++w) v += sy[(warp * SCAN_W + w) * 32 + lane];
    (warp ? p.part_bias : p.part_d)[(long long)b * p.C + c] = v;
  }
}

// One token of every row: four threads share a channel's states, each a
// quarter of them, and join their sums over the four.
template <typename IO>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs<IO> p, const int* __restrict__ active) {
  const long long id = (long long)blockIdx.x * 128 + threadIdx.x;
  const long long ch = id >> 2;
  const int q = (int)(id & 3);
  const int b = (int)min(ch / p.C, (long long)p.B - 1), c = (int)(ch % p.C);
  const bool on = ch < (long long)p.B * p.C;
  const bool live = on && (!active || __ldg(active + b));
  float y = 0.f, x = 0.f;
  if (live) {
    const int N = p.N, g = c / (p.C / p.G);
    x = to_f<IO>(p.x.at(b, 0)[c]);
    const float delta =
        step_size(to_f<IO>(p.dt.at(b, 0)[c]) + (p.dt_bias ? __ldg(p.dt_bias + c) : 0.f), p.softplus);
    const IO* bv = p.b.at(b, 0) + (long long)g * N;
    const IO* cv = p.c.at(b, 0) + (long long)g * N;
    float* h = p.state_out + ((long long)b * p.C + c) * N;
    for (int n = q; n < N; n += 4) {
      const float v = fmaf(exp2_approx(delta * (__ldg(p.a + (long long)c * N + n) * LOG2E)), h[n], delta * x * to_f<IO>(bv[n]));
      h[n] = v;
      y = fmaf(to_f<IO>(cv[n]), v, y);
    }
  }
  y += __shfl_xor_sync(0xffffffffu, y, 1);
  y += __shfl_xor_sync(0xffffffffu, y, 2);
  if (!on || q) return;
  if (live) {
    y = fmaf(p.d ? __ldg(p.d + c) : 0.f, x, y);
    if (p.z.p) {
      const float z = to_f<IO>(p.z.at(b, 0)[c]);
      y *= z * sigmoid(z);
    }
  }
  p.y.at(b, 0)[c] = from_f<IO>(y);
}

}  // namespace wtseq
