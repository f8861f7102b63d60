// Norms before and after a block with its gate and residual scale.
//
// A block of threads holds one row at a time in registers, NV chunks of V
// channels a thread: each input is read once and each output written once.  A
// block goes through its rows with the parameters of its channels, and for the
// gradients the sums over the rows, in registers; where these fit (8 values a
// thread) the next row's inputs are on their way while a row is worked on.
//
// Memory is the floor.  8x2048x2048 bf16 with an fp32 residual and all parts:
// forward 82 us (5.7 TB/s, 88% of the floor), gradients 177 us (4.2 TB/s, 64%;
// 126 registers leave 16 warps an SM).  One row a block at a time, loads only
// when needed, took 141 and 487 us.
// Rows that begin at odd addresses go by single channels: 8x2048x2047 takes 177
// and 522 us (the gradients spill 72 bytes a thread).  Rows of more than 4096
// channels have 16 or 32 values a thread, loads only when needed, and spilled
// gradients (0.5 to 2.5 KB): 8x800x5120 203 and 530 us, floors 70 and 110;
// 8x256x16384 193 and 802 us, floors 72 and 113.
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

constexpr int NORM_WARPS = 16;  // of a block, at most
constexpr int NORM_THREADS = 1024, NORM_GRAD_THREADS = 512;  // of an SM

// Sums over the block of N values, for all of its threads.  `s`: N rows of
// NORM_WARPS floats, zero where there is no warp, which the block does not
// write again before two more barriers.
template <int N> __device__ __forceinline__ void block_sum(float (&v)[N], float (*s)[NORM_WARPS]) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) s[k][threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
#pragma unroll
  for (int w = 0; w < NORM_WARPS; w += 4) {
    if (w >= warps) break;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float4 u = *reinterpret_cast<const float4*>(s[k] + w);
      v[k] += (u.x + u.y) + (u.z + u.w);
    }
  }
}

// The rows that a block goes through: every gridDim.x-th.
struct NormRows {
  int left, b, t, db, dt, T;  // rows to go; the present one
  __device__ __forceinline__ NormRows(int B, int T) : T(T) {
    left = B * T - (int)blockIdx.x;
    b = blockIdx.x / T, t = blockIdx.x - b * T;
    db = gridDim.x / T, dt = gridDim.x - db * T;
  }
  __device__ __forceinline__ void next() {
    left -= gridDim.x, b += db, t += dt;
    if (t >= T) t -= T, ++b;
  }
};
template <typename IO> __device__ __forceinline__ IO* row_at(const Rows<IO>& r, int b, int t) {
  return r.p + b * r.sb + (long long)t * (int)r.st;
}

// The channels of a thread's chunk i: V neighbours, which are all there or none,
// or (WIDE = false, for rows that begin at odd addresses) V channels a block
// apart, so that each access of a warp is still one piece of the row.
template <int V, bool WIDE> struct Cols {
  static __device__ __forceinline__ int at(int i, int k) {
    return WIDE ? (i * blockDim.x + threadIdx.x) * V + k : (i * V + k) * blockDim.x + threadIdx.x;
  }
  static __device__ __forceinline__ bool none(int i, int C) { return at(i, 0) >= C; }
  template <typename IO> static __device__ __forceinline__ void store(IO* row, int i, int C, const float (&f)[V]) {
    if constexpr (WIDE) {
      store_pack<IO, V>(row + at(i, 0), f);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (at(i, k) < C) row[at(i, k)] = from_f<IO>(f[k]);
    }
  }
  template <typename IO> static __device__ __forceinline__ void load(const IO* row, int i, int C, Raw<IO, V>& r) {
    if constexpr (WIDE) {
      r.load(row + at(i, 0));
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) r.r[k / r.W].v[k % r.W] = at(i, k) < C ? __ldg(row + at(i, k)) : from_f<IO>(0.f);
    }
  }
};

// The fp32 parameters of a thread's channels, the product of two (one where
// there is none): kept in registers, or loaded where they are used.
template <int V, int NV, bool WIDE, bool KEEP> struct Params {
  const float *p, *p2;
  Vals<V> kept[KEEP ? NV : 1];
  int C;
  __device__ __forceinline__ Vals<V> load(int i) const {
    float f[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = Cols<V, WIDE>::at(i, k);
      f[k] = c < C ? (p ? __ldg(p + c) : 1.f) * (p2 ? __ldg(p2 + c) : 1.f) : 0.f;
    }
    Vals<V> v;
    v.set(f);
    return v;
  }
  __device__ __forceinline__ Params(const float* p, const float* p2, int C) : p(p), p2(p2), C(C) {
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < NV; ++i) kept[i] = load(i);
    }
  }
  __device__ __forceinline__ Vals<V> get(int i) const {
    if constexpr (KEEP)
      return kept[i];
    else
      return load(i);
  }
};

// One row of an input as it lies in memory.
template <typename IO, int V, int NV, bool WIDE> struct RowIn {
  Raw<IO, V> r[NV];
  __device__ __forceinline__ void load(const Rows<IO>& in, int b, int t, int C) {
    if (!in.p) return;
    const IO* p = row_at(in, b, t);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!Cols<V, WIDE>::none(i, C)) Cols<V, WIDE>::load(p, i, C, r[i]);
    }
  }
};

// NT: the most threads of a block.  Rows of 8 values a thread run at 64
// registers, which fills an SM with 1024 threads (8 values of fp32 with an fp32
// residual spill 16 bytes for that, odd rows 48 to 56).
template <typename IO, typename RES, int V, int NV, bool WIDE, int NT>
__global__ void __launch_bounds__(NT, V * NV <= 8 ? NORM_THREADS / NT : 1) norm_forward_kernel(NormArgs<IO, RES> a) {
  constexpr bool AHEAD = V * NV <= 8;
  __shared__ __align__(16) float sums[2][2][1][NORM_WARPS];
  for (int i = threadIdx.x; i < 4 * NORM_WARPS; i += blockDim.x) sums[0][0][0][i] = 0.f;
  __syncthreads();
  const float per = 1.f / a.C;
  const Params<V, NV, WIDE, AHEAD> sw(a.w, a.scale, a.C), w_res(a.w_res, nullptr, a.C);  // res_out = res + sw u n1
  RowIn<IO, V, NV, WIDE> x, gate;
  RowIn<RES, V, NV, WIDE> res;
  NormRows now(a.B, a.T), then = now;  // the row to work on, and to load
  auto load = [&] {
    const int b = then.b, t = then.t;
    if (then.left <= 0 || t >= row_length(a.lengths, b, a.T)) return;
    x.load(a.x, b, t, a.C);
    gate.load(a.gate, b, t, a.C);
    res.load(a.res, b, t, a.C);
  };
  if (AHEAD) load(), then.next();
  int turn = 0;
  for (; now.left > 0; now.next()) {
    const int b = now.b, t = now.t;
    const bool live = t < row_length(a.lengths, b, a.T);
    if (!AHEAD) load(), then.next();
    float u[NV][V], r[NV][V];
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) u[i][k] = r[i][k] = 0.f;
        if (Cols<V, WIDE>::none(i, a.C)) continue;
        x.r[i].floats(u[i]);
        if (a.gate.p) {
          float g[V];
          gate.r[i].floats(g);
#pragma unroll
          for (int k = 0; k < V; ++k) u[i][k] *= g[k] * sigmoid(g[k]);
        }
        if (a.res.p) res.r[i].floats(r[i]);
      }
    }
    if (AHEAD) load(), then.next();
    if (!live) {
      const float zero[V] = {};
      for (int i = 0; i < NV; ++i) {
        if (Cols<V, WIDE>::none(i, a.C)) continue;
        if (a.y.p) Cols<V, WIDE>::store(row_at(a.y, b, t), i, a.C, zero);
        if (a.res_out.p) Cols<V, WIDE>::store(row_at(a.res_out, b, t), i, a.C, zero);
      }
      continue;
    }
    turn ^= 1;  // rows without barriers do not count
    float n1 = 1.f, n2 = 1.f;
    if (a.w) {
      float q[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) q[0] = fmaf(u[i][k], u[i][k], q[0]);
      block_sum(q, sums[turn][0]);
      n1 = rsqrtf(fmaf(q[0], per, a.eps));
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Cols<V, WIDE>::none(i, a.C)) continue;
      float f[V];
      sw.get(i).get(f);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        u[i][k] = fmaf(f[k], u[i][k] * n1, r[i][k]);
        q[0] = fmaf(u[i][k], u[i][k], q[0]);
      }
      if (a.res.p) Cols<V, WIDE>::store(row_at(a.res_out, b, t), i, a.C, u[i]);
    }
    if (a.w_res) {
      block_sum(q, sums[turn][1]);
      n2 = rsqrtf(fmaf(q[0], per, a.eps));
    }
    if (!a.y.p) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Cols<V, WIDE>::none(i, a.C)) continue;
      float f[V];
      if (a.w_res) {
        w_res.get(i).get(f);
#pragma unroll
        for (int k = 0; k < V; ++k) u[i][k] *= n2 * f[k];
      }
      Cols<V, WIDE>::store(row_at(a.y, b, t), i, a.C, u[i]);
    }
  }
}

// Gradients.  With t = dy w_res:
//   dr = dres_out + n2 t - r n2^3 mean(r t)      dw_res = sum dy r n2
//   dres = dr   S = sum dr u n1   dscale = S w   dw = S scale
//   du = n1 q - u n1^3 mean(u q), q = dr scale w
//   dx = du silu(gate)   dgate = du x silu'(gate)
// Without res, dr is dy.  dscale and dw share the sum over the rows, and scale
// and w are only needed as their product until the end.
template <typename IO, typename RES, int V, int NV, bool WIDE>
__global__ void __launch_bounds__(512, 1) norm_backward_kernel(NormArgs<IO, RES> a) {
  constexpr bool AHEAD = V * NV <= 8, KEEP = AHEAD;
  constexpr int P = Vals<V>::P;
  __shared__ __align__(16) float s1[2][1][NORM_WARPS], s2[2][2][NORM_WARPS], s3[2][1][NORM_WARPS];
  for (int i = threadIdx.x; i < 2 * NORM_WARPS; i += blockDim.x) s1[0][0][i] = s2[0][0][i] = s2[1][0][i] = s3[0][0][i] = 0.f;
  __syncthreads();
  const float per = 1.f / a.C;
  const Params<V, NV, WIDE, KEEP> sw(a.w, a.scale, a.C), w_res(a.w_res, nullptr, a.C);
  Vals<V> as[NV], ar[NV];  // S and dw_res
#pragma unroll
  for (int i = 0; i < NV; ++i) as[i].zero(), ar[i].zero();
  RowIn<IO, V, NV, WIDE> x, gate, dy;
  RowIn<RES, V, NV, WIDE> res, dres;
  NormRows now(a.B, a.T), then = now;  // the row to work on, and to load
  auto load = [&] {
    const int b = then.b, t = then.t;
    if (then.left <= 0 || t >= row_length(a.lengths, b, a.T)) return;
    x.load(a.x, b, t, a.C);
    gate.load(a.gate, b, t, a.C);
    res.load(a.res, b, t, a.C);
    dy.load(a.dy, b, t, a.C);
    dres.load(a.dres_out, b, t, a.C);
  };
  auto vals = [](const auto& raw) {
    float f[V];
    raw.floats(f);
    Vals<V> v;
    v.set(f);
    return v;
  };
  auto total = [](f32x2 v) {
    float lo, hi;
    unpair(v, lo, hi);
    return lo + hi;
  };
  if (AHEAD) load(), then.next();
  int turn = 0;
  for (; now.left > 0; now.next()) {
    const int b = now.b, t = now.t;
    const bool live = t < row_length(a.lengths, b, a.T);
    if (!AHEAD) load(), then.next();
    // u = x act; act = silu(gate) and xd = x silu'(gate) wait for the end
    Vals<V> u[NV], act[NV], xd[NV], r[NV], q[NV], g[NV];  // q: dy, then dr, then dr scale w
    f32x2 uu = 0;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        u[i].zero(), act[i].zero(), xd[i].zero(), r[i].zero(), q[i].zero(), g[i].zero();
        if (Cols<V, WIDE>::none(i, a.C)) continue;
        u[i] = vals(x.r[i]);
        if (a.gate.p) {
          act[i] = vals(gate.r[i]);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const f32x2 sg = sigmoid2(act[i].p[k]);
            xd[i].p[k] = mul2(u[i].p[k], dsilu2(act[i].p[k], sg));
            act[i].p[k] = mul2(act[i].p[k], sg);
            u[i].p[k] = mul2(u[i].p[k], act[i].p[k]);
          }
        }
#pragma unroll
        for (int k = 0; k < P; ++k) uu = fma2(u[i].p[k], u[i].p[k], uu);
        if (a.res.p) r[i] = vals(res.r[i]);
        if (a.dy.p) q[i] = vals(dy.r[i]);
        if (a.dres_out.p) g[i] = vals(dres.r[i]);
      }
    }
    if (AHEAD) load(), then.next();
    if (!live) {
      const float zero[V] = {};
      for (int i = 0; i < NV; ++i) {
        if (Cols<V, WIDE>::none(i, a.C)) continue;
        Cols<V, WIDE>::store(row_at(a.dx, b, t), i, a.C, zero);
        if (a.gate.p) Cols<V, WIDE>::store(row_at(a.dgate, b, t), i, a.C, zero);
        if (a.res.p) Cols<V, WIDE>::store(row_at(a.dres, b, t), i, a.C, zero);
      }
      continue;
    }
    turn ^= 1;  // rows without barriers do not count
    float n1 = 1.f;
    if (a.w) {
      float s[1] = {total(uu)};
      block_sum(s, s1[turn]);
      n1 = rsqrtf(fmaf(s[0], per, a.eps));
    }
    // from here on u is u n1
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < P; ++k) u[i].p[k] = mul2(u[i].p[k], twice(n1));
    if (a.res.p) {
      f32x2 rr = 0, rt = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (Cols<V, WIDE>::none(i, a.C)) continue;
        const Vals<V> f = sw.get(i), fr = w_res.get(i);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          r[i].p[k] = fma2(f.p[k], u[i].p[k], r[i].p[k]);
          rr = fma2(r[i].p[k], r[i].p[k], rr);
          rt = fma2(r[i].p[k], mul2(q[i].p[k], fr.p[k]), rt);
        }
      }
      float n2 = 0.f, m = 0.f;
      if (a.w_res) {
        float s[2] = {total(rr), total(rt)};
        block_sum(s, s2[turn]);
        n2 = rsqrtf(fmaf(s[0], per, a.eps));
        m = -s[1] * per * n2 * n2 * n2;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (Cols<V, WIDE>::none(i, a.C)) continue;
        const Vals<V> fr = w_res.get(i);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const f32x2 qn = mul2(q[i].p[k], twice(n2));  // zero without w_res, and m too
          ar[i].p[k] = fma2(qn, r[i].p[k], ar[i].p[k]);
          q[i].p[k] = fma2(r[i].p[k], twice(m), fma2(qn, fr.p[k], g[i].p[k]));
        }
        float f[V];
        q[i].get(f);
        Cols<V, WIDE>::store(row_at(a.dres, b, t), i, a.C, f);
      }
    }
    f32x2 uq = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Cols<V, WIDE>::none(i, a.C)) continue;
      const Vals<V> f = sw.get(i);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        as[i].p[k] = fma2(q[i].p[k], u[i].p[k], as[i].p[k]);
        q[i].p[k] = mul2(q[i].p[k], f.p[k]);
        uq = fma2(u[i].p[k], q[i].p[k], uq);
      }
    }
    if (a.w) {
      float s[1] = {total(uq)};
      block_sum(s, s3[turn]);
      const float m = -s[0] * per * n1;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) q[i].p[k] = fma2(u[i].p[k], twice(m), mul2(q[i].p[k], twice(n1)));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Cols<V, WIDE>::none(i, a.C)) continue;
      float f[V];
      if (a.gate.p) {
#pragma unroll
        for (int k = 0; k < P; ++k) {
          xd[i].p[k] = mul2(xd[i].p[k], q[i].p[k]);
          q[i].p[k] = mul2(q[i].p[k], act[i].p[k]);
        }
        xd[i].get(f);
        Cols<V, WIDE>::store(row_at(a.dgate, b, t), i, a.C, f);
      }
      q[i].get(f);
      Cols<V, WIDE>::store(row_at(a.dx, b, t), i, a.C, f);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (Cols<V, WIDE>::none(i, a.C)) continue;
    float* p = a.part + (long long)blockIdx.x * 3 * a.C;
    float f1[V], f2[V];
    as[i].get(f1), ar[i].get(f2);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = Cols<V, WIDE>::at(i, k);
      if (c >= a.C) continue;
      p[c] = f1[k] * (a.scale ? __ldg(a.scale + c) : 1.f);
      p[a.C + c] = f1[k] * (a.w ? __ldg(a.w + c) : 1.f);
      p[2 * a.C + c] = f2[k];
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
