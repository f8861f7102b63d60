// Selective state space scan: forward, gradients, one token.
//
// A block owns 32 channels (a lane each) of one batch row and SCAN_W warps
// that share out the N states; tokens go by in tiles of SCAN_T.  Per tile:
//   A  the warps share out the tokens and turn dt and x into delta and
//      delta x in shared memory, once for all states; b and c go there too;
//   B  each warp runs the recurrence of its J states, which live in registers,
//      four tokens at a time: J independent chains of multiply-adds, and sums
//      over the warp's states without an exchange between lanes;
//   C  the warps share out the tokens again, join the warps' sums and apply
//      d x and the gate.
// Tokens behind a row's length get delta = 0, x = 0: they leave h as it is.
//
// Rows of which there are too few to fill the GPU are cut into chunks of
// tiles, each chunk a block: a first pass finds each chunk's state from a zero
// start and its sum of delta (the decay over the chunk is exp(a sum delta)),
// and every chunk of the second pass joins those before it into its start.
#pragma once

#include "seq_common.cuh"

namespace wtseq {

constexpr int SCAN_T = 16;        // tokens of a tile
constexpr int SCAN_W = 4;         // warps of a block
constexpr int SCAN_R = SCAN_T / SCAN_W;  // tokens of a warp in A and C: one float4
constexpr int SCAN_LD = SCAN_T + 4;      // floats between states in the b, c tiles
constexpr int SCAN_SLOTS = 4;            // tiles of inputs in shared memory
static_assert(SCAN_R == 4, "a thread's tokens of a tile are one float4");

template <typename IO> struct ScanArgs {
  Rows<IO> x, dt, z, b, c, y, dy, dx, ddt, dz;
  const float *a, *d, *dt_bias, *state;
  float* state_out;
  const float* dstate_out;
  float* dstate;
  const int* lengths;
  float* ends;               // [chunks][B][N][C] states after each chunk from a zero start
  float* sums;               // [chunks][B][C] sums of delta over each chunk
  float* ckpt;               // [B][tiles][N][C] states before each tile
  float *part_b, *part_c;    // [C blocks][B][T][N]
  float *part_a;             // [B][C][N]
  float *part_d, *part_bias; // [B][C]
  int B, T, C, N, G, softplus;
  int blocks;       // blocks of 32 channels in a group
  int tiles;        // of a row
  int chunks;       // of a row
  int chunk_tiles;  // of a chunk
  int wide_x;       // 16-byte copies of the channels' rows
  int wide_bc;      // ... and of the rows of b and c
};

// The hardware's 2^v is low by 1.8e-8 on average for -0.5 < v < 0 (measured;
// less than half a step).  Over the hundreds of tokens that a slow state
// remembers that adds up, so exponents are raised by as much in the same
// multiply-add that forms them.
constexpr float EXP_BIAS = 1.8e-8f * 1.4426950408889634f;

__device__ __forceinline__ float step_size(float v, int use_softplus) { return use_softplus ? softplus(v) : v; }

__device__ __forceinline__ void copy16(void* dst, const void* src, bool valid) {  // zeros where not valid
  const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// A lane's share of the copies of one input, tile by tile, 16 bytes at a time
// where the rows suit that: pointers that only move on.  Tokens behind the
// length become zeros.  `wide` decides between the two forms below.
template <typename IO> struct RowCopy {  // [SCAN_T][32 channels]
  static constexpr int E = 16 / sizeof(IO), PER = 32 / E, ROWS = 32 / PER;  // elements, chunks a row, rows a pass
  const IO* p;
  int left, st, at;  // tokens left from the lane's first one on (none for a lane outside the channels)
  __device__ __forceinline__ RowCopy(const Rows<IO>& r, int b, int t0, int stop, long long col, long long width, bool wide) {
    const int lane = threadIdx.x & 31, t = wide ? lane / PER : 0, k = wide ? lane % PER * E : lane;
    const bool ok = col + k < width;
    p = r.at(b, t0 + t) + (ok ? col + k : 0);
    left = ok ? stop - t0 - t : 0;
    st = (int)r.st;
    at = t * 32 + k;
  }
  __device__ __forceinline__ void tile(bool wide, IO* s) {
    if (wide) {
#pragma unroll
      for (int k = 0; k < SCAN_T; k += ROWS) copy16(s + at + k * 32, p + (long long)k * st, k < left);
    } else {
#pragma unroll 4
      for (int k = 0; k < SCAN_T; ++k) s[at + k * 32] = k < left ? p[(long long)k * st] : from_f<IO>(0.f);
    }
    left -= SCAN_T;
    p += (long long)SCAN_T * st;
  }
};
template <typename IO> struct StateCopy {  // [SCAN_T][N states]
  static constexpr int E = 16 / sizeof(IO);
  const IO* p;
  int left, st, per, t, step;  // tokens left; chunks a row; the lane's first token, tokens a pass (0: not a whole number)
  __device__ __forceinline__ StateCopy(const Rows<IO>& r, int b, int t0, int stop, long long col, int N, bool wide) {
    const int lane = threadIdx.x & 31, e = wide ? E : 1;
    per = N / e;
    t = lane / per;
    step = 32 % per ? 0 : 32 / per;
    p = r.at(b, t0) + col;
    left = stop - t0;
    st = (int)r.st;
  }
  __device__ __forceinline__ void one(int t, int k, bool wide, int N, IO* s) const {
    if (wide)
      copy16(s + t * N + k, p + (long long)t * st + k, t < left);
    else
      s[t * N + k] = t < left ? p[(long long)t * st + k] : from_f<IO>(0.f);
  }
  __device__ __forceinline__ void tile(bool wide, int N, IO* s) {
    const int lane = threadIdx.x & 31, e = wide ? E : 1;
    if (step) {
      const int k = (lane - t * per) * e;
      for (int u = t; u < SCAN_T; u += step) one(u, k, wide, N, s);
    } else {
      for (int i = lane; i < SCAN_T * per; i += 32) one(i / per, i % per * e, wide, N, s);
    }
    left -= SCAN_T;
    p += (long long)SCAN_T * st;
  }
};

// b and c of a tile, [t][n], as fp32 [n][t]: a thread per token and two states.
template <typename IO, bool BOTH>
__device__ __forceinline__ void transpose_tiles(const IO* b, const IO* c, int N, float* tb, float* tc) {
  const int t = threadIdx.x % SCAN_T;
  if (N & 1) {
    for (int n = threadIdx.x / SCAN_T; n < N; n += SCAN_W * 32 / SCAN_T) {
      tb[n * SCAN_LD + t] = to_f<IO>(b[t * N + n]);
      if (BOTH) tc[n * SCAN_LD + t] = to_f<IO>(c[t * N + n]);
    }
    return;
  }
  for (int n = threadIdx.x / SCAN_T * 2; n < N; n += SCAN_W * 64 / SCAN_T) {
    const Pack<IO, 2> u = *reinterpret_cast<const Pack<IO, 2>*>(b + t * N + n);
    tb[n * SCAN_LD + t] = to_f<IO>(u.v[0]);
    tb[(n + 1) * SCAN_LD + t] = to_f<IO>(u.v[1]);
    if (BOTH) {
      const Pack<IO, 2> v = *reinterpret_cast<const Pack<IO, 2>*>(c + t * N + n);
      tc[n * SCAN_LD + t] = to_f<IO>(v.v[0]);
      tc[(n + 1) * SCAN_LD + t] = to_f<IO>(v.v[1]);
    }
  }
}

// What a block works on.
struct ScanPlace {
  int b, g, c, chunk, len, tile0, tile1;  // tile1: behind the last tile with tokens
  long long col;                          // of the block's first channel
  bool on;                                // whether the lane has a channel
};
template <typename IO> __device__ __forceinline__ ScanPlace scan_place(const ScanArgs<IO>& p) {
  ScanPlace w;
  const int per = p.C / p.G, lane = threadIdx.x & 31;
  unsigned i = blockIdx.x;
  const int blk = i % (p.blocks * p.G);
  i /= p.blocks * p.G;
  w.chunk = i % p.chunks;
  w.b = i / p.chunks;
  w.g = blk / p.blocks;
  const int off = (blk % p.blocks) * 32;
  w.on = off + lane < per;
  w.col = (long long)w.g * per + off;
  w.c = (int)w.col + (w.on ? lane : 0);
  w.len = row_length(p.lengths, w.b, p.T);
  w.tile0 = w.chunk * p.chunk_tiles;
  w.tile1 = min(w.tile0 + p.chunk_tiles, (w.len + SCAN_T - 1) / SCAN_T);
  return w;
}

// h before the row's first token.  Where rows are cut it comes from the place
// of the last chunk's end, which nothing needs and where the first pass puts
// it: state_out may be the same memory as state.
template <typename IO> __device__ __forceinline__ float scan_first(const ScanArgs<IO>& p, const ScanPlace& w, int n) {
  return p.state ? p.state[((long long)w.b * p.C + w.c) * p.N + n] : 0.f;
}
// h before the block's chunk: the row's first state joined with the chunks before.
template <typename IO> __device__ __forceinline__ float scan_start(const ScanArgs<IO>& p, const ScanPlace& w, int n, float a) {
  if (p.chunks == 1) return scan_first(p, w, n);
  float h = p.ends[(((p.chunks - 1ll) * p.B + w.b) * p.N + n) * p.C + w.c];
  for (int k = 0; k < w.chunk; ++k) {
    const long long r = (long long)k * p.B + w.b;
    h = fmaf(exp2_approx(p.sums[r * p.C + w.c] * a), h, p.ends[(r * p.N + n) * p.C + w.c]);
  }
  return h;
}

enum { SCAN_Y, SCAN_ENDS, SCAN_CKPT };  // y; the chunks' ends and sums; the states before each tile

// Bytes of shared memory, and where its parts lie.
template <typename IO> struct ScanSmem {
  IO *x, *dt, *z, *b, *c;  // [slots][T][32 or N]
  float *de, *dx;          // [2][W][32] float4: delta, delta x
  float *y;                // [2][W][W][32] float4: sums over a warp's states
  float *tb, *tc;          // [2][NP][LD], NP: N rounded up to the warps' states
  __host__ __device__ ScanSmem(char* s, int N, int NP) {
    auto take = [&](size_t n) {
      char* r = s;
      s += (n + 15) / 16 * 16;
      return r;
    };
    const size_t row = SCAN_SLOTS * SCAN_T * 32 * sizeof(IO), bc = SCAN_SLOTS * SCAN_T * N * sizeof(IO);
    de = (float*)take(2 * SCAN_T * 32 * 4);
    dx = (float*)take(2 * SCAN_T * 32 * 4);
    y = (float*)take(2 * SCAN_W * SCAN_T * 32 * 4);
    tb = (float*)take(2 * NP * SCAN_LD * 4);
    tc = (float*)take(2 * NP * SCAN_LD * 4);
    x = (IO*)take(row);
    dt = (IO*)take(row);
    z = (IO*)take(row);
    b = (IO*)take(bc);
    c = (IO*)take(bc);
    end = s;
  }
  char* end;
};

// Turn k of the loop copies tile k+2, does C of tile k-1, B of tile k and A of
// tile k+1: none reads what another of the same turn writes, so one barrier a
// turn is enough and the warps' phases overlap.
template <typename IO, int MODE, int J>
__global__ void __launch_bounds__(SCAN_W * 32, J <= 4 ? 5 : (J <= 8 ? 4 : 2)) scan_forward_kernel(const ScanArgs<IO> p) {
  extern __shared__ __align__(16) char scan_smem[];
  constexpr int NP = J * SCAN_W;
  const int N = p.N, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n0 = warp * J;
  const ScanSmem<IO> s(scan_smem, N, NP);
  const ScanPlace w = scan_place(p);
  const bool gated = MODE == SCAN_Y && p.z.p;
  if (MODE == SCAN_ENDS && w.chunk == p.chunks - 1) {  // nothing comes after
    for (int n = warp; w.on && n < N; n += SCAN_W)
      p.ends[(((long long)w.chunk * p.B + w.b) * N + n) * p.C + w.c] = scan_first(p, w, n);
    return;
  }
  const float bias = p.dt_bias ? __ldg(p.dt_bias + w.c) : 0.f;
  const float dskip = MODE == SCAN_Y && p.d ? __ldg(p.d + w.c) : 0.f;

  // warp 0 copies x, 1 dt, 2 z, 3 b and c
  static_assert(SCAN_W == 4, "a warp for each input");
  const int first = w.tile0 * SCAN_T, count = max(0, w.tile1 - w.tile0);
  RowCopy<IO> rows(warp == 2 && gated ? p.z : (warp == 1 ? p.dt : p.x), w.b, first, w.len, w.col, p.C, p.wide_x);
  StateCopy<IO> rows_b(p.b, w.b, first, w.len, (long long)w.g * N, N, p.wide_bc);
  StateCopy<IO> rows_c(p.c, w.b, first, w.len, (long long)w.g * N, N, p.wide_bc);
  IO* const raw = warp == 0 ? s.x : (warp == 1 ? s.dt : s.z);
  // the phases count tiles from the block's first; copies go in order
  auto copy = [&](int k) {
    if (k < count) {
      const int slot = k % SCAN_SLOTS;
      if (warp < 2 || warp == 2 && gated) {
        rows.tile(p.wide_x, raw + slot * (SCAN_T * 32));
      } else if (warp == 3) {
        rows_b.tile(p.wide_bc, N, s.b + slot * SCAN_T * N);
        if (MODE == SCAN_Y) rows_c.tile(p.wide_bc, N, s.c + slot * SCAN_T * N);
      }
    }
    copies_commit();
  };
  float sum = 0.f;  // of this thread's delta
  const int mine = w.len - first - warp * SCAN_R;  // tokens from this thread's first one on
  auto phase_a = [&](unsigned k) {
    const int slot = k % SCAN_SLOTS, buf = k & 1;
    const IO* const dt = s.dt + (slot * SCAN_T + warp * SCAN_R) * 32 + lane;
    const IO* const x = s.x + (slot * SCAN_T + warp * SCAN_R) * 32 + lane;
    float de[SCAN_R];
#pragma unroll
    for (int i = 0; i < SCAN_R; ++i) de[i] = to_f<IO>(dt[i * 32]) + bias;
    if (p.softplus) {
#pragma unroll
      for (int i = 0; i < SCAN_R; ++i) de[i] = softplus(de[i]);
    }
    const int left = mine - (int)k * SCAN_T;
    if (left < SCAN_R) {
#pragma unroll
      for (int i = 0; i < SCAN_R; ++i) de[i] = i < left ? de[i] : 0.f;
    }
    if (MODE == SCAN_ENDS) sum += (de[0] + de[1]) + (de[2] + de[3]);
    reinterpret_cast<float4*>(s.de)[(buf * SCAN_W + warp) * 32 + lane] = make_float4(de[0], de[1], de[2], de[3]);
    reinterpret_cast<float4*>(s.dx)[(buf * SCAN_W + warp) * 32 + lane] =
        make_float4(de[0] * to_f<IO>(x[0]), de[1] * to_f<IO>(x[32]), de[2] * to_f<IO>(x[64]), de[3] * to_f<IO>(x[96]));
    transpose_tiles<IO, MODE == SCAN_Y>(s.b + slot * SCAN_T * N, s.c + slot * SCAN_T * N, N, s.tb + buf * (NP * SCAN_LD),
                                        s.tc + buf * (NP * SCAN_LD));
  };
  f32x2 a2[J];  // a log2(e), twice
  float h[J];
  const f32x2 bias2 = twice(EXP_BIAS);
  auto phase_b = [&](unsigned k) {
    const int buf = k & 1;
    if (MODE == SCAN_CKPT && w.on) {
      float* to = p.ckpt + (((long long)w.b * p.tiles + w.tile0 + k) * N + n0) * p.C + w.c;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (n0 + j < N) to[(long long)j * p.C] = h[j];
    }
    const ulonglong2* de = reinterpret_cast<const ulonglong2*>(s.de) + buf * SCAN_W * 32 + lane;
    const ulonglong2* dx = reinterpret_cast<const ulonglong2*>(s.dx) + buf * SCAN_W * 32 + lane;
    const float* tb = s.tb + (buf * NP + n0) * SCAN_LD;
    const float* tc = s.tc + (buf * NP + n0) * SCAN_LD;
#pragma unroll
    for (int q = 0; q < SCAN_T / 4; ++q) {
      const ulonglong2 d = de[q * 32], u = dx[q * 32];
      f32x2 y01 = 0, y23 = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const ulonglong2 bq = *reinterpret_cast<const ulonglong2*>(tb + j * SCAN_LD + 4 * q);
        const f32x2 e01 = fma2(d.x, a2[j], bias2), e23 = fma2(d.y, a2[j], bias2);
        const f32x2 b01 = mul2(u.x, bq.x), b23 = mul2(u.y, bq.y);
        float e0, e1, e2, e3, b0, b1, b2, b3;
        unpair(e01, e0, e1), unpair(e23, e2, e3), unpair(b01, b0, b1), unpair(b23, b2, b3);
        const float h0 = fmaf(exp2_approx(e0), h[j], b0), h1 = fmaf(exp2_approx(e1), h0, b1);
        const float h2 = fmaf(exp2_approx(e2), h1, b2);
        h[j] = fmaf(exp2_approx(e3), h2, b3);
        if (MODE == SCAN_Y) {
          const ulonglong2 cq = *reinterpret_cast<const ulonglong2*>(tc + j * SCAN_LD + 4 * q);
          y01 = fma2(cq.x, pair(h0, h1), y01);
          y23 = fma2(cq.y, pair(h2, h[j]), y23);
        }
      }
      if (MODE == SCAN_Y)
        reinterpret_cast<ulonglong2*>(s.y)[((buf * SCAN_W + warp) * SCAN_W + q) * 32 + lane] = make_ulonglong2(y01, y23);
    }
  };
  IO* out = MODE == SCAN_Y ? p.y.at(w.b, first + warp * SCAN_R) + w.c : nullptr;
  auto phase_c = [&](unsigned k) {  // in order
    const int slot = k % SCAN_SLOTS, buf = k & 1;
    const ulonglong2* part = reinterpret_cast<const ulonglong2*>(s.y) + (buf * SCAN_W * SCAN_W + warp) * 32 + lane;
    f32x2 u01 = part[0].x, u23 = part[0].y;
#pragma unroll
    for (int i = 1; i < SCAN_W; ++i) u01 = add2(u01, part[i * SCAN_W * 32].x), u23 = add2(u23, part[i * SCAN_W * 32].y);
    float v[SCAN_R];
    unpair(u01, v[0], v[1]), unpair(u23, v[2], v[3]);
    const IO* const x = s.x + (slot * SCAN_T + warp * SCAN_R) * 32 + lane;
    const IO* const z = s.z + (slot * SCAN_T + warp * SCAN_R) * 32 + lane;
#pragma unroll
    for (int i = 0; i < SCAN_R; ++i) v[i] = fmaf(dskip, to_f<IO>(x[i * 32]), v[i]);
    if (gated) {
#pragma unroll
      for (int i = 0; i < SCAN_R; ++i) {
        const float zv = to_f<IO>(z[i * 32]);
        v[i] *= zv * sigmoid(zv);
      }
    }
    const int left = w.on ? mine - (int)k * SCAN_T : 0, st = (int)p.y.st;
#pragma unroll
    for (int i = 0; i < SCAN_R; ++i)
      if (i < left) out[(long long)i * st] = from_f<IO>(v[i]);
    out += (long long)SCAN_T * st;
  };

  copy(0);
  copy(1);
  for (int i = threadIdx.x; i < 2 * (NP - N) * SCAN_LD; i += SCAN_W * 32) {  // states that are not there
    const int k = i / ((NP - N) * SCAN_LD), r = i % ((NP - N) * SCAN_LD) + (k * NP + N) * SCAN_LD;
    s.tb[r] = s.tc[r] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float a = n0 + j < N ? __ldg(p.a + (long long)w.c * N + n0 + j) * LOG2E : 0.f;
    a2[j] = twice(a);
    h[j] = MODE == SCAN_ENDS || n0 + j >= N ? 0.f : scan_start(p, w, n0 + j, a);
  }
  copies_wait<0>();
  __syncthreads();
  if (count) {
    phase_a(0);
    __syncthreads();
  }
  for (int k = 0; k < count; ++k) {
    copy(k + 2);
    if (MODE == SCAN_Y && k > 0) phase_c(k - 1);
    phase_b(k);
    if (k + 1 < count) phase_a(k + 1);
    copies_wait<0>();
    __syncthreads();
  }
  if constexpr (MODE == SCAN_Y) {
    if (count) phase_c(count - 1);
    if (!w.on) return;
    const int t1 = min((w.tile0 + p.chunk_tiles) * SCAN_T, p.T);
    for (int t = max(w.len, w.tile0 * SCAN_T) + warp; t < t1; t += SCAN_W) p.y.at(w.b, t)[w.c] = from_f<IO>(0.f);
    // the chunk with the row's last token, or the first of an empty row
    if (p.state_out && w.chunk == max(0, (w.len + SCAN_T - 1) / SCAN_T - 1) / p.chunk_tiles)
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (n0 + j < N) p.state_out[((long long)w.b * p.C + w.c) * N + n0 + j] = h[j];
  }
  if constexpr (MODE == SCAN_ENDS) {
    const long long r = (long long)w.chunk * p.B + w.b;
    s.y[warp * 32 + lane] = sum;
    __syncthreads();
    if (!w.on) return;
    if (warp == 0) {
#pragma unroll
      for (int k = 1; k < SCAN_W; ++k) sum += s.y[k * 32 + lane];
      p.sums[r * p.C + w.c] = sum;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (n0 + j < N) p.ends[(r * N + n0 + j) * p.C + w.c] = h[j];
  }
}

// b or c of the tile's tokens as [n][t] floats, zero behind the length.
template <typename IO>
__device__ __forceinline__ void scan_load_bc(const Rows<IO>& r, int b, int g, int t0, int len, int N, float* s) {
  for (int i = threadIdx.x; i < SCAN_T * N; i += SCAN_W * 32) {
    const int t = i / N, n = i - t * N;
    s[n * SCAN_LD + t] = t0 + t < len ? to_f<IO>(r.at(b, t0 + t)[(long long)g * N + n]) : 0.f;
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
