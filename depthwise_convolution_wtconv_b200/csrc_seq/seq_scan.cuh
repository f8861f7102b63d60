// Selective state space scan: forward, gradients, one token.
//
// A block owns 32 channels (a lane each) of one batch row; its W warps share
// out the N states, SCAN_J each in registers.  Tokens go by in tiles of
// SCAN_T.  Per tile:
//   A  the warps share out the tokens and turn dt and x into delta and
//      delta x in shared memory, once for all states; b and c go there too;
//   B  each warp runs the recurrence of its states, four tokens at a time:
//      SCAN_J independent chains of multiply-adds, and sums over the warp's
//      states without an exchange between lanes;
//   C  the warps share out the tokens again, join the warps' sums and apply
//      d x and the gate.
// Tokens behind a row's length get delta = 0, x = 0: they leave h as it is.
//
// Bound by instructions: 610 a warp and tile, 274 of them B (16 values: per
// value an exponential, half a packed multiply-add each for its argument, the
// input and the sum, a multiply-add for h), the rest A, C and the copies, once
// for all states.  8x2048x2048 bf16 with 16 states: 286 us, where its 537 M
// exponentials alone take 115 us and its bytes 41 us.  Four states a warp: four
// chains keep the multiply-adds busy, and the warps together halve the share
// of A and C; delta of a whole tile in registers instead took 315 us.
//
// Rows of which there are too few to fill the GPU are cut into chunks of
// tiles, each chunk a block: a first pass finds each chunk's state from a zero
// start and its sum of delta (the decay over the chunk is exp(a sum delta)),
// and every chunk of the second pass joins those before it into its start.
// The gradients do the same from the other end.
#pragma once

#include "seq_common.cuh"

namespace wtseq {

constexpr int SCAN_T = 16;           // tokens of a tile
constexpr int SCAN_J = 4;            // states of a warp
constexpr int SCAN_S = 8;            // tokens between the states kept for the gradients
constexpr int SCAN_LD = SCAN_T + 4;  // floats between states in the b, c tiles
constexpr int SCAN_SLOTS = 4;        // tiles of inputs in shared memory, forward
constexpr int SCAN_GSLOTS = 3;       // ... gradients

template <typename IO> struct ScanArgs {
  Rows<IO> x, dt, z, b, c, y, dy, dx, ddt, dz;
  const float *a, *d, *dt_bias, *state;
  float* state_out;
  const float* dstate_out;
  float* dstate;
  const int* lengths;
  float* ends;               // [chunks][B][N][C] states after each chunk from a zero start
  float* sums;               // [chunks][B][C] sums of delta over each chunk
  float* grad_ends;          // [chunks][B][N][C] their gradients before each chunk, from zero behind it
  float* ckpt;               // [B][tiles * SCAN_T / SCAN_S][N][C] states before every SCAN_S tokens
  float *part_b, *part_c;    // [C blocks][B][T][N]
  float *part_a;             // [chunks][B][C][N]
  float *part_d, *part_bias; // [chunks][B][C]
  int B, T, C, N, G, softplus;
  int group, states;  // channels and states of a group as x, dt, z, dy and b, c hold them (rounded up if copied)
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

template <int BYTES> __device__ __forceinline__ void copy_async(void* dst, const void* src, bool valid) {  // zeros where not valid
  const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
  const int n = valid ? BYTES : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
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
// where the rows begin at such addresses (`wide`), one by one where not:
// pointers that only move on.  Tokens behind the length become zeros.
template <typename IO> struct RowCopy {  // [SCAN_T][32 channels]
  static constexpr int E = 16 / sizeof(IO), PER = 32 / E, ROWS = 32 / PER;  // elements, chunks a row, rows a pass
  const IO* p;
  int left, st, at;  // tokens left from the lane's first one on (for a lane outside the channels never any)
  __device__ __forceinline__ RowCopy() {}
  __device__ __forceinline__ RowCopy(const Rows<IO>& r, int b, int t0, int stop, long long col, long long width, bool wide) {
    const int lane = threadIdx.x & 31, t = wide ? lane / PER : 0, k = wide ? lane % PER * E : lane;
    const bool ok = col + k < width;
    p = r.at(b, t0 + t) + (ok ? col + k : 0);
    left = ok ? stop - t0 - t : -(1 << 30);
    st = (int)r.st;
    at = t * 32 + k;
  }
  __device__ __forceinline__ void tile(bool wide, int dir, IO* s) {  // then on to the next (1) or the one before (-1)
    if (wide) {
#pragma unroll
      for (int k = 0; k < SCAN_T; k += ROWS) copy16(s + at + k * 32, p + (long long)k * st, k < left);
    } else {
      IO v[SCAN_T];
#pragma unroll
      for (int k = 0; k < SCAN_T; ++k) v[k] = k < left ? __ldg(p + (long long)k * st) : from_f<IO>(0.f);
#pragma unroll
      for (int k = 0; k < SCAN_T; ++k) s[at + k * 32] = v[k];
    }
    left -= dir * SCAN_T;
    p += (long long)(dir * SCAN_T) * st;
  }
};
// The tiles of b or c, [SCAN_T][states]: the chunks of a row (four states, or
// one), and the lane's first token and state; `step` tokens a pass (0: not a whole number).
struct StateLanes {
  int per, t, k, step;
  __device__ __forceinline__ StateLanes(int N, int e) {
    const int lane = threadIdx.x & 31;
    per = N / e;
    t = lane / per;
    k = (lane - t * per) * e;
    step = 32 % per ? 0 : 32 / per;
  }
};
template <typename IO>
__device__ __forceinline__ void copy_states(const StateLanes& l, const Rows<IO>& r, const IO* p, int left, bool wide, int N, IO* s) {
  const int st = (int)r.st;
  auto one = [&](int t, int k) {
    if (wide)
      copy_async<4 * sizeof(IO)>(s + t * N + k, p + (long long)t * st + k, t < left);
    else
      s[t * N + k] = t < left ? p[(long long)t * st + k] : from_f<IO>(0.f);
  };
  if (l.step) {
    for (int u = l.t; u < SCAN_T; u += l.step) one(u, l.k);
  } else {
    const int e = wide ? 4 : 1;
    for (int i = threadIdx.x & 31; i < SCAN_T * l.per; i += 32) one(i / l.per, i % l.per * e);
  }
}

// The copies that a warp makes of a tile: the inputs r = 0 .. R-1 and then b
// and c are dealt to the warps in turn.
template <typename IO, int W, int R> struct TileCopies {
  static constexpr int MINE = (R + W - 1) / W;
  RowCopy<IO> rows[MINE];
  int to[MINE];  // the input's place among the slots, which follow one another; -1: none
  StateLanes lanes;
  const IO *bc, *other;  // the warp's next tile of b or c (of b and of c, where a block is one warp)
  int left;      // tokens from there on
  __device__ __forceinline__ TileCopies(const ScanArgs<IO>& p, const Rows<IO> (&in)[R], int row, int t0, int stop, long long col,
                                        int g)
      : lanes(p.states, p.wide_bc ? 4 : 1), left(stop - t0) {
    const int warp = threadIdx.x >> 5;
    bc = (W == 1 || warp == R % W ? p.b : p.c).at(row, t0) + (long long)g * p.states;
    other = p.c.at(row, t0) + (long long)g * p.states;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      Rows<IO> r = in[0];
      to[i] = -1;
#pragma unroll
      for (int k = i * W; k < R && k < (i + 1) * W; ++k)
        if (k == i * W + warp) r = in[k], to[i] = k;
      if (!r.p) to[i] = -1;
      if (to[i] >= 0) rows[i] = RowCopy<IO>(r, row, t0, stop, col, (long long)p.G * p.group, p.wide_x);
    }
  }
  __device__ __forceinline__ void tile(const ScanArgs<IO>& p, int slot, int slots, int dir, IO* x, IO* to_b, IO* to_c) {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < MINE; ++i)
      if (to[i] >= 0) rows[i].tile(p.wide_x, dir, x + (to[i] * slots + slot) * (SCAN_T * 32));
    if (W == 1) {  // both
      if (to_b) copy_states<IO>(lanes, p.b, bc, left, p.wide_bc, p.states, to_b + slot * SCAN_T * p.states);
      if (to_c) copy_states<IO>(lanes, p.c, other, left, p.wide_bc, p.states, to_c + slot * SCAN_T * p.states);
      other += (long long)(dir * SCAN_T) * (int)p.c.st;
    } else if (to_b && warp == R % W) {
      copy_states<IO>(lanes, p.b, bc, left, p.wide_bc, p.states, to_b + slot * SCAN_T * p.states);
    } else if (to_c && warp == (R + 1) % W) {
      copy_states<IO>(lanes, p.c, bc, left, p.wide_bc, p.states, to_c + slot * SCAN_T * p.states);
    }
    bc += (long long)(dir * SCAN_T) * (int)(W == 1 || warp == R % W ? p.b : p.c).st;
    left -= dir * SCAN_T;
  }
};

// b, c or both of a tile, [t][n] with n a multiple of four, as fp32 [n][t]: a
// thread per token and two states.
template <typename IO, int W, bool HAS_B, bool HAS_C>
__device__ __forceinline__ void transpose_tiles(const IO* b, const IO* c, int N, float* tb, float* tc) {
  const int t = threadIdx.x % SCAN_T;
  for (int n = threadIdx.x / SCAN_T * 2; n < N; n += W * 64 / SCAN_T) {
    if (HAS_B) {
      const Pack<IO, 2> u = *reinterpret_cast<const Pack<IO, 2>*>(b + t * N + n);
      tb[n * SCAN_LD + t] = to_f<IO>(u.v[0]);
      tb[(n + 1) * SCAN_LD + t] = to_f<IO>(u.v[1]);
    }
    if (HAS_C) {
      const Pack<IO, 2> v = *reinterpret_cast<const Pack<IO, 2>*>(c + t * N + n);
      tc[n * SCAN_LD + t] = to_f<IO>(v.v[0]);
      tc[(n + 1) * SCAN_LD + t] = to_f<IO>(v.v[1]);
    }
  }
}

// Copies of inputs whose rows cannot be read 16 bytes at a time, because a
// group's channels (or states) are no multiple of that: [B][T][G][to], the
// group rounded up and filled with zeros.  A thread makes E elements; block
// row y is input y.
template <typename IO> struct ScanPad {
  Rows<IO> in[6];
  IO* out[6];
  int from[6], to[6];  // channels or states of a group
  const int* lengths;
  int B, T, G;
};
template <typename IO> __global__ void __launch_bounds__(256) scan_pad_kernel(const ScanPad<IO> p) {
  constexpr int E = 4;
  const int k = blockIdx.y, from = p.from[k], to = p.to[k], per = p.G * to / E;
  const long long all = (long long)p.B * p.T * per;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const long long row = i / per;
    const int col = (int)(i - row * per) * E, g = col / to, o = col - g * to;
    const int b = (int)(row / p.T), t = (int)(row - (long long)b * p.T);
    if (t >= row_length(p.lengths, b, p.T)) continue;
    const IO* const r = p.in[k].at(b, t) + (long long)g * from;
    Pack<IO, E> v;
#pragma unroll
    for (int e = 0; e < E; ++e) v.v[e] = o + e < from ? __ldg(r + o + e) : from_f<IO>(0.f);
    *reinterpret_cast<Pack<IO, E>*>(p.out[k] + row * per * E + col) = v;
  }
}

// What a block works on.
struct ScanPlace {
  int b, g, c, chunk, len, tile0, tile1;  // tile1: behind the last tile with tokens
  long long col;                          // of the block's first channel, in x, dt, z and dy
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
  w.col = (long long)w.g * p.group + off;
  w.c = w.g * per + off + (w.on ? lane : 0);
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
// A state taken through n chunks, each 2^s h + end; part(i, s, end) gives them.
// 2^s may be beyond fp32 over a chunk where h 2^s is not (small states that
// grow, large ones that shrink, zero): what s has beyond 126 is a factor of its
// own.  Within it that is 1, and free (1x8192x2048 bf16: 235.3 us, 234.7
// without; a second loop for the rare case: 238.8).
template <typename F> __device__ __forceinline__ float scan_join(float first, int n, F part) {
  float h = first, s, end;
  for (int i = 0; i < n; ++i) {
    part(i, s, end);
    const float near = fmaxf(fminf(s, 126.f), -126.f), far = fminf(s - near, 126.f);
    h = fmaf(exp2_approx(near), exp2_approx(far) * h, end);
  }
  return h;
}
// h before the block's chunk: the row's first state joined with the chunks before.
template <typename IO> __device__ __forceinline__ float scan_start(const ScanArgs<IO>& p, const ScanPlace& w, int n, float a) {
  if (p.chunks == 1) return scan_first(p, w, n);
  return scan_join(p.ends[(((p.chunks - 1ll) * p.B + w.b) * p.N + n) * p.C + w.c], w.chunk, [&](int k, float& s, float& end) {
    const long long r = (long long)k * p.B + w.b;
    s = p.sums[r * p.C + w.c] * a, end = p.ends[(r * p.N + n) * p.C + w.c];
  });
}

// e behind the block's chunk: that of the row's last state joined with the chunks behind.
template <typename IO> __device__ __forceinline__ float scan_grad_start(const ScanArgs<IO>& p, const ScanPlace& w, int n, float a) {
  const float last = p.dstate_out ? p.dstate_out[((long long)w.b * p.C + w.c) * p.N + n] : 0.f;
  return scan_join(last, p.chunks - 1 - w.chunk, [&](int k, float& s, float& end) {
    const long long r = (p.chunks - 1ll - k) * p.B + w.b;
    s = p.sums[r * p.C + w.c] * a, end = p.grad_ends[(r * p.N + n) * p.C + w.c];
  });
}

// What a pass is for: y; the chunks' ends and sums; the states before every
// SCAN_S tokens; the gradients before each chunk (tokens last to first, with
// c dp in the place of b delta x).
enum { SCAN_Y, SCAN_ENDS, SCAN_CKPT, SCAN_GRAD_ENDS };

// A thread's tokens of a tile in A and C are R = SCAN_T / W neighbours, kept as
// [t / 4][lane][t % 4]: four tokens of a lane are one 16-byte access.
template <int R> __device__ __forceinline__ int token_slot(int t, int lane) { return ((t >> 2) * 32 + lane) * 4 + (t & 3); }
template <int R> __device__ __forceinline__ void put_tokens(float* s, const float (&v)[R]) {
  if constexpr (R >= 4) {
#pragma unroll
    for (int i = 0; i < R; i += 4) *reinterpret_cast<float4*>(s + i * 32) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else if constexpr (R == 2) {
    *reinterpret_cast<float2*>(s) = make_float2(v[0], v[1]);
  } else {
    s[0] = v[0];
  }
}
template <int R> __device__ __forceinline__ void get_tokens(const float* s, float (&v)[R]) {
  if constexpr (R >= 4) {
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(s + i * 32);
      v[i] = u.x, v[i + 1] = u.y, v[i + 2] = u.z, v[i + 3] = u.w;
    }
  } else if constexpr (R == 2) {
    const float2 u = *reinterpret_cast<const float2*>(s);
    v[0] = u.x, v[1] = u.y;
  } else {
    v[0] = s[0];
  }
}
// ... summed over the warps' parts
template <int W, int R> __device__ __forceinline__ void sum_tokens(const float* s, float (&v)[R]) {
  if constexpr (R >= 4) {
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      ulonglong2 u = *reinterpret_cast<const ulonglong2*>(s + i * 32);
#pragma unroll
      for (int w = 1; w < W; ++w) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(s + w * SCAN_T * 32 + i * 32);
        u.x = add2(u.x, x.x), u.y = add2(u.y, x.y);
      }
      unpair(u.x, v[i], v[i + 1]), unpair(u.y, v[i + 2], v[i + 3]);
    }
    return;
  }
  get_tokens<R>(s, v);
#pragma unroll
  for (int w = 1; w < W; ++w) {
    float u[R];
    get_tokens<R>(s + w * SCAN_T * 32, u);
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] += u[i];
  }
}

// Where the parts of the shared memory lie, and (end - start) its size.
template <typename IO> struct ScanSmem {
  float *de, *dx;          // [2][T/4][32] float4: delta, delta x
  float *y;                // [2][W][T/4][32] float4: sums over a warp's states
  float *tb, *tc;          // [2][NP][LD], NP: the warps' states
  IO *x, *dt, *z, *b, *c;  // [slots][T][32 or N], x to z one behind the other
  char* end;
  __host__ __device__ ScanSmem(char* s, int N, int W) {
    auto take = [&](size_t n) {
      char* r = s;
      s += (n + 15) / 16 * 16;
      return r;
    };
    const size_t row = SCAN_SLOTS * SCAN_T * 32 * sizeof(IO), bc = SCAN_SLOTS * SCAN_T * N * sizeof(IO);
    de = (float*)take(2 * SCAN_T * 32 * 4);
    dx = (float*)take(2 * SCAN_T * 32 * 4);
    y = (float*)take(2 * W * SCAN_T * 32 * 4);
    tb = (float*)take(2 * W * SCAN_J * SCAN_LD * 4);
    tc = (float*)take(2 * W * SCAN_J * SCAN_LD * 4);
    x = (IO*)take(row);
    dt = (IO*)take(row);
    z = (IO*)take(row);
    b = (IO*)take(bc);
    c = (IO*)take(bc);
    end = s;
  }
};

// Turn k of the loop copies tile k+2, does C of tile k-1, B of tile k and A of
// tile k+1: none reads what another of the same turn writes, so one barrier a
// turn is enough and the warps' phases overlap.
template <typename IO, int MODE, int W>
__global__ void __launch_bounds__(W * 32, W >= 16 ? 1 : 20 / W) scan_forward_kernel(const ScanArgs<IO> p) {
  extern __shared__ __align__(16) char scan_smem[];
  constexpr int J = SCAN_J, NP = J * W, R = SCAN_T / W;
  constexpr bool BACK = MODE == SCAN_GRAD_ENDS;
  constexpr int DIR = BACK ? -1 : 1;
  const int N = p.N, NS = p.states, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n0 = warp * J;
  const ScanSmem<IO> s(scan_smem, NS, W);
  const ScanPlace w = scan_place(p);
  const bool gated = (MODE == SCAN_Y || BACK) && p.z.p;
  if (BACK && w.chunk == 0) return;  // nothing comes before
  if (MODE == SCAN_ENDS && w.chunk == p.chunks - 1) {  // nothing comes after
    for (int n = warp; w.on && n < N; n += W)
      p.ends[(((long long)w.chunk * p.B + w.b) * N + n) * p.C + w.c] = scan_first(p, w, n);
    return;
  }
  const float bias = p.dt_bias ? __ldg(p.dt_bias + w.c) : 0.f;
  const float dskip = MODE == SCAN_Y && p.d ? __ldg(p.d + w.c) : 0.f;
  const int count = max(0, w.tile1 - w.tile0);
  const int first = max(0, BACK ? (w.tile1 - 1) * SCAN_T : w.tile0 * SCAN_T);  // token of the first tile to do
  const Rows<IO> none = {nullptr, 0, 0}, in[3] = {BACK ? p.dy : p.x, p.dt, gated ? p.z : none};
  TileCopies<IO, W, 3> copies(p, in, w.b, first, w.len, w.col, w.g);
  // the phases count tiles from the block's first to do; copies and C go in order
  auto copy = [&](int k) {
    if (k < count) copies.tile(p, k % SCAN_SLOTS, SCAN_SLOTS, DIR, s.x, BACK ? nullptr : s.b, MODE == SCAN_Y || BACK ? s.c : nullptr);
    copies_commit();
  };
  float sum = 0.f;                               // of this thread's delta
  const int mine = w.len - first - warp * R;     // tokens from this thread's first one on
  const int own = token_slot<R>(warp * R, lane);  // its place in a tile
  auto phase_a = [&](unsigned k) {
    const int slot = k % SCAN_SLOTS, buf = k & 1;
    const IO* const dt = s.dt + (slot * SCAN_T + warp * R) * 32 + lane;
    const IO* const x = s.x + (slot * SCAN_T + warp * R) * 32 + lane;
    float de[R], dx[R];
#pragma unroll
    for (int i = 0; i < R; ++i) de[i] = to_f<IO>(dt[i * 32]) + bias;
    if (p.softplus) {
#pragma unroll
      for (int i = 0; i < R; ++i) de[i] = softplus(de[i]);
    }
    const int left = mine - DIR * (int)k * SCAN_T;
    if (left < R) {
#pragma unroll
      for (int i = 0; i < R; ++i) de[i] = i < left ? de[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (MODE == SCAN_ENDS || BACK) sum += de[i];
      dx[i] = to_f<IO>(x[i * 32]);
      if (!BACK) {
        dx[i] *= de[i];
      } else if (gated) {
        const float z = to_f<IO>(s.z[(slot * SCAN_T + warp * R + i) * 32 + lane]);
        dx[i] *= z * sigmoid(z);
      }
    }
    put_tokens<R>(s.de + buf * SCAN_T * 32 + own, de);
    put_tokens<R>(s.dx + buf * SCAN_T * 32 + own, dx);
    transpose_tiles<IO, W, !BACK, MODE == SCAN_Y || BACK>(s.b + slot * SCAN_T * NS, s.c + slot * SCAN_T * NS, NS,
                                                          s.tb + buf * (NP * SCAN_LD), s.tc + buf * (NP * SCAN_LD));
  };
  f32x2 a2[J];  // a log2(e), twice
  float h[J];
  const f32x2 bias2 = twice(EXP_BIAS);
  auto phase_b = [&](unsigned k) {
    const int buf = k & 1;
    const ulonglong2* de = reinterpret_cast<const ulonglong2*>(s.de) + buf * SCAN_T * 8 + lane;
    const ulonglong2* dx = reinterpret_cast<const ulonglong2*>(s.dx) + buf * SCAN_T * 8 + lane;
    const float* tb = s.tb + (buf * NP + n0) * SCAN_LD;
    const float* tc = s.tc + (buf * NP + n0) * SCAN_LD;
    if constexpr (BACK) {
#pragma unroll
      for (int q = SCAN_T / 4 - 1; q >= 0; --q) {
        const ulonglong2 d = de[q * 32], u = dx[q * 32];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const ulonglong2 cq = *reinterpret_cast<const ulonglong2*>(tc + j * SCAN_LD + 4 * q);
          float e0, e1, e2, e3, c0, c1, c2, c3;
          unpair(fma2(d.x, a2[j], bias2), e0, e1), unpair(fma2(d.y, a2[j], bias2), e2, e3);
          unpair(mul2(u.x, cq.x), c0, c1), unpair(mul2(u.y, cq.y), c2, c3);
          h[j] = exp2_approx(e3) * (h[j] + c3);
          h[j] = exp2_approx(e2) * (h[j] + c2);
          h[j] = exp2_approx(e1) * (h[j] + c1);
          h[j] = exp2_approx(e0) * (h[j] + c0);
        }
      }
    } else {
#pragma unroll
    for (int q = 0; q < SCAN_T / 4; ++q) {
      if (MODE == SCAN_CKPT && q % (SCAN_S / 4) == 0 && w.on) {
        float* to = p.ckpt + ((((long long)w.b * p.tiles + w.tile0 + k) * SCAN_T + q * 4) / SCAN_S * N + n0) * p.C + w.c;
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (n0 + j < N) to[(long long)j * p.C] = h[j];
      }
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
        reinterpret_cast<ulonglong2*>(s.y)[((buf * W + warp) * (SCAN_T / 4) + q) * 32 + lane] = make_ulonglong2(y01, y23);
    }
    }
  };
  IO* out = MODE == SCAN_Y ? p.y.at(w.b, first + warp * R) + w.c : nullptr;
  auto phase_c = [&](unsigned k) {
    const int slot = k % SCAN_SLOTS, buf = k & 1;
    float v[R];
    sum_tokens<W, R>(s.y + buf * W * SCAN_T * 32 + own, v);
    const IO* const x = s.x + (slot * SCAN_T + warp * R) * 32 + lane;
    const IO* const z = s.z + (slot * SCAN_T + warp * R) * 32 + lane;
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = fmaf(dskip, to_f<IO>(x[i * 32]), v[i]);
    if (gated) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float zv = to_f<IO>(z[i * 32]);
        v[i] *= zv * sigmoid(zv);
      }
    }
    const int left = w.on ? mine - (int)k * SCAN_T : 0, st = (int)p.y.st;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < left) out[(long long)i * st] = from_f<IO>(v[i]);
    out += (long long)SCAN_T * st;
  };

  copy(0);
  copy(1);
  for (int i = threadIdx.x; i < 2 * (NP - NS) * SCAN_LD; i += W * 32) {  // states that are not there
    const int k = i / ((NP - NS) * SCAN_LD), r = i % ((NP - NS) * SCAN_LD) + (k * NP + NS) * SCAN_LD;
    s.tb[r] = s.tc[r] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float a = n0 + j < N ? __ldg(p.a + (long long)w.c * N + n0 + j) * LOG2E : 0.f;
    a2[j] = twice(a);
    h[j] = MODE == SCAN_ENDS || BACK || n0 + j >= N ? 0.f : scan_start(p, w, n0 + j, a);
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
    for (int t = max(w.len, first) + warp; t < t1; t += W) p.y.at(w.b, t)[w.c] = from_f<IO>(0.f);
    // the chunk with the row's last token, or the first of an empty row
    if (p.state_out && w.chunk == max(0, (w.len + SCAN_T - 1) / SCAN_T - 1) / p.chunk_tiles)
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (n0 + j < N) p.state_out[((long long)w.b * p.C + w.c) * N + n0 + j] = h[j];
  }
  if constexpr (MODE == SCAN_ENDS || BACK) {
    const long long r = (long long)w.chunk * p.B + w.b;
    s.y[warp * 32 + lane] = sum;
    __syncthreads();
    if (!w.on) return;
    if (warp == 0 && (!BACK || w.chunk == p.chunks - 1)) {  // the last chunk has no other pass that needs its sum
#pragma unroll
      for (int k = 1; k < W; ++k) sum += s.y[k * 32 + lane];
      p.sums[r * p.C + w.c] = sum;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (n0 + j < N) (BACK ? p.grad_ends : p.ends)[(r * N + n0 + j) * p.C + w.c] = h[j];
  }
}

// Gradients, tiles last to first, from the states before every SCAN_S tokens.
// With dp = dy silu(z), e_t = c_t dp_t + a_{t+1} e_{t+1} (the gradient of h_t)
// and k_t = a_t h_{t-1} (what is kept of the state):
//   dc = sum_c dp h   db = sum_c e delta x   da = sum e k delta
//   ddelta = sum_n e (a k + b x)   dx = d dp + delta sum_n e b
// The sums over the channels are sums over lanes.  They take an exchange a
// value, but no selecting, because register j of lane l holds the state
// j ^ (l & 3): neighbours that exchange two registers each complete one of the
// two states.  Only the quarter that remains after two such turns is summed by
// halving the values and the lanes that they lie on.
// 8x1024x2048 bf16, 16 states: 652 us with the pass that keeps the states (128
// us) and the sums (25 us); 2200 instructions a warp and tile at 0.45 a clock,
// 128 registers, of which 80 to 124 bytes a thread are spilled (448 in blocks of
// one warp).  fp32: 853 us.  Selecting in every turn, as for 32 values over 32
// lanes, cost two instructions more a value.
template <typename IO> struct ScanGradSmem {
  float *de, *dx, *dp;          // [T/4][32] float4: delta, delta x, dp
  float* y;                     // [3][W][T/4][32] float4: sums over a warp's states of c h, e a k, e b
  float *tb, *tc;               // [NP][LD]
  IO *x, *dt, *dy, *z, *b, *c;  // [slots][T][32 or N], x to z one behind the other
  char* end;
  __host__ __device__ ScanGradSmem(char* s, int N, int W) {
    auto take = [&](size_t n) {
      char* r = s;
      s += (n + 15) / 16 * 16;
      return r;
    };
    const size_t row = SCAN_GSLOTS * SCAN_T * 32 * sizeof(IO), bc = SCAN_GSLOTS * SCAN_T * N * sizeof(IO);
    de = (float*)take(SCAN_T * 32 * 4);
    dx = (float*)take(SCAN_T * 32 * 4);
    dp = (float*)take(SCAN_T * 32 * 4);
    y = (float*)take(3 * W * SCAN_T * 32 * 4);
    tb = (float*)take(W * SCAN_J * SCAN_LD * 4);
    tc = (float*)take(W * SCAN_J * SCAN_LD * 4);
    x = (IO*)take(row);
    dt = (IO*)take(row);
    dy = (IO*)take(row);
    z = (IO*)take(row);
    b = (IO*)take(bc);
    c = (IO*)take(bc);
    end = s;
  }
};

// The sums over the four lanes l ^ 0..3 of what they hold of one state, for
// the state of register 0: fed register by register.
__device__ __forceinline__ void quad_sum(int j, const float (&x)[4], float (&lo)[4], float (&hi)[4]) {
  float (&v)[4] = j < 2 ? lo : hi;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (j % 2 == 0)
      v[i] = x[i];
    else
      v[i] += __shfl_xor_sync(0xffffffffu, x[i], 1);
    if (j == 3) lo[i] += __shfl_xor_sync(0xffffffffu, hi[i], 2);
  }
}

template <typename IO, int W>
__global__ void __launch_bounds__(W * 32, W >= 16 ? 1 : 16 / W) scan_backward_kernel(const ScanArgs<IO> p) {
  extern __shared__ __align__(16) char scan_smem[];
  constexpr int J = SCAN_J, NP = J * W, R = SCAN_T / W;
  static_assert(J == 4 && SCAN_S == 8 && SCAN_T == 2 * SCAN_S, "the exchanges below are written for these");
  const int N = p.N, NS = p.states, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n0 = warp * J;
  const ScanGradSmem<IO> s(scan_smem, NS, W);
  const ScanPlace w = scan_place(p);
  const bool gated = p.z.p;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + w.c) : 0.f, dskip = p.d ? __ldg(p.d + w.c) : 0.f;
  const int count = max(0, w.tile1 - w.tile0), last = (w.tile0 + count - 1) * SCAN_T;
  const Rows<IO> in[4] = {p.x, p.dt, p.dy, p.z};
  TileCopies<IO, W, 4> copies(p, in, w.b, max(last, 0), w.len, w.col, w.g);
  // turn k works on the tile from token last - k * SCAN_T on
  auto copy = [&](int k) {
    if (k < count) copies.tile(p, k % SCAN_GSLOTS, SCAN_GSLOTS, -1, s.x, s.b, s.c);
    copies_commit();
  };
  const int own = token_slot<R>(warp * R, lane);
  float acc_d = 0.f, acc_bias = 0.f;
  auto phase_a = [&](int k) {
    const int at = (k % SCAN_GSLOTS * SCAN_T + warp * R) * 32 + lane;
    const int left = w.on ? w.len - (last - k * SCAN_T) - warp * R : 0;
    float de[R], dx[R], dp[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      de[i] = to_f<IO>(s.dt[at + i * 32]) + bias;
      dp[i] = to_f<IO>(s.dy[at + i * 32]);
    }
    if (p.softplus) {
#pragma unroll
      for (int i = 0; i < R; ++i) de[i] = softplus(de[i]);
    }
    if (gated) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float z = to_f<IO>(s.z[at + i * 32]);
        dp[i] *= z * sigmoid(z);
      }
    }
    if (left < R) {
#pragma unroll
      for (int i = 0; i < R; ++i) de[i] = i < left ? de[i] : 0.f, dp[i] = i < left ? dp[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) dx[i] = i < left ? de[i] * to_f<IO>(s.x[at + i * 32]) : 0.f;
    put_tokens<R>(s.de + own, de);
    put_tokens<R>(s.dx + own, dx);
    put_tokens<R>(s.dp + own, dp);
    transpose_tiles<IO, W, true, true>(s.b + k % SCAN_GSLOTS * SCAN_T * NS, s.c + k % SCAN_GSLOTS * SCAN_T * NS, NS, s.tb, s.tc);
  };

  // the states of this lane's registers
  int nj[J];
  f32x2 a2[J], da2[J];
  float e[J], kept[J];  // kept: states before the next SCAN_S tokens to do
  const f32x2 bias2 = twice(EXP_BIAS);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    nj[j] = n0 + (j ^ (lane & 3));
    const bool there = nj[j] < N;
    const float a = there ? __ldg(p.a + (long long)w.c * N + nj[j]) * LOG2E : 0.f;
    a2[j] = twice(a);
    e[j] = there && w.on ? scan_grad_start(p, w, nj[j], a) : 0.f;
    da2[j] = 0;
  }
  auto fetch = [&](int token) {
    const long long r = ((long long)w.b * p.tiles * SCAN_T + token) / SCAN_S;
#pragma unroll
    for (int j = 0; j < J; ++j) kept[j] = token >= 0 && nj[j] < N ? __ldg(p.ckpt + (r * N + nj[j]) * p.C + w.c) : 0.f;
  };
  // [C blocks of the group][B][T][N] partial sums over this block's channels
  const int blk = blockIdx.x % (p.blocks * p.G) % p.blocks;
  const long long part0 = (((long long)blk * p.G + w.g) * p.B + w.b) * p.T;
  float* const part = (lane & 16 ? p.part_c : p.part_b) + part0 * N + n0 + (lane & 3);
  auto phase_b = [&](int k) {
    const int t0 = last - k * SCAN_T;
#pragma unroll 1
    for (int sub = SCAN_T / SCAN_S - 1; sub >= 0; --sub) {
      const ulonglong2* de = reinterpret_cast<const ulonglong2*>(s.de) + sub * 64 + lane;
      const ulonglong2* dx = reinterpret_cast<const ulonglong2*>(s.dx) + sub * 64 + lane;
      const ulonglong2* dp = reinterpret_cast<const ulonglong2*>(s.dp) + sub * 64 + lane;
      ulonglong2* sy = reinterpret_cast<ulonglong2*>(s.y) + (warp * 4 + sub * 2) * 32 + lane;
      float h[J], v[16];  // v: db, then dc, of SCAN_S tokens
      f32x2 kv[2][J][2];
#pragma unroll
      for (int j = 0; j < J; ++j) h[j] = w.on ? kept[j] : 0.f;
      fetch(t0 + (sub - 1) * SCAN_S);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const ulonglong2 d = de[q * 32], u = dx[q * 32], g = dp[q * 32];
        f32x2 y01 = 0, y23 = 0;
        float lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const ulonglong2 bq = *reinterpret_cast<const ulonglong2*>(s.tb + nj[j] * SCAN_LD + sub * SCAN_S + 4 * q);
          const ulonglong2 cq = *reinterpret_cast<const ulonglong2*>(s.tc + nj[j] * SCAN_LD + sub * SCAN_S + 4 * q);
          float e0, e1, e2, e3, b0, b1, b2, b3;
          unpair(fma2(d.x, a2[j], bias2), e0, e1), unpair(fma2(d.y, a2[j], bias2), e2, e3);
          unpair(mul2(u.x, bq.x), b0, b1), unpair(mul2(u.y, bq.y), b2, b3);
          e0 = exp2_approx(e0), e1 = exp2_approx(e1), e2 = exp2_approx(e2), e3 = exp2_approx(e3);
          const float k0 = e0 * h[j], h0 = k0 + b0, k1 = e1 * h0, h1 = k1 + b1, k2 = e2 * h1, h2 = k2 + b2, k3 = e3 * h2;
          h[j] = k3 + b3;
          kv[q][j][0] = pair(k0, k1), kv[q][j][1] = pair(k2, k3);
          const f32x2 h01 = pair(h0, h1), h23 = pair(h2, h[j]);
          y01 = fma2(cq.x, h01, y01), y23 = fma2(cq.y, h23, y23);
          float x[4];
          unpair(mul2(g.x, h01), x[0], x[1]), unpair(mul2(g.y, h23), x[2], x[3]);
          quad_sum(j, x, lo, hi);
        }
        sy[q * 32] = make_ulonglong2(y01, y23);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[8 + q * 4 + i] = lo[i];
      }
#pragma unroll
      for (int q = 1; q >= 0; --q) {
        const ulonglong2 d = de[q * 32], u = dx[q * 32], g = dp[q * 32];
        float g0, g1, g2, g3;
        unpair(g.x, g0, g1), unpair(g.y, g2, g3);
        f32x2 ek01 = 0, ek23 = 0, eb01 = 0, eb23 = 0;
        float lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const ulonglong2 bq = *reinterpret_cast<const ulonglong2*>(s.tb + nj[j] * SCAN_LD + sub * SCAN_S + 4 * q);
          const ulonglong2 cq = *reinterpret_cast<const ulonglong2*>(s.tc + nj[j] * SCAN_LD + sub * SCAN_S + 4 * q);
          float c0, c1, c2, c3, a0, a1, a2_, a3;
          unpair(cq.x, c0, c1), unpair(cq.y, c2, c3);
          // the decays again: an exponential costs less than the registers that would keep it
          unpair(fma2(d.x, a2[j], bias2), a0, a1), unpair(fma2(d.y, a2[j], bias2), a2_, a3);
          const float e3 = fmaf(c3, g3, e[j]), e2 = fmaf(c2, g2, exp2_approx(a3) * e3), e1 = fmaf(c1, g1, exp2_approx(a2_) * e2),
                      e0 = fmaf(c0, g0, exp2_approx(a1) * e1);
          e[j] = exp2_approx(a0) * e0;
          const f32x2 e01 = pair(e0, e1), e23 = pair(e2, e3);
          float x[4];
          unpair(mul2(u.x, e01), x[0], x[1]), unpair(mul2(u.y, e23), x[2], x[3]);
          quad_sum(j, x, lo, hi);
          const f32x2 q01 = mul2(e01, kv[q][j][0]), q23 = mul2(e23, kv[q][j][1]);
          ek01 = fma2(a2[j], q01, ek01), ek23 = fma2(a2[j], q23, ek23);
          da2[j] = fma2(d.x, q01, da2[j]), da2[j] = fma2(d.y, q23, da2[j]);
          eb01 = fma2(bq.x, e01, eb01), eb23 = fma2(bq.y, e23, eb23);
        }
        sy[W * SCAN_T * 8 + q * 32] = make_ulonglong2(ek01, ek23);
        sy[2 * W * SCAN_T * 8 + q * 32] = make_ulonglong2(eb01, eb23);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[q * 4 + i] = lo[i];
      }
      // over the eight groups of four lanes: lane bits 4, 3, 2 become the bits of db or dc and of the token
#pragma unroll
      for (int o = 8; o >= 2; o >>= 1) {
        const bool up = lane & (2 * o);
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * o);
        }
      }
      const int t = t0 + sub * SCAN_S + (lane >> 1 & 6);  // lane bits 3, 2 are the token's bits 2, 1
      if (n0 + (lane & 3) < N) {
        if (t < w.len) part[(long long)t * N] = v[0];
        if (t + 1 < w.len) part[(long long)(t + 1) * N] = v[1];
      }
    }
  };
  auto phase_c = [&](int k) {
    const int at = (k % SCAN_GSLOTS * SCAN_T + warp * R) * 32 + lane, t = last - k * SCAN_T + warp * R;
    const int left = w.on ? w.len - t : 0;
    float y[R], ek[R], eb[R], de[R], dp[R];
    sum_tokens<W, R>(s.y + own, y);
    sum_tokens<W, R>(s.y + W * SCAN_T * 32 + own, ek);
    sum_tokens<W, R>(s.y + 2 * W * SCAN_T * 32 + own, eb);
    get_tokens<R>(s.de + own, de);
    get_tokens<R>(s.dp + own, dp);
    float dv[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float x = to_f<IO>(s.x[at + i * 32]);
      y[i] = fmaf(dskip, x, y[i]);
      dv[i] = fmaf(x, eb[i], LN2 * ek[i]);
      if (i < left) acc_d = fmaf(dp[i], x, acc_d);
      eb[i] = fmaf(dskip, dp[i], de[i] * eb[i]);
    }
    if (p.softplus) {
#pragma unroll
      for (int i = 0; i < R; ++i) dv[i] *= sigmoid(to_f<IO>(s.dt[at + i * 32]) + bias);
    }
    if (gated) {
      IO* const out = p.dz.at(w.b, t) + w.c;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float z = to_f<IO>(s.z[at + i * 32]), g = to_f<IO>(s.dy[at + i * 32]);
        if (i < left) out[(long long)i * (int)p.dz.st] = from_f<IO>(g * y[i] * dsilu(z, sigmoid(z)));
      }
    }
    IO *const out_x = p.dx.at(w.b, t) + w.c, *const out_t = p.ddt.at(w.b, t) + w.c;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i >= left) continue;
      out_x[(long long)i * (int)p.dx.st] = from_f<IO>(eb[i]);
      out_t[(long long)i * (int)p.ddt.st] = from_f<IO>(dv[i]);
      acc_bias += dv[i];
    }
  };

  copy(0);
  copy(1);
  for (int i = threadIdx.x; i < (NP - NS) * SCAN_LD; i += W * 32) s.tb[NS * SCAN_LD + i] = s.tc[NS * SCAN_LD + i] = 0.f;
  fetch(last + SCAN_T - SCAN_S);
  copies_wait<0>();
  __syncthreads();
  if (count) {
    phase_a(0);
    __syncthreads();
  }
  for (int k = 0; k < count; ++k) {
    copy(k + 2);
    phase_b(k);
    copies_wait<0>();
    __syncthreads();
    phase_c(k);  // reads its own tokens of what A wrote, and A writes them again
    if (k + 1 < count) phase_a(k + 1);
    __syncthreads();
  }
  // rows behind the length
  const int t1 = min((w.tile0 + p.chunk_tiles) * SCAN_T, p.T);
  for (int t = max(w.len, w.tile0 * SCAN_T) + warp; t < t1; t += W) {
    if (w.on) {
      p.dx.at(w.b, t)[w.c] = from_f<IO>(0.f);
      p.ddt.at(w.b, t)[w.c] = from_f<IO>(0.f);
      if (gated) p.dz.at(w.b, t)[w.c] = from_f<IO>(0.f);
    }
    for (int n = lane; n < N; n += 32) p.part_b[(part0 + t) * N + n] = p.part_c[(part0 + t) * N + n] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    if (!w.on || nj[j] >= N) continue;
    float a, b;
    unpair(da2[j], a, b);
    p.part_a[(((long long)w.chunk * p.B + w.b) * p.C + w.c) * N + nj[j]] = a + b;
    if (p.dstate && w.chunk == 0) p.dstate[((long long)w.b * p.C + w.c) * N + nj[j]] = e[j];
  }
  s.y[warp * 32 + lane] = acc_d;
  s.y[(W + warp) * 32 + lane] = acc_bias;
  __syncthreads();
  if (warp == 0 && w.on) {
#pragma unroll
    for (int k = 1; k < W; ++k) acc_d += s.y[k * 32 + lane], acc_bias += s.y[(W + k) * 32 + lane];
    p.part_d[((long long)w.chunk * p.B + w.b) * p.C + w.c] = acc_d;
    p.part_bias[((long long)w.chunk * p.B + w.b) * p.C + w.c] = acc_bias;
  }
}

// The sums over blocks, batch rows and chunks of all gradients, in one launch:
// db and dc (type of the I/O), da, dd and ddt_bias, each in its share of the
// blocks.
template <typename IO> struct ScanSums {
  const float* part[5];
  long long P[5], n[5], first[6];  // parts and values of a sum; its first block
  Rows<IO> db, dc;
  float* to[5];
  int B, T, N;
};
template <typename IO> struct ScanSumRows {
  Rows<IO> out;
  int B, T, N;
  __device__ __forceinline__ void put(long long i, float v) const {
    const int n = (int)(i % N);  // i = ((g * B + b) * T + t) * N + n
    long long r = i / N;
    const long long t = r % T;
    r /= T;
    out.at((int)(r % B), t)[r / B * N + n] = from_f<IO>(v);
  }
};
struct ScanSumFloats {
  float* out;
  __device__ __forceinline__ void put(long long i, float v) const { out[i] = v; }
};
template <typename IO> __global__ void __launch_bounds__(256) scan_sums_kernel(const ScanSums<IO> p) {
  const long long x = blockIdx.x;
  if (x < p.first[1])
    sum_block<8>(p.part[0], p.P[0], p.n[0], p.n[0], x, ScanSumRows<IO>{p.db, p.B, p.T, p.N});
  else if (x < p.first[2])
    sum_block<8>(p.part[1], p.P[1], p.n[1], p.n[1], x - p.first[1], ScanSumRows<IO>{p.dc, p.B, p.T, p.N});
  else if (x < p.first[3])
    sum_block<8>(p.part[2], p.P[2], p.n[2], p.n[2], x - p.first[2], ScanSumFloats{p.to[2]});
  else if (x < p.first[4])
    sum_block<8>(p.part[3], p.P[3], p.n[3], p.n[3], x - p.first[3], ScanSumFloats{p.to[3]});
  else
    sum_block<8>(p.part[4], p.P[4], p.n[4], p.n[4], x - p.first[4], ScanSumFloats{p.to[4]});
}

// One token of every row: four threads share a channel's states and join their
// sums over the four.  With VEC, four states at a time: the state, 8 bytes a
// state of traffic where everything else is less than one, goes in 16-byte
// accesses, whole sectors of a row at once.  64x4096 bf16 with 16 states, 34
// MB of state: 12 us where three states take turns, which the L2 nearly holds,
// 18 us with states from memory (floor 5.7); the call from Python takes 14.
// Blocks take a column of 32 channels through every gridDim.y-th row, so that
// what does not depend on the row is found once.
template <typename IO, bool VEC>
__global__ void __launch_bounds__(128) scan_step_kernel(const ScanArgs<IO> p, const int* __restrict__ active) {
  const int q = threadIdx.x & 3, c = blockIdx.x * 32 + (threadIdx.x >> 2), N = p.N;
  const bool on = c < p.C;
  const int g = on && p.G > 1 ? c / (p.C / p.G) * N : 0;
  const float bias = on && p.dt_bias ? __ldg(p.dt_bias + c) : 0.f, skip = on && p.d ? __ldg(p.d + c) : 0.f;
  const float* const av = p.a + (long long)(on ? c : 0) * N;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const bool live = on && (!active || __ldg(active + b));
    float y = 0.f, x = 0.f, z = 0.f;
    if (live) {
      const IO* const bv = p.b.p + b * p.b.sb + g;
      const IO* const cv = p.c.p + b * p.c.sb + g;
      float* const h = p.state_out + ((long long)b * p.C + c) * N;
      x = to_f<IO>(__ldg(p.x.p + b * p.x.sb + c));
      if (p.z.p) z = to_f<IO>(__ldg(p.z.p + b * p.z.sb + c));
      const float v = to_f<IO>(__ldg(p.dt.p + b * p.dt.sb + c)) + bias;
      auto step = [&] { return p.softplus ? softplus(v) : v; };
      if constexpr (VEC) {
        for (int n = q * 4; n < N; n += 16) {
          float hv[4], a[4], bf[4], cf[4];
          load_pack<float, 4>(h + n, hv);
          load_pack<float, 4>(av + n, a);
          load_pack<IO, 4>(bv + n, bf);
          load_pack<IO, 4>(cv + n, cf);
          const float d = step(), dx = d * x, dl = d * LOG2E;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hv[i] = fmaf(exp2_approx(fmaf(dl, a[i], EXP_BIAS)), hv[i], dx * bf[i]);
            y = fmaf(cf[i], hv[i], y);
          }
          store_pack<float, 4>(h + n, hv);
        }
      } else {
        const float d = step();
        for (int n = q; n < N; n += 4) {
          const float s = fmaf(exp2_approx(fmaf(d * LOG2E, __ldg(av + n), EXP_BIAS)), h[n], d * x * to_f<IO>(bv[n]));
          h[n] = s;
          y = fmaf(to_f<IO>(cv[n]), s, y);
        }
      }
    }
    y += __shfl_xor_sync(0xffffffffu, y, 1);
    y += __shfl_xor_sync(0xffffffffu, y, 2);
    if (!on || q) continue;
    if (live) {
      y = fmaf(skip, x, y);
      if (p.z.p) y *= z * sigmoid(z);
    }
    p.y.p[b * p.y.sb + c] = from_f<IO>(y);
  }
}

}  // namespace wtseq
