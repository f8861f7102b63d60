// C entries of the sequence operators (wtconv_seq.h): argument checks on the
// host, choice of the variant, launches.

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <type_traits>

#include "seq_causal.cuh"
#include "seq_common.cuh"
#include "seq_norm.cuh"
#include "seq_scan.cuh"

using namespace wtseq;

namespace {

constexpr long long MAX_ELEMENTS = 1ll << 56;  // byte offsets stay within 64 bits
constexpr long long MAX_TOKEN_STRIDE = INT_MAX;  // kernels hold it in 32 bits
constexpr int MAX_TOKENS = 1 << 30;  // of a row: token counts and tiles stay within 32 bits
constexpr int MAX_ROW = INT_MAX - 4095;  // elements of a token's row: kernels hold a channel, rounded up to a block's, in 32 bits
constexpr int SMS = 148;

size_t elt(wtconv_dtype t) { return t == WTCONV_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
size_t rup16(size_t n) { return (n + 15) & ~(size_t)15; }

bool dtype_ok(wtconv_dtype t) { return t == WTCONV_F32 || t == WTCONV_BF16; }

// Rows of an activation that the call needs.  Output rows must not overlap:
// tokens behind one another within a batch row, or batch rows within a token.
wtconv_status check_rows(const wtconv_rows* r, size_t e, int B, int T, long long C, bool output) {
  if (!r || !r->data || r->batch_stride < 0 || r->token_stride < 0) return WTCONV_ERR_ARG;
  if (r->batch_stride > MAX_ELEMENTS / B || (T > 1 && r->token_stride > MAX_TOKEN_STRIDE)) return WTCONV_ERR_ARG;
  if (output) {
    const bool by_row = (T == 1 || r->token_stride >= C) &&
                        (B == 1 || r->batch_stride >= (long long)(T - 1) * r->token_stride + C);
    const bool by_token = (B == 1 || r->batch_stride >= C) &&
                          (T == 1 || r->token_stride >= (long long)(B - 1) * r->batch_stride + C);
    if (!by_row && !by_token) return WTCONV_ERR_ARG;
  }
  return aligned(r->data, e) ? WTCONV_OK : WTCONV_ERR_ALIGN;
}

// A pointer that may be NULL, aligned to its elements.
wtconv_status check_ptr(const void* p, size_t e, bool required) {
  if (!p) return required ? WTCONV_ERR_ARG : WTCONV_OK;
  return aligned(p, e) ? WTCONV_OK : WTCONV_ERR_ALIGN;
}

wtconv_status check_ws(const void* ws, size_t have, size_t need) {
  if (!need) return WTCONV_OK;
  if (!ws || have < need) return WTCONV_ERR_WORKSPACE;
  return aligned(ws, 16) ? WTCONV_OK : WTCONV_ERR_ALIGN;
}

// Whether an output begins where an input does and threads would read there what
// others have written: such calls are refused.  `in_place`: the call's every
// value of that input is read by the thread that writes there, before it does
// (the single-token calls and the norms), which is so if the rows are the same.
typedef std::initializer_list<const void*> Pointers;
const void* at(const wtconv_rows* r) { return r ? r->data : nullptr; }
bool begins_with(Pointers outs, Pointers ins) {
  for (const void* o : outs)
    for (const void* i : ins)
      if (o && o == i) return true;
  return false;
}
bool in_place(const wtconv_rows* out, const wtconv_rows* in, int B, int T) {
  return (B == 1 || out->batch_stride == in->batch_stride) && (T == 1 || out->token_stride == in->token_stride);
}

#define TRY(call)                                   \
  do {                                              \
    const wtconv_status try_status = (call);        \
    if (try_status != WTCONV_OK) return try_status; \
  } while (0)

// Whether V channels at a time of these rows can be one access (or 16-byte
// accesses).
bool wide(const wtconv_rows* r, int V, size_t e, int B, int T) {
  if (!r) return true;
  const size_t bytes = std::min<size_t>(16, V * e);
  return aligned(r->data, bytes) && (B == 1 || r->batch_stride * e % bytes == 0) &&
         (T == 1 || r->token_stride * e % bytes == 0);
}
bool wide(const void* p, int V, size_t e) { return aligned(p, std::min<size_t>(16, V * e)); }

wtconv_status launched() { return cudaGetLastError() == cudaSuccess ? WTCONV_OK : WTCONV_ERR_CUDA; }
bool grid_ok(long long blocks) { return blocks <= INT_MAX; }

// ------------------------------------------------------ causal convolution
wtconv_status check_causal(const wtconv_causal_desc* d) {
  if (!d || d->B <= 0 || d->T <= 0 || d->T > MAX_TOKENS || d->C <= 0 || d->k <= 0 || !dtype_ok(d->io)) return WTCONV_ERR_ARG;
  if (d->C > MAX_ROW || (long long)d->B * d->T > MAX_ELEMENTS / d->C) return WTCONV_ERR_ARG;
  return d->k > WTCONV_CAUSAL_MAX_K ? WTCONV_ERR_UNSUPPORTED : WTCONV_OK;
}

// Tokens of a thread's strip: long ones repeat little at their ends, short ones
// give the GPU more threads.  The longest of 16 .. most that leaves `fill`
// threads, of four channels each, for every SM.
int causal_strip(const wtconv_causal_desc* d, int most, int fill) {
  int strip = most;
  while (strip > 16 && (long long)d->B * ceil_div(d->T, strip) * ceil_div(d->C, 4) < (long long)SMS * fill) strip /= 2;
  return strip;
}
int causal_forward_strip(const wtconv_causal_desc* d) { return causal_strip(d, 64, 768); }
int causal_grad_strip(const wtconv_causal_desc* d) { return causal_strip(d, 128, 256); }
long long causal_grad_strips(const wtconv_causal_desc* d) { return ceil_div(d->T, causal_grad_strip(d) * CAUSAL_GY); }
size_t causal_ws(const wtconv_causal_desc* d) {
  return (size_t)(d->B * causal_grad_strips(d)) * d->C * (d->k + 1) * sizeof(float);
}

template <typename IO> CausalArgs<IO> causal_args(const wtconv_causal_desc* d, const wtconv_rows* x, const float* w,
                                                  const float* bias) {
  CausalArgs<IO> a = {};
  a.x = rows_of<IO>(x, d->T);
  a.w = w;
  a.bias = bias;
  a.B = d->B;
  a.T = d->T;
  a.C = d->C;
  a.silu = d->silu;
  return a;
}

// Calls f with the number of taps as a compile-time constant.
template <int V_> struct Int { static constexpr int value = V_; };
template <typename F> wtconv_status with_taps(int k, F f) {
  switch (k) {
    case 1: return f(Int<1>());
    case 2: return f(Int<2>());
    case 3: return f(Int<3>());
    case 4: return f(Int<4>());
    case 5: return f(Int<5>());
    case 6: return f(Int<6>());
    case 7: return f(Int<7>());
    default: return f(Int<8>());
  }
}

template <typename IO, int V> wtconv_status causal_forward(const CausalArgs<IO>& a, int k, cudaStream_t st) {
  const long long blocks = ceil_div((long long)(a.C / V) * a.strips * a.B, 128);
  if (!grid_ok(blocks)) return WTCONV_ERR_UNSUPPORTED;
  return with_taps(k, [&](auto K) {
    causal_forward_kernel<IO, K.value, V><<<(unsigned)blocks, 128, 0, st>>>(a);
    return launched();
  });
}

template <typename IO, int V>
wtconv_status causal_backward(const CausalArgs<IO>& a, int k, float* dw, float* dbias, cudaStream_t st) {
  const long long groups = (long long)a.strips * a.B, blocks = ceil_div(a.C / V, 32) * groups;
  if (!grid_ok(blocks)) return WTCONV_ERR_UNSUPPORTED;
  TRY(with_taps(k, [&](auto K) {
    causal_backward_kernel<IO, K.value, V><<<(unsigned)blocks, 256, 0, st>>>(a);
    return launched();
  }));
  const long long n = (long long)a.C * (k + 1);
  launch_sum(a.part, groups, n, n, CausalSums{dw, dbias, k}, st);
  return launched();
}

template <typename IO, int V>
wtconv_status causal_step(const CausalArgs<IO>& a, int k, const int* active, cudaStream_t st) {
  const long long blocks = ceil_div((long long)(a.C / V) * a.B, 128);
  if (!grid_ok(blocks)) return WTCONV_ERR_UNSUPPORTED;
  return with_taps(k, [&](auto K) {
    causal_step_kernel<IO, K.value, V><<<(unsigned)blocks, 128, 0, st>>>(a, active);
    return launched();
  });
}

// -------------------------------------------------------------------- scan
// A group's channels and states as the kernels read them: rounded up to 16
// bytes and to four, by copies where that is more than there are.
long long scan_group(const wtconv_scan_desc* d) {
  const long long e = 16 / elt(d->io);
  return ceil_div(d->C / d->G, e) * e;
}
int scan_states(const wtconv_scan_desc* d) { return (d->N + 3) / 4 * 4; }

wtconv_status check_scan(const wtconv_scan_desc* d) {
  if (!d || d->B <= 0 || d->T <= 0 || d->T > MAX_TOKENS || d->C <= 0 || d->N <= 0 || d->G <= 0 || d->C % d->G || !dtype_ok(d->io))
    return WTCONV_ERR_ARG;
  if (d->N > WTCONV_SCAN_MAX_N) return WTCONV_ERR_UNSUPPORTED;
  if (d->G * scan_group(d) > MAX_ROW || (long long)d->G * scan_states(d) > MAX_ROW) return WTCONV_ERR_ARG;
  return (long long)d->B * d->T > MAX_ELEMENTS / d->C / 64 ? WTCONV_ERR_ARG : WTCONV_OK;
}

int scan_blocks(const wtconv_scan_desc* d) { return (int)ceil_div(d->C / d->G, 32); }

// Chunks of a row: as many as it takes to give every SM SCAN_FILL blocks, of
// at least SCAN_CHUNK tiles.  A cut row pays the recurrence twice, so rows are
// cut only where whole ones leave half of that idle.
// At most SCAN_CHUNKS, since a chunk joins all those before it one by one.
constexpr int SCAN_FILL = 4, SCAN_CHUNK = 4, SCAN_CHUNKS = 64;
void scan_plan(const wtconv_scan_desc* d, int* chunks, int* chunk_tiles) {
  const long long rows = (long long)d->B * scan_blocks(d) * d->G, tiles = ceil_div(d->T, SCAN_T);
  long long n = 1;
  if (rows * 2 <= SMS * SCAN_FILL) n = std::max(1ll, std::min(std::min<long long>(SCAN_CHUNKS, SMS * SCAN_FILL / rows), tiles / SCAN_CHUNK));
  *chunk_tiles = (int)ceil_div(tiles, n);
  *chunks = (int)ceil_div(tiles, *chunk_tiles);
}

struct ScanWs {  // bytes into the workspace, each part on 16
  size_t ends, sums, grad_ends, pads, ckpt, part_b, part_c, part_a, part_d, part_bias, end;
};
ScanWs scan_ws(const wtconv_scan_desc* d, bool backward) {
  ScanWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += rup16(n);
    return r;
  };
  int chunks, per;
  scan_plan(d, &chunks, &per);
  const size_t tokens = (size_t)d->B * d->T, bc = (size_t)d->B * d->C, cut = chunks > 1 ? chunks : 0;
  w.ends = take(cut * bc * d->N * 4);
  w.sums = take(cut * bc * 4);
  w.grad_ends = take(backward ? cut * bc * d->N * 4 : 0);
  w.pads = at;
  if (scan_group(d) != d->C / d->G)
    for (int k = 0; k < (backward ? 4 : 3); ++k) take(tokens * d->G * scan_group(d) * elt(d->io));
  if (scan_states(d) != d->N)
    for (int k = 0; k < 2; ++k) take(tokens * d->G * scan_states(d) * elt(d->io));
  if (backward) {
    w.ckpt = take(ceil_div(d->T, SCAN_T) * (SCAN_T / SCAN_S) * bc * d->N * 4);
    w.part_b = take(scan_blocks(d) * tokens * d->G * d->N * 4);
    w.part_c = take(scan_blocks(d) * tokens * d->G * d->N * 4);
    w.part_a = take(chunks * bc * d->N * 4);
    w.part_d = take(chunks * bc * 4);
    w.part_bias = take(chunks * bc * 4);
  }
  w.end = at;
  return w;
}

template <typename IO>
ScanArgs<IO> scan_args(const wtconv_scan_desc* d, const wtconv_rows* x, const wtconv_rows* dt, const float* a,
                       const wtconv_rows* b, const wtconv_rows* c, const float* skip, const wtconv_rows* z,
                       const float* dt_bias) {
  ScanArgs<IO> p = {};
  p.x = rows_of<IO>(x, d->T);
  p.dt = rows_of<IO>(dt, d->T);
  p.z = rows_of<IO>(z, d->T);
  p.b = rows_of<IO>(b, d->T);
  p.c = rows_of<IO>(c, d->T);
  p.a = a;
  p.d = skip;
  p.dt_bias = dt_bias;
  p.B = d->B;
  p.T = d->T;
  p.C = d->C;
  p.N = d->N;
  p.G = d->G;
  p.softplus = d->softplus;
  p.blocks = scan_blocks(d);
  p.tiles = (int)ceil_div(d->T, SCAN_T);
  p.group = d->C / d->G;
  p.states = d->N;
  return p;
}

wtconv_status check_scan_inputs(const wtconv_scan_desc* d, const wtconv_rows* x, const wtconv_rows* dt, const float* a,
                                const wtconv_rows* b, const wtconv_rows* c, const float* skip, const wtconv_rows* z,
                                const float* dt_bias) {
  const size_t e = elt(d->io);
  const long long gn = (long long)d->G * d->N;
  TRY(check_rows(x, e, d->B, d->T, d->C, false));
  TRY(check_rows(dt, e, d->B, d->T, d->C, false));
  TRY(check_rows(b, e, d->B, d->T, gn, false));
  TRY(check_rows(c, e, d->B, d->T, gn, false));
  if (z) TRY(check_rows(z, e, d->B, d->T, d->C, false));
  TRY(check_ptr(a, 4, true));
  TRY(check_ptr(skip, 4, false));
  return check_ptr(dt_bias, 4, false);
}

// Lets a kernel have `most` bytes of shared memory.  The limit belongs to the
// kernel, and other host threads launch it with other counts of states, so
// `most` is what the kernel needs at the most states that its blocks hold: every
// call sets the same.
template <typename K> wtconv_status allow_smem(K kernel, size_t most) {
  if (most <= 48 * 1024) return WTCONV_OK;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) == cudaSuccess
             ? WTCONV_OK
             : WTCONV_ERR_CUDA;
}

// Calls f with the warps of a block: SCAN_J states each, but up to four where
// so few blocks leave an SM with less than four warps.  Warps without a state
// still take their share of the tokens in A and C, which is most of the work of
// a block of four states (8x77x121 bf16, N = 4: gradients 70 us in blocks of
// one warp, 39 us in blocks of four).
template <typename F> wtconv_status with_warps(int N, long long blocks, F f) {
  int W = N <= SCAN_J ? 1 : (N <= 2 * SCAN_J ? 2 : (N <= 4 * SCAN_J ? 4 : (N <= 8 * SCAN_J ? 8 : 16)));
  while (W < 4 && blocks * W < SMS * 4) W *= 2;
  switch (W) {
    case 1: return f(Int<1>());
    case 2: return f(Int<2>());
    case 4: return f(Int<4>());
    case 8: return f(Int<8>());
    default: return f(Int<16>());
  }
}
static_assert(WTCONV_SCAN_MAX_N == 16 * SCAN_J, "a block has at most 16 warps");

template <typename IO, int MODE> wtconv_status run_scan_pass(const ScanArgs<IO>& p, cudaStream_t st) {
  const long long blocks = (long long)p.B * p.blocks * p.G * p.chunks;
  if (!grid_ok(blocks)) return WTCONV_ERR_UNSUPPORTED;
  return with_warps(p.N, blocks, [&](auto W) {
    auto smem_of = [&](int states) { return (size_t)(ScanSmem<IO>(nullptr, states, W.value).end - (char*)nullptr); };
    const size_t smem = smem_of(p.states);
    TRY((allow_smem(scan_forward_kernel<IO, MODE, W.value>, smem_of(W.value * SCAN_J))));
    scan_forward_kernel<IO, MODE, W.value><<<(unsigned)blocks, W.value * 32, smem, st>>>(p);
    return launched();
  });
}

// The plan of a pass, the copies that it needs, and the chunks' ends where
// rows are cut.
template <typename IO>
wtconv_status scan_prepare(const wtconv_scan_desc* d, ScanArgs<IO>& p, bool backward, char* ws, cudaStream_t st) {
  const ScanWs w = scan_ws(d, backward);
  scan_plan(d, &p.chunks, &p.chunk_tiles);
  p.ends = reinterpret_cast<float*>(ws + w.ends);
  p.sums = reinterpret_cast<float*>(ws + w.sums);
  p.grad_ends = reinterpret_cast<float*>(ws + w.grad_ends);
  ScanPad<IO> pad = {};
  pad.lengths = p.lengths;
  pad.B = p.B, pad.T = p.T, pad.G = p.G;
  int n = 0;
  char* at = ws + w.pads;
  auto copy = [&](Rows<IO>& r, int from, int to) {
    if (!r.p) return;
    pad.in[n] = r, pad.from[n] = from, pad.to[n] = to;
    pad.out[n] = reinterpret_cast<IO*>(at);
    const long long row = (long long)p.G * to;
    r = Rows<IO>{pad.out[n], row * p.T, row};
    at += rup16((size_t)p.B * p.T * row * sizeof(IO));
    ++n;
  };
  if (scan_group(d) != p.group) {
    copy(p.x, p.group, scan_group(d)), copy(p.dt, p.group, scan_group(d)), copy(p.z, p.group, scan_group(d));
    if (backward) copy(p.dy, p.group, scan_group(d));
    p.group = scan_group(d);
  }
  if (scan_states(d) != p.states) {
    copy(p.b, p.states, scan_states(d)), copy(p.c, p.states, scan_states(d));
    p.states = scan_states(d);
  }
  if (n) {
    scan_pad_kernel<IO><<<dim3(SMS * 4, n), 256, 0, st>>>(pad);
    TRY(launched());
  }
  auto fits = [&](const Rows<IO>& r, size_t bytes) {
    return aligned(r.p, bytes) && (p.B == 1 || r.sb * sizeof(IO) % bytes == 0) && (p.T == 1 || r.st * sizeof(IO) % bytes == 0);
  };
  p.wide_x = fits(p.x, 16) && fits(p.dt, 16) && fits(p.z, 16) && (!backward || fits(p.dy, 16));
  p.wide_bc = fits(p.b, 4 * sizeof(IO)) && fits(p.c, 4 * sizeof(IO));
  return p.chunks > 1 ? run_scan_pass<IO, SCAN_ENDS>(p, st) : WTCONV_OK;
}

template <typename IO>
wtconv_status run_scan_backward(const wtconv_scan_desc* d, ScanArgs<IO>& p, const wtconv_rows* db, const wtconv_rows* dc,
                                float* da, float* dd, float* ddt_bias, char* ws, cudaStream_t st) {
  // the sums take the most blocks
  if (!grid_ok(2 * ceil_div((long long)p.G * p.B * p.T * p.N, 32) + (long long)p.C * (p.N + 2)) ||
      !grid_ok((long long)p.B * p.blocks * p.G * ceil_div(p.tiles, SCAN_CHUNK)))
    return WTCONV_ERR_UNSUPPORTED;
  TRY(scan_prepare<IO>(d, p, true, ws, st));
  const ScanWs w = scan_ws(d, true);
  p.ckpt = reinterpret_cast<float*>(ws + w.ckpt);
  p.part_b = reinterpret_cast<float*>(ws + w.part_b);
  p.part_c = reinterpret_cast<float*>(ws + w.part_c);
  p.part_a = reinterpret_cast<float*>(ws + w.part_a);
  p.part_d = reinterpret_cast<float*>(ws + w.part_d);
  p.part_bias = reinterpret_cast<float*>(ws + w.part_bias);
  TRY((run_scan_pass<IO, SCAN_CKPT>(p, st)));
  if (p.chunks > 1) TRY((run_scan_pass<IO, SCAN_GRAD_ENDS>(p, st)));
  const long long blocks = (long long)p.B * p.blocks * p.G * p.chunks, parts = (long long)p.chunks * p.B;
  TRY(with_warps(p.N, blocks, [&](auto W) {
    auto smem_of = [&](int states) { return (size_t)(ScanGradSmem<IO>(nullptr, states, W.value).end - (char*)nullptr); };
    const size_t smem = smem_of(p.states);
    TRY((allow_smem(scan_backward_kernel<IO, W.value>, smem_of(W.value * SCAN_J))));
    scan_backward_kernel<IO, W.value><<<(unsigned)blocks, W.value * 32, smem, st>>>(p);
    return launched();
  }));
  ScanSums<IO> sums = {};
  sums.db = rows_of<IO>(db, p.T), sums.dc = rows_of<IO>(dc, p.T);
  sums.B = p.B, sums.T = p.T, sums.N = p.N;
  long long first = 0;
  int k = 0;
  auto add = [&](const float* part, long long P, long long n, float* to) {
    sums.part[k] = part, sums.P[k] = P, sums.n[k] = n, sums.to[k] = to;
    sums.first[k++] = first;
    first += to || k <= 2 ? ceil_div(n, 32) : 0;
  };
  const long long bc = (long long)p.G * p.B * p.T * p.N;
  add(p.part_b, p.blocks, bc, nullptr);
  add(p.part_c, p.blocks, bc, nullptr);
  add(p.part_a, parts, (long long)p.C * p.N, da);
  add(p.part_d, parts, p.C, dd);
  add(p.part_bias, parts, p.C, ddt_bias);
  sums.first[k] = first;
  scan_sums_kernel<IO><<<(unsigned)first, 256, 0, st>>>(sums);
  return launched();
}

// -------------------------------------------------------------------- norm
wtconv_status check_norm(const wtconv_norm_desc* d) {
  if (!d || d->B <= 0 || d->T <= 0 || d->T > MAX_TOKENS || d->C <= 0 || !dtype_ok(d->io) || !dtype_ok(d->res) || !(d->eps >= 0.f))
    return WTCONV_ERR_ARG;
  if ((long long)d->B * d->T > MAX_ELEMENTS / d->C) return WTCONV_ERR_ARG;
  return d->C > WTCONV_NORM_MAX_C || (long long)d->B * d->T > INT_MAX ? WTCONV_ERR_UNSUPPORTED : WTCONV_OK;
}

wtconv_status check_norm_inputs(const wtconv_norm_desc* d, const wtconv_rows* x, const wtconv_rows* gate, const float* w,
                                const wtconv_rows* res, const float* scale, const float* w_res, const int* lengths) {
  if ((!gate && !w && !res) || (!res && (scale || w_res))) return WTCONV_ERR_ARG;
  TRY(check_rows(x, elt(d->io), d->B, d->T, d->C, false));
  if (gate) TRY(check_rows(gate, elt(d->io), d->B, d->T, d->C, false));
  if (res) TRY(check_rows(res, elt(d->res), d->B, d->T, d->C, false));
  TRY(check_ptr(w, 4, false));
  TRY(check_ptr(scale, 4, false));
  TRY(check_ptr(w_res, 4, false));
  return check_ptr(lengths, 4, false);
}

// Whether an output of the norms begins at an input with other rows or of another type.
struct NormRowsOf {
  const wtconv_rows* r;
  wtconv_dtype t;
};
bool norm_overlap(const wtconv_norm_desc* d, std::initializer_list<NormRowsOf> outs, std::initializer_list<NormRowsOf> ins,
                  Pointers params) {
  for (const NormRowsOf& o : outs) {
    if (begins_with({at(o.r)}, params)) return true;
    for (const NormRowsOf& i : ins)
      if (at(o.r) && at(o.r) == at(i.r) && (o.t != i.t || !in_place(o.r, i.r, d->B, d->T))) return true;
  }
  return false;
}

// Blocks for rows that `threads` threads hold: enough for the SMs' registers,
// so that each goes through its share of the rows (of the gradients, whose
// blocks leave a partial sum each, fewer).
int norm_blocks(const wtconv_norm_desc* d, int threads, int per_sm) {
  const long long most = (long long)SMS * std::max(1, std::min(16, per_sm / threads));
  return (int)std::min<long long>((long long)d->B * d->T, most);
}
// Chunks of V channels a thread: 8 values while 512 threads hold the row, then
// 16 and 32.  Threads of a row.
int norm_threads(int C, int V, int nv) { return (int)ceil_div(ceil_div(ceil_div(C, V), nv), 32) * 32; }
int norm_chunks(int C, int V) {
  int nv = 8 / V;
  while (nv < 32 / V && norm_threads(C, V, nv) > 512) nv *= 2;
  return nv;
}
int norm_threads(int C, int V) { return norm_threads(C, V, norm_chunks(C, V)); }
// Channels of a chunk of neighbours, 16 bytes of them; of a chunk at odd rows.
constexpr int norm_wide(size_t e) { return (int)(16 / e); }
constexpr int NORM_ODD = 8;
// The most blocks of the gradients: the size of the workspace does not depend
// on whether the rows suit wide loads.
int norm_grad_blocks(const wtconv_norm_desc* d) {
  const int threads = std::min(norm_threads(d->C, NORM_ODD), norm_threads(d->C, norm_wide(elt(d->io))));
  return norm_blocks(d, threads, NORM_GRAD_THREADS);
}

template <typename IO, typename RES>
NormArgs<IO, RES> norm_args(const wtconv_norm_desc* d, const wtconv_rows* x, const wtconv_rows* gate, const float* w,
                            const wtconv_rows* res, const float* scale, const float* w_res, const int* lengths) {
  NormArgs<IO, RES> a = {};
  a.x = rows_of<IO>(x, d->T);
  a.gate = rows_of<IO>(gate, d->T);
  a.res = rows_of<RES>(res, d->T);
  a.w = w;
  a.scale = scale;
  a.w_res = w_res;
  a.lengths = lengths;
  a.B = d->B;
  a.T = d->T;
  a.C = d->C;
  a.eps = d->eps;
  return a;
}

// Calls f with V, NV, whether chunks are neighbouring channels, and the threads.
template <int V, typename F> wtconv_status norm_shape(int C, F f) {
  constexpr int N1 = 8 / V, N2 = 16 / V, N3 = 32 / V;
  const int nv = norm_chunks(C, V), threads = norm_threads(C, V);
  if (nv == N1) return f(Int<V>(), Int<N1>(), threads);
  if (nv == N2) return f(Int<V>(), Int<N2>(), threads);
  return f(Int<V>(), Int<N3>(), threads);
}
template <typename IO, typename F> wtconv_status norm_variant(int C, bool vec, F f) {
  if (vec) return norm_shape<norm_wide(sizeof(IO))>(C, [&](auto v, auto nv, int t) { return f(v, nv, std::true_type(), t); });
  return norm_shape<NORM_ODD>(C, [&](auto v, auto nv, int t) { return f(v, nv, std::false_type(), t); });
}

// Calls f with the I/O type (and the type of the residual).
template <typename F> wtconv_status with_io(wtconv_dtype io, F f) {
  return io == WTCONV_F32 ? f(float()) : f(__nv_bfloat16());
}

}  // namespace

extern "C" {

size_t wtconv_causal_workspace_size(const wtconv_causal_desc* desc) {
  return check_causal(desc) == WTCONV_OK ? causal_ws(desc) : 0;
}

wtconv_status wtconv_causal_forward(const wtconv_causal_desc* desc, const wtconv_rows* x, const float* w,
                                    const float* bias, const void* state, const int* lengths, const wtconv_rows* y,
                                    void* state_out, void* stream) {
  TRY(check_causal(desc));
  const size_t e = elt(desc->io);
  const int B = desc->B, T = desc->T, C = desc->C;
  TRY(check_rows(x, e, B, T, C, false));
  TRY(check_rows(y, e, B, T, C, true));
  TRY(check_ptr(w, 4, true));
  TRY(check_ptr(bias, 4, false));
  TRY(check_ptr(lengths, 4, false));
  TRY(check_ptr(state, e, false));
  TRY(check_ptr(state_out, e, false));
  const void *const s0 = desc->k > 1 ? state : nullptr, *const s1 = desc->k > 1 ? state_out : nullptr;
  if (begins_with({at(y), s1}, {at(x), w, bias, lengths}) || begins_with({at(y)}, {s0})) return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    CausalArgs<IO> a = causal_args<IO>(desc, x, w, bias);
    a.y = rows_of<IO>(y, T);
    a.state = static_cast<const IO*>(state);
    a.state_out = static_cast<IO*>(state_out);
    a.lengths = lengths;
    a.strip = causal_forward_strip(desc);
    a.strips = (int)ceil_div(T, a.strip);
    // Channels of a thread, the most that the rows allow: eight would fill the registers with taps and windows.  Four
    // against two, in us: 4x4096x4096 bf16 at k 2, 4, 5, 7, 8 49, 60, 59, 74, 84 against 56, 62, 65, 96, 92; 4x2048x4096
    // fp32 78, 81, 107, 132, 111 against 77, 78, 101, 120, 104: there two are the faster, by 1 to 9%.
    auto fits = [&](int V) {
      return C % V == 0 && wide(w, 4, 4) && wide(x, V, e, B, T) && wide(y, V, e, B, T) && wide(state, V, e) && wide(state_out, V, e);
    };
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (fits(4)) return causal_forward<IO, 4>(a, desc->k, st);
    return fits(2) ? causal_forward<IO, 2>(a, desc->k, st) : causal_forward<IO, 1>(a, desc->k, st);
  });
}

wtconv_status wtconv_causal_backward(const wtconv_causal_desc* desc, const wtconv_rows* x, const wtconv_rows* dy,
                                     const float* w, const float* bias, const void* state, const int* lengths,
                                     const void* dstate_out, const wtconv_rows* dx, float* dw, float* dbias,
                                     void* dstate, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_causal(desc));
  const size_t e = elt(desc->io);
  const int B = desc->B, T = desc->T, C = desc->C;
  TRY(check_rows(x, e, B, T, C, false));
  TRY(check_rows(dy, e, B, T, C, false));
  TRY(check_rows(dx, e, B, T, C, true));
  TRY(check_ptr(w, 4, true));
  TRY(check_ptr(dw, 4, true));
  TRY(check_ptr(bias, 4, false));
  TRY(check_ptr(dbias, 4, bias != nullptr));
  TRY(check_ptr(lengths, 4, false));
  TRY(check_ptr(state, e, false));
  TRY(check_ptr(dstate_out, e, false));
  TRY(check_ptr(dstate, e, false));
  TRY(check_ws(ws, ws_bytes, causal_ws(desc)));
  const bool held = desc->k > 1;
  if (begins_with({at(dx), held ? dstate : nullptr}, {at(x), at(dy), w, bias, lengths, held ? dstate_out : nullptr}) ||
      begins_with({at(dx)}, {held ? state : nullptr}))
    return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    CausalArgs<IO> a = causal_args<IO>(desc, x, w, bias);
    a.dy = rows_of<IO>(dy, T);
    a.dx = rows_of<IO>(dx, T);
    a.state = static_cast<const IO*>(state);
    a.dstate_out = static_cast<const IO*>(dstate_out);
    a.dstate = static_cast<IO*>(dstate);
    a.lengths = lengths;
    a.part = static_cast<float*>(ws);
    a.strip = causal_grad_strip(desc);
    a.strips = (int)causal_grad_strips(desc);
    // Taps, windows, sums and loads ahead of four 16-bit or two 32-bit channels fill the registers (bf16: 100 to 213 at
    // k 2 to 8, one block an SM from k 5 on).  Four against two, in us: 8x2048x2048 bf16 at k 2, 4, 5, 7, 8 54, 62, 92,
    // 101, 104 against 78, 83, 85, 99, 108.
    auto fits = [&](int V) {
      return C % V == 0 && wide(w, 4, 4) && wide(x, V, e, B, T) && wide(dy, V, e, B, T) && wide(dx, V, e, B, T) &&
             wide(state, V, e) && wide(dstate_out, V, e) && wide(dstate, V, e);
    };
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if constexpr (sizeof(IO) == 2) {
      if (fits(4)) return causal_backward<IO, 4>(a, desc->k, dw, dbias, st);
    }
    return fits(2) ? causal_backward<IO, 2>(a, desc->k, dw, dbias, st) : causal_backward<IO, 1>(a, desc->k, dw, dbias, st);
  });
}

wtconv_status wtconv_causal_step(const wtconv_causal_desc* desc, const wtconv_rows* x, const float* w,
                                 const float* bias, const int* active, const wtconv_rows* y, void* state,
                                 void* stream) {
  TRY(check_causal(desc));
  if (desc->T != 1) return WTCONV_ERR_ARG;
  const size_t e = elt(desc->io);
  const int B = desc->B, C = desc->C;
  TRY(check_rows(x, e, B, 1, C, false));
  TRY(check_rows(y, e, B, 1, C, true));
  TRY(check_ptr(w, 4, true));
  TRY(check_ptr(bias, 4, false));
  TRY(check_ptr(active, 4, false));
  TRY(check_ptr(state, e, desc->k > 1));
  const void* const held = desc->k > 1 ? state : nullptr;
  if (begins_with({at(y)}, {w, bias, active, held}) || begins_with({held}, {at(x), w, bias, active}) ||
      (at(y) == at(x) && !in_place(y, x, B, 1)))
    return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    CausalArgs<IO> a = causal_args<IO>(desc, x, w, bias);
    a.y = rows_of<IO>(y, 1);
    a.state_out = static_cast<IO*>(state);
    constexpr int V = 4;
    const bool vec = C % V == 0 && wide(w, 4, 4) && wide(x, V, e, B, 1) && wide(y, V, e, B, 1) && wide(state, V, e);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return vec ? causal_step<IO, V>(a, desc->k, active, st) : causal_step<IO, 1>(a, desc->k, active, st);
  });
}

size_t wtconv_scan_workspace_size(const wtconv_scan_desc* desc, int backward) {
  if (check_scan(desc) != WTCONV_OK || (backward != 0 && backward != 1)) return 0;
  return scan_ws(desc, backward).end;
}

wtconv_status wtconv_scan_forward(const wtconv_scan_desc* desc, const wtconv_rows* x, const wtconv_rows* dt,
                                  const float* a, const wtconv_rows* b, const wtconv_rows* c, const float* d,
                                  const wtconv_rows* z, const float* dt_bias, const float* state, const int* lengths,
                                  const wtconv_rows* y, float* state_out, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_scan(desc));
  TRY(check_scan_inputs(desc, x, dt, a, b, c, d, z, dt_bias));
  TRY(check_rows(y, elt(desc->io), desc->B, desc->T, desc->C, true));
  TRY(check_ptr(state, 4, false));
  TRY(check_ptr(state_out, 4, false));
  TRY(check_ptr(lengths, 4, false));
  TRY(check_ws(ws, ws_bytes, wtconv_scan_workspace_size(desc, 0)));
  if (begins_with({at(y), state_out}, {at(x), at(dt), at(b), at(c), at(z), a, d, dt_bias, lengths}) || begins_with({at(y)}, {state}))
    return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    ScanArgs<IO> p = scan_args<IO>(desc, x, dt, a, b, c, d, z, dt_bias);
    p.y = rows_of<IO>(y, desc->T);
    p.state = state;
    p.state_out = state_out;
    p.lengths = lengths;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    TRY(scan_prepare<IO>(desc, p, false, static_cast<char*>(ws), st));
    return run_scan_pass<IO, SCAN_Y>(p, st);
  });
}

wtconv_status wtconv_scan_backward(const wtconv_scan_desc* desc, const wtconv_rows* x, const wtconv_rows* dt,
                                   const float* a, const wtconv_rows* b, const wtconv_rows* c, const float* d,
                                   const wtconv_rows* z, const float* dt_bias, const float* state, const int* lengths,
                                   const wtconv_rows* dy, const float* dstate_out, const wtconv_rows* dx,
                                   const wtconv_rows* ddt, float* da, const wtconv_rows* db, const wtconv_rows* dc,
                                   float* dd, const wtconv_rows* dz, float* ddt_bias, float* dstate, void* ws,
                                   size_t ws_bytes, void* stream) {
  TRY(check_scan(desc));
  TRY(check_scan_inputs(desc, x, dt, a, b, c, d, z, dt_bias));
  const size_t e = elt(desc->io);
  const int B = desc->B, T = desc->T, C = desc->C;
  const long long gn = (long long)desc->G * desc->N;
  if ((d != nullptr) != (dd != nullptr) || (z != nullptr) != (dz != nullptr) ||
      (dt_bias != nullptr) != (ddt_bias != nullptr))
    return WTCONV_ERR_ARG;
  TRY(check_rows(dy, e, B, T, C, false));
  TRY(check_rows(dx, e, B, T, C, true));
  TRY(check_rows(ddt, e, B, T, C, true));
  TRY(check_rows(db, e, B, T, gn, true));
  TRY(check_rows(dc, e, B, T, gn, true));
  if (dz) TRY(check_rows(dz, e, B, T, C, true));
  TRY(check_ptr(da, 4, true));
  TRY(check_ptr(dd, 4, false));
  TRY(check_ptr(ddt_bias, 4, false));
  TRY(check_ptr(state, 4, false));
  TRY(check_ptr(dstate_out, 4, false));
  TRY(check_ptr(dstate, 4, false));
  TRY(check_ptr(lengths, 4, false));
  TRY(check_ws(ws, ws_bytes, wtconv_scan_workspace_size(desc, 1)));
  const Pointers outs = {at(dx), at(ddt), at(db), at(dc), at(dz)};
  const Pointers ins = {at(x), at(dt), at(b), at(c), at(z), at(dy), a, d, dt_bias, lengths, dstate_out};
  if (begins_with(outs, ins) || begins_with(outs, {state}) || begins_with({dstate}, ins)) return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    ScanArgs<IO> p = scan_args<IO>(desc, x, dt, a, b, c, d, z, dt_bias);
    p.dy = rows_of<IO>(dy, T);
    p.dx = rows_of<IO>(dx, T);
    p.ddt = rows_of<IO>(ddt, T);
    p.dz = rows_of<IO>(dz, T);
    p.state = state;
    p.dstate_out = dstate_out;
    p.dstate = dstate;
    p.lengths = lengths;
    return run_scan_backward<IO>(desc, p, db, dc, da, dd, ddt_bias, static_cast<char*>(ws),
                                 static_cast<cudaStream_t>(stream));
  });
}

wtconv_status wtconv_scan_step(const wtconv_scan_desc* desc, const wtconv_rows* x, const wtconv_rows* dt,
                               const float* a, const wtconv_rows* b, const wtconv_rows* c, const float* d,
                               const wtconv_rows* z, const float* dt_bias, const int* active, const wtconv_rows* y,
                               float* state, void* stream) {
  TRY(check_scan(desc));
  if (desc->T != 1) return WTCONV_ERR_ARG;
  TRY(check_scan_inputs(desc, x, dt, a, b, c, d, z, dt_bias));
  TRY(check_rows(y, elt(desc->io), desc->B, 1, desc->C, true));
  TRY(check_ptr(state, 4, true));
  TRY(check_ptr(active, 4, false));
  if (begins_with({at(y)}, {at(b), at(c), a, d, dt_bias, active, state}) ||
      begins_with({state}, {at(x), at(dt), at(b), at(c), at(z), a, d, dt_bias, active}))
    return WTCONV_ERR_ARG;
  for (const wtconv_rows* in : {x, dt, z})
    if (at(y) == at(in) && !in_place(y, in, desc->B, 1)) return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    ScanArgs<IO> p = scan_args<IO>(desc, x, dt, a, b, c, d, z, dt_bias);
    p.y = rows_of<IO>(y, 1);
    p.state_out = state;
    // blocks of 128 threads to fill the SMs, each with its share of the rows
    const long long columns = ceil_div(p.C, 32);
    const dim3 grid((unsigned)columns, (unsigned)std::min<long long>({p.B, 65535, std::max(1ll, SMS * 16 / columns)}));
    const size_t e = sizeof(IO);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.N % 4 == 0 && wide(a, 4, 4) && wide(state, 4, 4) && wide(b, 4, e, p.B, 1) && wide(c, 4, e, p.B, 1))
      scan_step_kernel<IO, true><<<grid, 128, 0, st>>>(p, active);
    else
      scan_step_kernel<IO, false><<<grid, 128, 0, st>>>(p, active);
    return launched();
  });
}

size_t wtconv_norm_workspace_size(const wtconv_norm_desc* desc) {
  if (check_norm(desc) != WTCONV_OK) return 0;
  return rup16((size_t)norm_grad_blocks(desc) * 3 * desc->C * sizeof(float));
}

wtconv_status wtconv_norm_forward(const wtconv_norm_desc* desc, const wtconv_rows* x, const wtconv_rows* gate,
                                  const float* w, const wtconv_rows* res, const float* scale, const float* w_res,
                                  const int* lengths, const wtconv_rows* y, const wtconv_rows* res_out, void* stream) {
  TRY(check_norm(desc));
  TRY(check_norm_inputs(desc, x, gate, w, res, scale, w_res, lengths));
  const int B = desc->B, T = desc->T, C = desc->C;
  if ((res != nullptr) != (res_out != nullptr) || (!res || w_res ? !y : y != nullptr)) return WTCONV_ERR_ARG;
  if (y) TRY(check_rows(y, elt(desc->io), B, T, C, true));
  if (res_out) TRY(check_rows(res_out, elt(desc->res), B, T, C, true));
  if (norm_overlap(desc, {{y, desc->io}, {res_out, desc->res}}, {{x, desc->io}, {gate, desc->io}, {res, desc->res}},
                   {w, scale, w_res, lengths}))
    return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    return with_io(desc->res, [&](auto rio) {
      using RES = decltype(rio);
      NormArgs<IO, RES> a = norm_args<IO, RES>(desc, x, gate, w, res, scale, w_res, lengths);
      a.y = rows_of<IO>(y, T);
      a.res_out = rows_of<RES>(res_out, T);
      constexpr int V = norm_wide(sizeof(IO));
      const bool vec = C % V == 0 && wide(x, V, sizeof(IO), B, T) && wide(gate, V, sizeof(IO), B, T) &&
                       wide(y, V, sizeof(IO), B, T) && wide(res, V, sizeof(RES), B, T) &&
                       wide(res_out, V, sizeof(RES), B, T);
      return norm_variant<IO>(C, vec, [&](auto v, auto nv, auto wide, int threads) {
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const int blocks = norm_blocks(desc, threads, v.value * nv.value <= 8 ? NORM_THREADS : 512);
        if constexpr (v.value * nv.value <= 8) {
          if (threads <= 256) {
            norm_forward_kernel<IO, RES, v.value, nv.value, wide.value, 256><<<blocks, threads, 0, st>>>(a);
            return launched();
          }
        }
        norm_forward_kernel<IO, RES, v.value, nv.value, wide.value, 512><<<blocks, threads, 0, st>>>(a);
        return launched();
      });
    });
  });
}

wtconv_status wtconv_norm_backward(const wtconv_norm_desc* desc, const wtconv_rows* x, const wtconv_rows* gate,
                                   const float* w, const wtconv_rows* res, const float* scale, const float* w_res,
                                   const int* lengths, const wtconv_rows* dy, const wtconv_rows* dres_out,
                                   const wtconv_rows* dx, const wtconv_rows* dgate, float* dw,
                                   const wtconv_rows* dres, float* dscale, float* dw_res, void* ws, size_t ws_bytes,
                                   void* stream) {
  TRY(check_norm(desc));
  TRY(check_norm_inputs(desc, x, gate, w, res, scale, w_res, lengths));
  const int B = desc->B, T = desc->T, C = desc->C;
  if ((gate != nullptr) != (dgate != nullptr) || (w != nullptr) != (dw != nullptr) ||
      (res != nullptr) != (dres != nullptr) || (scale != nullptr) != (dscale != nullptr) ||
      (w_res != nullptr) != (dw_res != nullptr) || (dres_out && !res) || (!res || w_res ? !dy : dy != nullptr))
    return WTCONV_ERR_ARG;
  if (dy) TRY(check_rows(dy, elt(desc->io), B, T, C, false));
  if (dres_out) TRY(check_rows(dres_out, elt(desc->res), B, T, C, false));
  TRY(check_rows(dx, elt(desc->io), B, T, C, true));
  if (dgate) TRY(check_rows(dgate, elt(desc->io), B, T, C, true));
  if (dres) TRY(check_rows(dres, elt(desc->res), B, T, C, true));
  TRY(check_ptr(dw, 4, false));
  TRY(check_ptr(dscale, 4, false));
  TRY(check_ptr(dw_res, 4, false));
  TRY(check_ws(ws, ws_bytes, wtconv_norm_workspace_size(desc)));
  if (norm_overlap(desc, {{dx, desc->io}, {dgate, desc->io}, {dres, desc->res}},
                   {{x, desc->io}, {gate, desc->io}, {res, desc->res}, {dy, desc->io}, {dres_out, desc->res}},
                   {w, scale, w_res, lengths}))
    return WTCONV_ERR_ARG;
  return with_io(desc->io, [&](auto io) {
    using IO = decltype(io);
    return with_io(desc->res, [&](auto rio) {
      using RES = decltype(rio);
      NormArgs<IO, RES> a = norm_args<IO, RES>(desc, x, gate, w, res, scale, w_res, lengths);
      a.dy = rows_of<IO>(dy, T);
      a.dres_out = rows_of<RES>(dres_out, T);
      a.dx = rows_of<IO>(dx, T);
      a.dgate = rows_of<IO>(dgate, T);
      a.dres = rows_of<RES>(dres, T);
      a.part = static_cast<float*>(ws);
      constexpr int V = norm_wide(sizeof(IO));
      const size_t e = sizeof(IO), re = sizeof(RES);
      const bool vec = C % V == 0 && wide(x, V, e, B, T) && wide(gate, V, e, B, T) && wide(dy, V, e, B, T) &&
                       wide(dx, V, e, B, T) && wide(dgate, V, e, B, T) && wide(res, V, re, B, T) &&
                       wide(dres_out, V, re, B, T) && wide(dres, V, re, B, T);
      cudaStream_t st = static_cast<cudaStream_t>(stream);
      int blocks = 0;
      TRY((norm_variant<IO>(C, vec, [&](auto v, auto nv, auto wide, int threads) {
        blocks = norm_blocks(desc, threads, NORM_GRAD_THREADS);
        norm_backward_kernel<IO, RES, v.value, nv.value, wide.value><<<blocks, threads, 0, st>>>(a);
        return launched();
      })));
      if (!dw && !dscale && !dw_res) return WTCONV_OK;
      launch_sum(a.part, blocks, 3ll * C, 3ll * C, NormSums{dw, dscale, dw_res, C}, st);
      return launched();
    });
  });
}

}  // extern "C"
