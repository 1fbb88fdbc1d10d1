// gdn_conv.hip -- short causal depthwise convolution over packed or batched
// sequences, channels last, its gradient, and its single-token step.
//
//   u_t = bias + sum_{k<W} w_k x_{t-W+1+k},      y_t = u_t  or  u_t sigmoid(u_t)
// per channel, the W-1 inputs before a sequence's start taken from its initial
// state (zero without one).  The state that continues a sequence is its last
// W-1 inputs, oldest first.
//
// Bound: memory -- one read of x and one write of y (2 W flops an element).  A
// thread owns 16 bytes of channels (8 bf16 or 4 fp32; in the gradient four of
// either type; one where widths or pointers do not allow that) and walks `run`
// consecutive tokens with the last W-1 inputs in registers, so that x is
// fetched once but for W-1 rows per run, which the neighbouring run's thread
// brings into cache as well.  Threads are numbered channels first over the
// runs, so a wave stays full for any channel count.
// Measured (bf16, W = 4): 8,192 x 6,144 in 38 us (201 MB, most of it from cache);
// 49,828 x 2,304 in 92 us (459 MB, 5.0 TB/s), its gradient in 175 us + 7 us for the
// weights' sums (689 MB; with some 35 vector instructions an element, two of them
// transcendental, the arithmetic takes about 120 us beside the traffic's 141).
// fp32: 8,192 x 6,144 in 83 us (403 MB, 4.8 TB/s), its gradient in 170.  One channel a
// thread: 8,192 x 1,001 bf16 in 12.3 us (2.7 TB/s) and 45 us (1.1), by the two-byte
// accesses' instructions.
// A token for each of 16 sequences of 6,144 channels: 6 us, all of it latency.
#include "gdn_layer.h"

namespace gdn {

namespace {

constexpr int CONV_NT = 256;
constexpr int CONV_AHEAD = 4;  // rows requested together

// The sequence that holds a token, and the next one that holds any.  Token
// indices are 32 bits (the C ABI takes fewer than 2^31 tokens); only addresses
// are 64.
struct SeqCursor {
  const int32_t* cu;
  int N, T, tokens;
  int n, start, end;  // clamped to [0, tokens]: a bad device copy of cu reads nothing out of bounds
  __device__ __forceinline__ explicit SeqCursor(const ConvParams& p)
      : cu(p.cu), N(p.N), T(p.T), tokens((int)p.tokens), n(0), start(0), end(0) {}
  __device__ __forceinline__ void bounds() {
    if (cu) {
      start = min(max(cu[n], 0), tokens);
      end = min(max(cu[n + 1], 0), tokens);
    } else {
      start = n * T;
      end = start + T;
    }
  }
  // false: no sequence holds token t (it lies behind the last one)
  __device__ __forceinline__ bool seek(int t) {
    if (cu) {
      int lo = 0, hi = N - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      n = lo;
    } else {
      n = t / T;
    }
    bounds();
    return t >= start && t < end;
  }
  // to the sequence that starts where this one ended; false behind the last
  __device__ __forceinline__ bool next() {
    const int t = end;
    do {
      if (++n >= N) return false;
      bounds();
    } while (end <= start);
    return start == t;
  }
};

template <class E, int V, int W>
struct ConvTaps {
  float w[W][V], b[V];
  __device__ __forceinline__ void load(const ConvParams& p, int c0) { load(p.w, p.bias, c0); }
  __device__ __forceinline__ void load(const void* wp, const void* bp, int c0) {
    typedef VecIO<E, V> IO;
    // the V channels' taps are V W consecutive entries: W accesses
    float f[W * V];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      float g[V];
      IO::get(IO::load(static_cast<const E*>(wp) + (int64_t)c0 * W + k * V), g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[k * V + e] = g[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][e] = f[e * W + k];
      b[e] = 0.f;
    }
    if (bp) IO::get(IO::load(static_cast<const E*>(bp) + c0), b);
  }
};

// The input at position pos (relative to the sequence's start; negative: the
// initial state) of sequence n.
template <class E, int V, int W>
__device__ __forceinline__ void conv_input(const ConvParams& p, const SeqCursor& c, int pos, int c0, float (&f)[V]) {
  typedef VecIO<E, V> IO;
  if (pos >= 0) {
    IO::get(IO::load(static_cast<const E*>(p.x) + (int64_t)(c.start + pos) * p.x_stride + c0), f);
  } else if (p.init) {
    IO::get(IO::load(static_cast<const E*>(p.init) + ((int64_t)c.n * (W - 1) + pos + W - 1) * p.D + c0), f);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = 0.f;
  }
}

// Blocks [0, nb_run) walk the runs; the rest write the final states.
template <class E, int V, int W>
__global__ __launch_bounds__(CONV_NT) void conv_fwd_kernel(ConvParams p, int64_t nb_run) {
  typedef VecIO<E, V> IO;
  const int CV = p.D / V;
  if (blockIdx.x >= nb_run) {
    const int64_t i = (blockIdx.x - nb_run) * CONV_NT + threadIdx.x;  // (sequence, row, channels)
    if (i >= (int64_t)p.N * (W - 1) * CV) return;
    const int c0 = (int)(i % CV) * V, j = (int)(i / CV % (W - 1));
    SeqCursor c(p);
    c.n = (int)(i / CV / (W - 1));
    c.bounds();
    float f[V];
    conv_input<E, V, W>(p, c, max(c.end - c.start, 0) - (W - 1) + j, c0, f);
    store_vec<E, V>(static_cast<E*>(p.fin) + ((int64_t)c.n * (W - 1) + j) * p.D + c0, f);
    return;
  }
  const int64_t i = blockIdx.x * (int64_t)CONV_NT + threadIdx.x;
  const int64_t run = i / CV;
  if (run >= p.nruns) return;
  const int c0 = (int)(i - run * CV) * V;
  const int t0 = (int)run * p.run, t1 = min((int)p.tokens, t0 + p.run);
  SeqCursor c(p);
  if (!c.seek(t0)) return;  // rows behind the last sequence stay as they are
  ConvTaps<E, V, W> tap;
  tap.load(p, c0);
  float win[W][V];  // inputs t-W+1 .. t
#pragma unroll
  for (int k = 0; k < W - 1; ++k) conv_input<E, V, W>(p, c, t0 - c.start - (W - 1) + k, c0, win[k]);
  const E* xp = static_cast<const E*>(p.x) + t0 * p.x_stride + c0;
  E* yp = static_cast<E*>(p.y) + (int64_t)t0 * p.D + c0;
  typename IO::raw raw[CONV_AHEAD];
  for (int t = t0; t < t1; t += CONV_AHEAD) {
#pragma unroll
    for (int a = 0; a < CONV_AHEAD; ++a) {
      if (t + a < t1) raw[a] = IO::load(xp);
      xp += p.x_stride;
    }
#pragma unroll
    for (int a = 0; a < CONV_AHEAD; ++a) {
      if (t + a >= t1) break;
      if (t + a == c.end) {
        if (!c.next()) return;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) conv_input<E, V, W>(p, c, k - (W - 1), c0, win[k]);
      }
      IO::get(raw[a], win[W - 1]);
      float y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = tap.b[e];
#pragma unroll
        for (int k = 0; k < W; ++k) u += tap.w[k][e] * win[k][e];
        y[e] = p.silu ? silu_gate<E>(u) : u;
      }
      store_vec<E, V>(yp, y);
      yp += p.D;
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) win[k][e] = win[k + 1][e];
    }
  }
}

// Gradient.  With du_t = dy_t act'(u_t) (u recomputed from x):
//   dx_s = sum_k w_k du_{s+W-1-k}     dw_k = sum_t du_t x_{t-W+1+k}     dbias = sum_t du_t
// where s may lie in the initial state, and the final state's gradient is added
// to the positions it copied.  A thread walks its run and the W-1 tokens behind
// it, with the W partial sums of dx that are still open in registers; dw and
// dbias sum the run's own tokens, one fp32 row of parts per run, joined by
// conv_dw_kernel in a fixed order.
// Blocks [0, nb_run) walk the runs; the rest write dinit of empty sequences.
template <class E, int V, int W>
__global__ __launch_bounds__(CONV_NT) void conv_bwd_kernel(ConvParams p, int64_t nb_run) {
  typedef VecIO<E, V> IO;
  const int CV = p.D / V;
  if (blockIdx.x >= nb_run) {
    const int64_t i = (blockIdx.x - nb_run) * CONV_NT + threadIdx.x;
    if (i >= (int64_t)p.N * (W - 1) * CV) return;
    const int c0 = (int)(i % CV) * V;
    SeqCursor c(p);
    c.n = (int)(i / CV / (W - 1));
    c.bounds();
    if (c.end > c.start) return;
    float f[V] = {};
    const int64_t off = (i / CV) * p.D + c0;
    if (p.dfin) IO::get(IO::load(static_cast<const E*>(p.dfin) + off), f);
    store_vec<E, V>(static_cast<E*>(p.dinit) + off, f);
    return;
  }
  const int64_t i = blockIdx.x * (int64_t)CONV_NT + threadIdx.x;
  const int64_t run = i / CV;
  if (run >= p.nruns) return;
  const int c0 = (int)(i - run * CV) * V;
  const int t0 = (int)run * p.run, t1 = min((int)p.tokens, t0 + p.run);
  SeqCursor c(p);
  float dw[W][V] = {}, db[V] = {};
  if (c.seek(t0)) {
    ConvTaps<E, V, W> tap;
    tap.load(p, c0);
    float win[W][V], acc[W][V] = {};  // inputs and open dx sums of positions t-W+1 .. t
#pragma unroll
    for (int k = 0; k < W - 1; ++k) conv_input<E, V, W>(p, c, t0 - c.start - (W - 1) + k, c0, win[k]);
    const E* xp = static_cast<const E*>(p.x) + t0 * p.x_stride + c0;
    const E* gp = static_cast<const E*>(p.dy) + (int64_t)t0 * p.D + c0;
    // the sum of position s (of the current sequence) is complete
    auto emit = [&](int s, const float (&a)[V]) {
      const bool tok = s >= c.start;
      if (tok ? (s < t0 || s >= t1) : (!p.dinit || c.start < t0 || c.start >= t1)) return;
      float f[V];
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = a[e];
      if (p.dfin && s >= c.end - (W - 1)) {
        float g[V];
        IO::get(IO::load(static_cast<const E*>(p.dfin) + ((int64_t)c.n * (W - 1) + s - (c.end - (W - 1))) * p.D + c0), g);
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] += g[e];
      }
      if (tok) stream_vec<E, V>(static_cast<E*>(p.dx) + (int64_t)s * p.D + c0, f);
      else store_vec<E, V>(static_cast<E*>(p.dinit) + ((int64_t)c.n * (W - 1) + s - c.start + W - 1) * p.D + c0, f);
    };
    // tokens t0 .. t1 + W - 2, of which those behind t1 only while the sequence lasts
    const int last = min((int)p.tokens, t1 + W - 1);
    bool more = true;
    typename IO::raw rx[CONV_AHEAD], rg[CONV_AHEAD];
    for (int t = t0; t < last && more; t += CONV_AHEAD) {
#pragma unroll
      for (int a = 0; a < CONV_AHEAD; ++a) {
        if (t + a < last) {
          rx[a] = IO::load(xp);
          rg[a] = IO::load(gp);
        }
        xp += p.x_stride;
        gp += p.D;
      }
#pragma unroll
      for (int a = 0; a < CONV_AHEAD; ++a) {
        const int s = t + a;
        if (s >= last || !more) break;
        IO::get(rx[a], win[W - 1]);
        float g[V];
        IO::get(rg[a], g);
        const bool mine = s < t1;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float u = tap.b[e];
#pragma unroll
          for (int k = 0; k < W; ++k) u += tap.w[k][e] * win[k][e];
          // computed either way and chosen (fp32's longer gate would become a branch, which
          // waits for every load: 8,192 x 1,001 in 44 us instead of 36)
          float gated = g[e] * dsilu_gate(u, fast_sigmoid<E>(u));
          if constexpr (sizeof(E) == 4) pin(gated);
          const float du = p.silu ? gated : g[e];
#pragma unroll
          for (int k = 0; k < W; ++k) acc[k][e] += tap.w[k][e] * du;
          if (mine) {
            db[e] += du;
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][e] += du * win[k][e];
          }
        }
        emit(s - (W - 1), acc[0]);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            acc[k][e] = k + 1 < W ? acc[k + 1 < W ? k + 1 : k][e] : 0.f;
            if (k + 1 < W) win[k][e] = win[k + 1 < W ? k + 1 : k][e];
          }
        if (s + 1 == c.end) {
#pragma unroll
          for (int k = 0; k < W - 1; ++k) {
            emit(s + 1 - (W - 1) + k, acc[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[k][e] = 0.f;
          }
          more = s + 1 < t1 && c.next();
          if (more) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) conv_input<E, V, W>(p, c, k - (W - 1), c0, win[k]);
          }
        }
      }
    }
  }
  float* part = p.part + run * (W + 1) * p.D + c0;
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) part[(int64_t)k * p.D + e] = k < W ? dw[k < W ? k : 0][e] : db[e];
}

// dw and dbias: column sums of the runs' parts in 64 bits (an fp32 sum has at most a
// run's terms), 32 columns a workgroup, sixteen threads a column, each over every
// sixteenth run.
constexpr int DW_COLS = 32, DW_ROWS = 16;
template <class E, int W>
__global__ __launch_bounds__(DW_COLS * DW_ROWS) void conv_dw_kernel(ConvParams p) {
  __shared__ double red[DW_ROWS][DW_COLS + 1];
  const int cl = threadIdx.x % DW_COLS, rl = threadIdx.x / DW_COLS;
  const int64_t cols = (int64_t)(W + 1) * p.D, col = blockIdx.x * (int64_t)DW_COLS + cl;
  double s = 0.;
  if (col < cols) {
#pragma unroll 8
    for (int64_t r = rl; r < p.nruns; r += DW_ROWS) s += p.part[r * cols + col];
  }
  red[rl][cl] = s;
  __syncthreads();
  if (rl == 0 && col < cols) {
    s = 0.;
#pragma unroll
    for (int r = 0; r < DW_ROWS; ++r) s += red[r][cl];
    const int k = (int)(col / p.D), d = (int)(col % p.D);
    if (k < W) static_cast<E*>(p.dw)[(int64_t)d * W + k] = to_e<E>((float)s);
    else if (p.dbias) static_cast<E*>(p.dbias)[d] = to_e<E>((float)s);
  }
}

// One token for each of N sequences: y from the slot's W-1 inputs and x, then
// the slot drops its oldest input and takes x.
template <class E, int V, int W>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvStepParams p) {
  typedef VecIO<E, V> IO;
  const int CV = p.D / V;
  const int64_t i = blockIdx.x * 64ll + threadIdx.x;
  if (i >= (int64_t)p.N * CV) return;
  const int n = (int)(i / CV), c0 = (int)(i - (int64_t)n * CV) * V;
  const int slot = p.state_idx ? p.state_idx[n] : n;
  if (slot < 0 || slot >= p.num_slots) return;  // padding entry
  E* st = static_cast<E*>(p.state) + (int64_t)slot * (W - 1) * p.D + c0;
  typename IO::raw raw[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) raw[k] = IO::load(st + (int64_t)k * p.D);
  raw[W - 1] = IO::load(static_cast<const E*>(p.x) + n * p.x_stride + c0);
  ConvTaps<E, V, W> tap;
  tap.load(p.w, p.bias, c0);
  float y[V];
#pragma unroll
  for (int e = 0; e < V; ++e) y[e] = tap.b[e];
#pragma unroll
  for (int k = 0; k < W; ++k) {
    float f[V];
    IO::get(raw[k], f);
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] += tap.w[k][e] * f[e];
    if (k > 0) store_vec<E, V>(st + (int64_t)(k - 1) * p.D, f);
  }
  if (p.silu) {
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = silu_gate<E>(y[e]);
  }
  store_vec<E, V>(static_cast<E*>(p.y) + (int64_t)n * p.D + c0, y);
}

template <class E, int V, int W>
hipError_t conv_launch(const ConvParams& p, bool bwd, hipStream_t st) {
  const int64_t CV = p.D / V;
  const int64_t nb_run = (p.nruns * CV + CONV_NT - 1) / CONV_NT;
  const bool tail = bwd ? p.dinit != nullptr : p.fin != nullptr;
  const int64_t nb = nb_run + (tail ? ((int64_t)p.N * (W - 1) * CV + CONV_NT - 1) / CONV_NT : 0);
  if (nb == 0) return hipSuccess;
  if (bwd) hipLaunchKernelGGL((conv_bwd_kernel<E, V, W>), dim3(nb), dim3(CONV_NT), 0, st, p, nb_run);
  else hipLaunchKernelGGL((conv_fwd_kernel<E, V, W>), dim3(nb), dim3(CONV_NT), 0, st, p, nb_run);
  return hipGetLastError();
}

// The gradient takes four channels a thread in either type: with eight its open
// sums, taps and parts need 212 registers, which leaves two waves a SIMD (199 us
// against 192 us for 49,828 x 2,304 bf16, W = 4, both before the streamed stores).
template <class E, int W>
hipError_t conv_launch_v(bool vec, const ConvParams& p, bool bwd, hipStream_t st) {
  if (!vec) return conv_launch<E, 1, W>(p, bwd, st);
  return bwd ? conv_launch<E, 4, W>(p, bwd, st) : conv_launch<E, kVec<E>, W>(p, bwd, st);
}
template <class E>
hipError_t conv_launch_w(int W, bool vec, const ConvParams& p, bool bwd, hipStream_t st) {
  if (W == 2) return conv_launch_v<E, 2>(vec, p, bwd, st);
  if (W == 3) return conv_launch_v<E, 3>(vec, p, bwd, st);
  if (W == 4) return conv_launch_v<E, 4>(vec, p, bwd, st);
  return hipErrorInvalidValue;
}

template <class E, int V, int W>
hipError_t step_launch(const ConvStepParams& p, hipStream_t st) {
  const int64_t nb = ((int64_t)p.N * (p.D / V) + 63) / 64;
  hipLaunchKernelGGL((conv_step_kernel<E, V, W>), dim3(nb), dim3(64), 0, st, p);
  return hipGetLastError();
}
template <class E>
hipError_t step_launch_w(int W, bool vec, const ConvStepParams& p, hipStream_t st) {
  if (W == 2) return vec ? step_launch<E, kVec<E>, 2>(p, st) : step_launch<E, 1, 2>(p, st);
  if (W == 3) return vec ? step_launch<E, kVec<E>, 3>(p, st) : step_launch<E, 1, 3>(p, st);
  if (W == 4) return vec ? step_launch<E, kVec<E>, 4>(p, st) : step_launch<E, 1, 4>(p, st);
  return hipErrorInvalidValue;
}

template <class E>
hipError_t dw_launch(int W, const ConvParams& p, hipStream_t st) {
  const int64_t nb = ((int64_t)(W + 1) * p.D + DW_COLS - 1) / DW_COLS;
  const dim3 g(nb), b(DW_COLS * DW_ROWS);
  if (W == 2) hipLaunchKernelGGL((conv_dw_kernel<E, 2>), g, b, 0, st, p);
  else if (W == 3) hipLaunchKernelGGL((conv_dw_kernel<E, 3>), g, b, 0, st, p);
  else if (W == 4) hipLaunchKernelGGL((conv_dw_kernel<E, 4>), g, b, 0, st, p);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_fwd(int dtype, int W, bool vec, const ConvParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? conv_launch_w<bf16>(W, vec, p, false, st) : conv_launch_w<float>(W, vec, p, false, st);
}
hipError_t launch_conv_bwd(int dtype, int W, bool vec, const ConvParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? conv_launch_w<bf16>(W, vec, p, true, st) : conv_launch_w<float>(W, vec, p, true, st);
}
hipError_t launch_conv_dw(int dtype, int W, const ConvParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? dw_launch<bf16>(W, p, st) : dw_launch<float>(W, p, st);
}
hipError_t launch_conv_step(int dtype, int W, bool vec, const ConvStepParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? step_launch_w<bf16>(W, vec, p, st) : step_launch_w<float>(W, vec, p, st);
}

}  // namespace gdn
