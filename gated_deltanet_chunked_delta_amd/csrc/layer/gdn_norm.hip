// gdn_norm.hip -- gated group norm, channels last: every token's G groups of D
// channels are normalised on their own.
//
//   v = x                      (gate after the norm, or no gate)
//     = x silu(z)              (gate before it)
//   n = (v - mean) / sqrt(mean((v - mean)^2) + eps),   mean = 0 unless centred
//   o = n w + bias,   y = o silu(z) (gate after) or o
//
// Bound: memory -- x, z read and y written once (backward: x, z, dy read, dx,
// dz written).  A row (token and group) is held in registers by TPR threads,
// NV 16-byte vectors each, so that statistics, output and gradients take one
// read; TPR is the smallest power of two that covers the row with as few
// vectors as possible, so several short rows (a head of 64 or 128 channels)
// share a wave.  Rows too long for that are re-read by a whole workgroup.
// Measured (bf16, gated): 32,768 x 16 heads of 128 in 70 us (403 MB, 5.8 TB/s);
// 16,384 rows of 2,000 in 37 us (197 MB) and the gradient in 76 us (328 MB,
// 4.3 TB/s); 64 x 16 heads of 128 in 7 us, all of it latency.  Widths off 16 bytes take
// one element a thread and access, and past 1,024 of them the re-reading kernels:
// 16,384 x 999 bf16 in 41 us (2.4 TB/s) and 115 us (1.4), x 1,999 in 91 us and 565 us.
#include "gdn_layer.h"

namespace gdn {

namespace {

constexpr int NORM_NT = 256;
enum { GATE_NONE = 0, GATE_BEFORE = 1, GATE_AFTER = 2 };

// Sum over the TPR threads of a row, in each of them.  red: one float per wave.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int o = 1; o < (TPR < 64 ? TPR : 64); o <<= 1) x += __shfl_xor(x, o, 64);
  if (TPR > 64) {
    __syncthreads();
    if (lane_id() == 0) red[wave_id()] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < NORM_NT / 64; ++w) x += red[w];
  }
  return x;
}

// Hides a loaded vector's value from the optimizer, so that its conversions on
// either side are two computations and not one result held between them.
__device__ __forceinline__ void hide(bf16x8& r) {
  typedef uint32_t u32x4 __attribute__((__vector_size__(16)));
  u32x4 v = __builtin_bit_cast(u32x4, r);
  asm volatile("" : "+v"(v));
  r = __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ void hide(f32x4& r) { asm volatile("" : "+v"(r)); }
__device__ __forceinline__ void hide(float& r) { asm volatile("" : "+v"(r)); }
__device__ __forceinline__ void hide(bf16& r) {
  uint32_t v = __builtin_bit_cast(uint16_t, r);
  asm volatile("" : "+v"(v));
  r = __builtin_bit_cast(bf16, (uint16_t)v);
}

// One row's vectors, as loaded.
template <class E, int V, int TPR, int NV>
struct NormRow {
  typedef VecIO<E, V> IO;
  typename IO::raw v[NV];
  __device__ __forceinline__ void load(const void* base, int64_t off, int D, int lane) {
    const E* p = static_cast<const E*>(base) + off;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      v[i] = c < D ? IO::load(p + c) : IO::zero();
    }
  }
};

// RW rows at a time for each group of TPR threads, requested together: a row of
// one vector a thread alone leaves too little in flight.
template <class E, int V, int TPR, int NV, int RW, int GATE>
__global__ __launch_bounds__(NORM_NT) void norm_fwd_kernel(NormParams p) {
  typedef VecIO<E, V> IO;
  __shared__ float red[NORM_NT / 64];
  constexpr int RPB = NORM_NT / TPR;
  const int lane = threadIdx.x % TPR;
  const int64_t rows = p.R * p.G;
  const int64_t r0 = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * (RPB * RW) + threadIdx.x / TPR;
  constexpr bool before = GATE == GATE_BEFORE, after = GATE == GATE_AFTER;
  const float inv = 1.f / p.D;
  NormRow<E, V, TPR, NV> x[RW], z[RW];
  int grp[RW];
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    const uint32_t r = (uint32_t)min(r0 + k * RPB, rows - 1), tok = r / (uint32_t)p.G;
    grp[k] = (int)(r - tok * (uint32_t)p.G);
    x[k].load(p.x, tok * p.x_stride + (int64_t)grp[k] * p.D, p.D, lane);
    if (GATE) z[k].load(p.z, tok * p.z_stride + (int64_t)grp[k] * p.D, p.D, lane);
  }
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    const int64_t r = r0 + k * RPB;
    float v[NV][V], act[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      IO::get(x[k].v[i], v[i]);
      if (GATE) {
        IO::get(z[k].v[i], act[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) act[i][e] = silu_gate<E>(act[i][e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (before) v[i][e] *= act[i][e];
        s += v[i][e];
      }
    }
    float mean = 0.f;
    if (p.center) mean = row_sum<TPR>(s, red) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * TPR + lane) * V < p.D;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[i][e] = in ? v[i][e] - mean : 0.f;
        s += v[i][e] * v[i][e];
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(s, red) * inv + p.eps);
    if (r >= rows) continue;  // the same for a whole row's threads
    const int64_t wo = p.shared ? 0 : (int64_t)grp[k] * p.D;
    E* yp = static_cast<E*>(p.y) + r * p.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c >= p.D) continue;
      float w[V], b[V], y[V];
      IO::get(IO::load(static_cast<const E*>(p.w) + wo + c), w);
      if (p.bias) IO::get(IO::load(static_cast<const E*>(p.bias) + wo + c), b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[e] = v[i][e] * rstd * w[e];
        if (p.bias) y[e] += b[e];
        if (after) y[e] *= act[i][e];
      }
      stream_vec<E, V>(yp + c, y);
    }
  }
}

// Gradient.  With do = dy silu(z) (gate after) or dy, dn = do w:
//   dv = (dn - n mean(dn n) - [centred] mean(dn)) rstd
//   dx = dv (silu(z) with the gate before),  dw = sum do n,  dbias = sum do
//   dz = silu'(z) (dv x  with the gate before,  dy o  after it)
// p.blocks workgroups per weight group walk that group's rows, each thread
// always on the same columns, and keep dw and dbias in registers; their parts
// are joined by norm_dw_kernel in 64 bits and a fixed order.  Rows of one vector a
// thread are requested one ahead; a row is held as loaded (16 bytes a vector) and
// converted where it is used, which leaves registers for four vectors a thread.
template <class E, int V, int TPR, int NV, bool BIAS, int GATE>
__global__ __launch_bounds__(NORM_NT) void norm_bwd_kernel(NormParams p) {
  typedef VecIO<E, V> IO;
  constexpr int RPB = NORM_NT / TPR;
  __shared__ float red[NORM_NT / 64];
  __shared__ float cols[RPB > 1 ? RPB * TPR * V : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int wg = p.shared ? 0 : blockIdx.x / p.blocks, blk = blockIdx.x % p.blocks;
  const int64_t rows = p.shared ? p.R * p.G : p.R;  // of this weight group
  constexpr bool before = GATE == GATE_BEFORE, after = GATE == GATE_AFTER;
  const float inv = 1.f / p.D;
  // the next row in registers too, where that leaves room for three waves a SIMD
  constexpr bool AHEAD = NV == 1;
  float dw[NV][V] = {}, db[BIAS ? NV : 1][V] = {};
  NormRow<E, V, TPR, NV> x, z, gy, nx, nz, ng;
  auto request = [&](int64_t row) {
    const uint32_t rr = (uint32_t)min(row, rows - 1), tok = p.shared ? rr / (uint32_t)p.G : rr;
    const int g = p.shared ? (int)(rr - tok * (uint32_t)p.G) : wg;
    nx.load(p.x, tok * p.x_stride + (int64_t)g * p.D, p.D, lane);
    if (GATE) nz.load(p.z, tok * p.z_stride + (int64_t)g * p.D, p.D, lane);
    ng.load(p.dy, ((int64_t)tok * p.G + g) * p.D, p.D, lane);
  };
  if (AHEAD && (int64_t)blk * RPB < rows) request((int64_t)blk * RPB + sub);
  for (int64_t base = (int64_t)blk * RPB; base < rows; base += (int64_t)p.blocks * RPB) {
    const int64_t rr = min(base + sub, rows - 1);
    const bool live = base + sub < rows;
    const int64_t off = (p.shared ? rr : rr * p.G + wg) * p.D;
    if (!AHEAD) request(base + sub);
    x = nx;
    z = nz;
    gy = ng;
    if (AHEAD && base + (int64_t)p.blocks * RPB < rows) request(base + (int64_t)p.blocks * RPB + sub);
    float n[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      IO::get(x.v[i], n[i]);
      if (before) {
        float t[V];
        IO::get(z.v[i], t);
#pragma unroll
        for (int e = 0; e < V; ++e) n[i][e] *= silu_gate<E>(t[e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) s += n[i][e];
    }
    float mean = 0.f;
    if (p.center) mean = row_sum<TPR>(s, red) * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * TPR + lane) * V < p.D;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        n[i][e] = in ? n[i][e] - mean : 0.f;
        s += n[i][e] * n[i][e];
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(s, red) * inv + p.eps);
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (GATE) hide(z.v[i]);
      float w[V] = {}, d[V];
      if (c < p.D) IO::get(IO::load(static_cast<const E*>(p.w) + (int64_t)wg * p.D + c), w);
      IO::get(gy.v[i], d);
      if (after) {
        float t[V];
        IO::get(z.v[i], t);
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] *= silu_gate<E>(t[e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        n[i][e] *= rstd;
        const float dn = d[e] * w[e];
        c1 += dn * n[i][e];
        c2 += dn;
        if (live) {
          dw[i][e] += d[e] * n[i][e];
          if (BIAS) db[BIAS ? i : 0][e] += d[e];
        }
      }
    }
    c1 = row_sum<TPR>(c1, red) * inv;
    c2 = p.center ? row_sum<TPR>(c2, red) * inv : 0.f;
    if (!live) continue;  // (one row a workgroup: all threads live)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c >= p.D) continue;
      if (GATE) hide(z.v[i]);
      hide(gy.v[i]);
      typename IO::raw wr = IO::load(static_cast<const E*>(p.w) + (int64_t)wg * p.D + c);
      hide(wr);
      float w[V], d[V], dx[V];
      IO::get(wr, w);
      IO::get(gy.v[i], d);
      if (GATE) {
        float t[V], xv[V], b[V] = {}, dz[V];
        IO::get(z.v[i], t);
        if (before) IO::get(x.v[i], xv);
        else if (BIAS) IO::get(IO::load(static_cast<const E*>(p.bias) + (int64_t)wg * p.D + c), b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float sg = fast_sigmoid<E>(t[e]), act = t[e] * sg;
          const float dv = ((after ? d[e] * act : d[e]) * w[e] - n[i][e] * c1 - c2) * rstd;
          dx[e] = before ? dv * act : dv;
          dz[e] = (before ? dv * xv[e] : d[e] * (n[i][e] * w[e] + b[e])) * dsilu_gate(t[e], sg);
        }
        stream_vec<E, V>(static_cast<E*>(p.dz) + off + c, dz);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) dx[e] = (d[e] * w[e] - n[i][e] * c1 - c2) * rstd;
      }
      stream_vec<E, V>(static_cast<E*>(p.dx) + off + c, dx);
    }
  }
  // this workgroup's column sums: over its RPB rows' threads, then out
  constexpr int kinds = BIAS ? 2 : 1;
  float* part = p.part + ((int64_t)wg * p.blocks + blk) * kinds * p.D;
#pragma unroll
  for (int kind = 0; kind < kinds; ++kind) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      float s[V];
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] = kind ? db[BIAS ? i : 0][e] : dw[i][e];
      if (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) cols[(sub * V + e) * TPR + lane] = s[e];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            s[e] = 0.f;
            for (int r = 0; r < RPB; ++r) s[e] += cols[(r * V + e) * TPR + lane];
          }
        }
      }
      if (sub == 0 && c < p.D) {
#pragma unroll
        for (int e = 0; e < V; ++e) part[(int64_t)kind * p.D + c + e] = s[e];
      }
    }
  }
}

// Rows too long for registers: a workgroup per row re-reads it for each pass.
template <class E>
struct LongRow {
  const E *x, *z, *w, *b, *dy;
  bool before, after;
  float mean, rstd;
  __device__ __forceinline__ float gated(int c) const {
    const float v = to_f(x[c]);
    return before ? v * silu_gate<E>(to_f(z[c])) : v;
  }
  __device__ __forceinline__ void stats(const NormParams& p, float* red) {
    const float inv = 1.f / p.D;
    mean = 0.f;
    float s = 0.f;
    if (p.center) {
      for (int c = threadIdx.x; c < p.D; c += NORM_NT) s += gated(c);
      mean = row_sum<NORM_NT>(s, red) * inv;
      s = 0.f;
    }
    for (int c = threadIdx.x; c < p.D; c += NORM_NT) {
      const float v = gated(c) - mean;
      s += v * v;
    }
    rstd = 1.f / sqrtf(row_sum<NORM_NT>(s, red) * inv + p.eps);
  }
};
template <class E>
__device__ __forceinline__ LongRow<E> long_row(const NormParams& p, int64_t tok, int g) {
  LongRow<E> a;
  a.x = static_cast<const E*>(p.x) + tok * p.x_stride + (int64_t)g * p.D;
  a.z = static_cast<const E*>(p.z) + (p.z ? tok * p.z_stride + (int64_t)g * p.D : 0);
  const int64_t wo = p.shared ? 0 : (int64_t)g * p.D;
  a.w = static_cast<const E*>(p.w) + wo;
  a.b = p.bias ? static_cast<const E*>(p.bias) + wo : nullptr;
  a.dy = p.dy ? static_cast<const E*>(p.dy) + (tok * p.G + g) * p.D : nullptr;
  a.before = p.z && p.gate_first;
  a.after = p.z && !p.gate_first;
  return a;
}

template <class E>
__global__ __launch_bounds__(NORM_NT) void norm_fwd_long_kernel(NormParams p) {
  __shared__ float red[NORM_NT / 64];
  const int64_t r = blockIdx.y * (int64_t)gridDim.x + blockIdx.x, tok = r / p.G;
  if (r >= p.R * p.G) return;
  LongRow<E> a = long_row<E>(p, tok, (int)(r - tok * p.G));
  a.stats(p, red);
  E* y = static_cast<E*>(p.y) + r * p.D;
  for (int c = threadIdx.x; c < p.D; c += NORM_NT) {
    float o = (a.gated(c) - a.mean) * a.rstd * to_f(a.w[c]);
    if (a.b) o += to_f(a.b[c]);
    if (a.after) o *= silu_gate<E>(to_f(a.z[c]));
    y[c] = to_e<E>(o);
  }
}

template <class E>
__global__ __launch_bounds__(NORM_NT) void norm_bwd_long_kernel(NormParams p) {
  __shared__ float red[NORM_NT / 64];
  const int wg = p.shared ? 0 : blockIdx.x / p.blocks, blk = blockIdx.x % p.blocks;
  const int64_t rows = p.shared ? p.R * p.G : p.R;
  const float inv = 1.f / p.D;
  const int kinds = p.dbias ? 2 : 1;
  float* part = p.part + ((int64_t)wg * p.blocks + blk) * kinds * p.D;  // thread-owned columns
  for (int c = threadIdx.x; c < p.D; c += NORM_NT)
    for (int k = 0; k < kinds; ++k) part[(int64_t)k * p.D + c] = 0.f;
  for (int64_t r = blk; r < rows; r += p.blocks) {
    const int64_t tok = p.shared ? r / p.G : r;
    const int g = p.shared ? (int)(r - tok * p.G) : wg;
    LongRow<E> a = long_row<E>(p, tok, g);
    a.stats(p, red);
    float c1 = 0.f, c2 = 0.f;
    for (int c = threadIdx.x; c < p.D; c += NORM_NT) {
      const float gd = to_f(a.dy[c]) * (a.after ? silu_gate<E>(to_f(a.z[c])) : 1.f);
      const float n = (a.gated(c) - a.mean) * a.rstd, dn = gd * to_f(a.w[c]);
      c1 += dn * n;
      c2 += dn;
      part[c] += gd * n;
      if (p.dbias) part[p.D + c] += gd;
    }
    c1 = row_sum<NORM_NT>(c1, red) * inv;
    c2 = p.center ? row_sum<NORM_NT>(c2, red) * inv : 0.f;
    E* dx = static_cast<E*>(p.dx) + (tok * p.G + g) * p.D;
    E* dz = p.z ? static_cast<E*>(p.dz) + (tok * p.G + g) * p.D : nullptr;
    for (int c = threadIdx.x; c < p.D; c += NORM_NT) {
      const float z = p.z ? to_f(a.z[c]) : 0.f, sg = fast_sigmoid<E>(z), act = z * sg, dy = to_f(a.dy[c]);
      const float n = (a.gated(c) - a.mean) * a.rstd;
      const float dn = (a.after ? dy * act : dy) * to_f(a.w[c]);
      const float dv = (dn - n * c1 - c2) * a.rstd;
      dx[c] = to_e<E>(a.before ? dv * act : dv);
      if (dz) {
        const float dact = a.before ? dv * to_f(a.x[c]) : dy * (n * to_f(a.w[c]) + (a.b ? to_f(a.b[c]) : 0.f));
        dz[c] = to_e<E>(dact * dsilu_gate(z, sg));
      }
    }
  }
}

// dw and dbias: sums of the workgroups' parts in 64 bits, 32 columns a workgroup,
// sixteen threads a column.
constexpr int NDW_ROWS = 16;
template <class E>
__global__ __launch_bounds__(32 * NDW_ROWS) void norm_dw_kernel(NormParams p) {
  __shared__ double red[NDW_ROWS][33];
  const int kinds = p.dbias ? 2 : 1;
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t cols = (int64_t)kinds * p.D, col = blockIdx.x * 32ll + cl;
  const int wg = blockIdx.y;
  double s = 0.;
  if (col < cols) {
    const float* q = p.part + (int64_t)wg * p.blocks * cols + col;
#pragma unroll 8
    for (int b = rl; b < p.blocks; b += NDW_ROWS) s += q[b * cols];
  }
  red[rl][cl] = s;
  __syncthreads();
  if (rl == 0 && col < cols) {
    s = 0.;
#pragma unroll
    for (int r = 0; r < NDW_ROWS; ++r) s += red[r][cl];
    if (col < p.D) static_cast<E*>(p.dw)[(int64_t)wg * p.D + col] = to_e<E>((float)s);
    else static_cast<E*>(p.dbias)[(int64_t)wg * p.D + col - p.D] = to_e<E>((float)s);
  }
}

// A launch has fewer than 2^32 threads in x: more workgroups go on in y.
dim3 grid_2d(int64_t n) {
  constexpr int64_t most = 1 << 23;
  return n <= most ? dim3((uint32_t)n) : dim3((uint32_t)most, (uint32_t)((n + most - 1) / most));
}

// Enough workgroups of rpb rows at a time for NORM_ROWS rows a thread (as far as one
// launch goes: 2^24 workgroups in all).
void norm_grad_blocks(NormParams& p, int rpb) {
  const int64_t rows = p.shared ? p.R * p.G : p.R, most = ((1 << 24) - 1) / (p.shared ? 1 : p.G);
  p.blocks = max(p.blocks, (int)min((rows + rpb * NORM_ROWS - 1) / (rpb * NORM_ROWS), most));
}

template <class E, int V, int TPR, int NV, int GATE>
hipError_t norm_run_gate(NormParams& p, bool bwd, hipStream_t st) {
  const int64_t rows = p.R * p.G;
  if (bwd) {
    norm_grad_blocks(p, NORM_NT / TPR);
    const dim3 grid(p.blocks * (p.shared ? 1 : p.G));
    if (p.dbias) hipLaunchKernelGGL((norm_bwd_kernel<E, V, TPR, NV, true, GATE>), grid, dim3(NORM_NT), 0, st, p);
    else hipLaunchKernelGGL((norm_bwd_kernel<E, V, TPR, NV, false, GATE>), grid, dim3(NORM_NT), 0, st, p);
  } else {
    // four vectors a thread in flight, as long as the chip stays full of workgroups
    constexpr int RPB = NORM_NT / TPR, RW = V == 1 || NV >= 4 ? 1 : 4 / NV;
    if (rows >= (int64_t)RPB * RW * 1024)
      hipLaunchKernelGGL((norm_fwd_kernel<E, V, TPR, NV, RW, GATE>), grid_2d((rows + RPB * RW - 1) / (RPB * RW)), dim3(NORM_NT), 0, st, p);
    else
      hipLaunchKernelGGL((norm_fwd_kernel<E, V, TPR, NV, 1, GATE>), grid_2d((rows + RPB - 1) / RPB), dim3(NORM_NT), 0, st, p);
  }
  return hipGetLastError();
}
template <class E, int V, int TPR, int NV>
hipError_t norm_run(NormParams& p, bool bwd, hipStream_t st) {
  if (!p.z) return norm_run_gate<E, V, TPR, NV, GATE_NONE>(p, bwd, st);
  return p.gate_first ? norm_run_gate<E, V, TPR, NV, GATE_BEFORE>(p, bwd, st) : norm_run_gate<E, V, TPR, NV, GATE_AFTER>(p, bwd, st);
}

template <class E, int V>
hipError_t norm_pick(NormParams& p, bool bwd, hipStream_t st) {
  const int nv = (p.D + V - 1) / V;  // vectors in a row
  if constexpr (V > 1) {
    if (nv <= 8) return norm_run<E, V, 8, 1>(p, bwd, st);
    if (nv <= 16) return norm_run<E, V, 16, 1>(p, bwd, st);
    if (nv <= 32) return norm_run<E, V, 32, 1>(p, bwd, st);
  }
  if (nv <= 64) return norm_run<E, V, 64, 1>(p, bwd, st);
  if constexpr (V > 1)
    if (nv <= 128) return norm_run<E, V, 64, 2>(p, bwd, st);
  if (nv <= 256) return norm_run<E, V, 64, 4>(p, bwd, st);
  if constexpr (V > 1)
    if (nv <= 512) return norm_run<E, V, 256, 2>(p, bwd, st);
  if (nv <= 1024) return norm_run<E, V, 256, 4>(p, bwd, st);
  if (bwd) norm_grad_blocks(p, 1);
  if (bwd)
    hipLaunchKernelGGL((norm_bwd_long_kernel<E>), dim3(p.blocks * (p.shared ? 1 : p.G)), dim3(NORM_NT), 0, st, p);
  else
    hipLaunchKernelGGL((norm_fwd_long_kernel<E>), grid_2d(p.R * p.G), dim3(NORM_NT), 0, st, p);
  return hipGetLastError();
}

template <class E>
hipError_t norm_any(bool vec, NormParams p, bool bwd, hipStream_t st) {
  hipError_t e = vec ? norm_pick<E, kVec<E>>(p, bwd, st) : norm_pick<E, 1>(p, bwd, st);
  if (e != hipSuccess || !bwd) return e;
  const int kinds = p.dbias ? 2 : 1;
  hipLaunchKernelGGL((norm_dw_kernel<E>), dim3((kinds * (int64_t)p.D + 31) / 32, p.shared ? 1 : p.G),
                     dim3(32 * NDW_ROWS), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(int dtype, bool vec, const NormParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? norm_any<bf16>(vec, p, false, st) : norm_any<float>(vec, p, false, st);
}
hipError_t launch_norm_bwd(int dtype, bool vec, const NormParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? norm_any<bf16>(vec, p, true, st) : norm_any<float>(vec, p, true, st);
}

}  // namespace gdn
