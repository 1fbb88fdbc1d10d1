// gdn_addnorm.hip -- residual norm (rows of D channels), its output in the input's
// type or in 8 bits with a scale a row, its gradient; rows in 8 bits alone.
//
//   s = x + r (stored in r's type),  y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   top = max(max |y|, 2^-100),  scale = top / 448,  q = e4m3(448 y / top)
//   dv = (dy w - n mean(dy w n)) rstd + ds,  n = s rstd,  dw = sum over rows of dy n
//
// Bound: memory.  A row lies in the registers of TPR threads, NV vectors of 16 bytes
// of x each, so that the sum, the statistics, the largest magnitude and the output
// take one read.  A wave a row (TPR = 64) needs no barrier for its sums; few rows
// (a decode batch) are spread over 256 threads each.  Rows too long for registers are
// re-read by a workgroup.
// Measured (bf16): 32,768 x 2,048 with residual, in 8 bits 74-101 us (470 MB, 6.3-4.7
// TB/s, by what the caches hold), 64 rows 4 us, all of it latency; 12,345 x 2,304 on an fp32
// stream forward 59-66 us (341 MB), gradient 97-104 us (455 MB, 4.5 TB/s) and 6 us for the
// weight's sums; 6,144 x 2,048 in 8 bits 8 us.
#include "gdn_block.h"

namespace gdn {

namespace {

constexpr int AN_NT = 256;
enum { OUT_Y = 0, OUT_Q = 1, OUT_QUANT = 2 };  // the norm's output, the same in 8 bits, x in 8 bits

template <class E> constexpr int kAV = 16 / (int)sizeof(E);  // elements of one vector

// Sum (or maximum) over the TPR threads of a row, in each of them.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_join(float x, float* red) {
#pragma unroll
  for (int o = 1; o < (TPR < 64 ? TPR : 64); o <<= 1) {
    const float t = __shfl_xor(x, o, 64);
    x = MAX ? fmaxf(x, t) : x + t;
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;  // waves of a row
    __syncthreads();
    if (lane_id() == 0) red[wave_id()] = x;
    __syncthreads();
    const float* q = red + wave_id() / W * W;
    x = q[0];
#pragma unroll
    for (int w = 1; w < W; ++w) x = MAX ? fmaxf(x, q[w]) : x + q[w];
  }
  return x;
}

// 448 v / top, rounded to e4m3.  v 448 comes first and the quotient is corrected once,
// so that one that lies halfway between two 8-bit values comes out exactly (v bf16: v 448
// is exact) and is rounded to even; 448 = 0.875 * 2^9 keeps large v in range.
struct Quant {
  float top, inv;
  __device__ __forceinline__ explicit Quant(float most) : top(fmaxf(most, 0x1p-100f)) { inv = 1.f / top; }
  __device__ __forceinline__ float scale() const { return top / 448.f; }
  __device__ __forceinline__ float operator()(float v) const {
    const float t = 0.875f * v, q = t * inv;
    return fmaf(fmaf(-q, top, t), inv, q) * 512.f;
  }
};
// n of the V values of a vector as bytes.
template <int V>
__device__ __forceinline__ void st_q8(uint8_t* p, int n, const float (&f)[V]) {
  uint32_t d[V / 4];
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    int t = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j], f[4 * j + 1], 0, false);
    d[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2], f[4 * j + 3], t, true);
  }
  typedef uint32_t u32_any __attribute__((aligned(1)));
  if (n >= V) {
    if constexpr (V == 8) {
      typedef uint32_t u32x2 __attribute__((__vector_size__(8)));
      typedef u32x2 u32x2_any __attribute__((aligned(1)));
      __builtin_nontemporal_store(u32x2{d[0], d[1]}, reinterpret_cast<u32x2_any*>(p));
    } else {
      __builtin_nontemporal_store(d[0], reinterpret_cast<u32_any*>(p));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = (uint8_t)(d[i / 4] >> (8 * (i % 4)));
  }
}

// Adds r's vector to v and rounds the sum to r's type, as it is stored.
template <class E, class RT, int V>
__device__ __forceinline__ void add_residual(const AddNormParams& p, int64_t row, int c, float (&v)[V]) {
  float t[V];
  ld_part<V>(static_cast<const RT*>(p.r) + row * p.r_stride + c, p.D - c, t);
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = to_f(to_e<RT>(v[e] + t[e]));
}

template <class E, int TPR, int NV, int OUT>
__global__ __launch_bounds__(AN_NT) void addnorm_fwd_kernel(AddNormParams p, int res_f32) {
  constexpr int V = kAV<E>, RPB = AN_NT / TPR;
  __shared__ float red[AN_NT / 64];
  const int lane = threadIdx.x % TPR;
  const int64_t r0 = block_2d() * RPB + threadIdx.x / TPR, row = min(r0, p.R - 1);
  const bool live = r0 < p.R;
  const E* xp = static_cast<const E*>(p.x) + row * p.x_stride;
  float v[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * V;
    ld_part<V>(xp + c, p.D - c, v[i]);
  }
  if constexpr (OUT != OUT_QUANT) {
    if (p.r) {
      // (the two types apart, so that all loads of either are requested together)
      if (res_f32) {
#pragma unroll
        for (int i = 0; i < NV; ++i) add_residual<E, float, V>(p, row, (i * TPR + lane) * V, v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) add_residual<E, E, V>(p, row, (i * TPR + lane) * V, v[i]);
      }
      if (live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + lane) * V;
          if (res_f32) st_part<V>(static_cast<float*>(p.s) + row * p.D + c, p.D - c, v[i]);
          else st_part<V>(static_cast<E*>(p.s) + row * p.D + c, p.D - c, v[i]);
        }
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) ss += v[i][e] * v[i][e];
    const float rstd = 1.f / sqrtf(row_join<TPR, false>(ss, red) / p.D + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      float w[V];
      ld_part<V>(static_cast<const E*>(p.w) + c, p.D - c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = v[i][e] * rstd * w[e];
    }
  }
  if constexpr (OUT == OUT_Y) {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      st_part<V>(static_cast<E*>(p.y) + row * p.D + c, p.D - c, v[i]);
    }
  } else {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) most = fmaxf(most, fabsf(v[i][e]));
    const Quant q(row_join<TPR, true>(most, red));
    if (!live) return;
    if (lane == 0) p.q_scale[row] = q.scale();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = q(v[i][e]);
      st_q8<V>(p.q + row * p.D + c, p.D - c, v[i]);
    }
  }
}

// Rows too long for registers: a workgroup per row re-reads the sum, which each
// thread has stored itself, for every pass.
template <class E, int OUT>
__global__ __launch_bounds__(AN_NT) void addnorm_fwd_long_kernel(AddNormParams p, int res_f32) {
  constexpr int V = kAV<E>;
  __shared__ float red[AN_NT / 64];
  const int64_t row = block_2d();
  if (row >= p.R) return;
  const bool res = OUT != OUT_QUANT && p.r != nullptr;
  const E* xp = static_cast<const E*>(p.x) + row * p.x_stride;
  auto sum_at = [&](int c, float (&v)[V]) {
    if (!res) ld_part<V>(xp + c, p.D - c, v);
    else if (res_f32) ld_part<V>(static_cast<const float*>(p.s) + row * p.D + c, p.D - c, v);
    else ld_part<V>(static_cast<const E*>(p.s) + row * p.D + c, p.D - c, v);
  };
  float rstd = 1.f;
  if constexpr (OUT != OUT_QUANT) {
    float ss = 0.f;
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V) {
      float v[V];
      ld_part<V>(xp + c, p.D - c, v);
      if (res && res_f32) {
        add_residual<E, float, V>(p, row, c, v);
        st_part<V>(static_cast<float*>(p.s) + row * p.D + c, p.D - c, v);
      } else if (res) {
        add_residual<E, E, V>(p, row, c, v);
        st_part<V>(static_cast<E*>(p.s) + row * p.D + c, p.D - c, v);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) ss += v[e] * v[e];
    }
    rstd = 1.f / sqrtf(row_join<AN_NT, false>(ss, red) / p.D + p.eps);
  }
  auto out_at = [&](int c, float (&v)[V]) {
    sum_at(c, v);
    if constexpr (OUT != OUT_QUANT) {
      float w[V];
      ld_part<V>(static_cast<const E*>(p.w) + c, p.D - c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = v[e] * rstd * w[e];
    }
  };
  if constexpr (OUT == OUT_Y) {
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V) {
      float v[V];
      out_at(c, v);
      st_part<V>(static_cast<E*>(p.y) + row * p.D + c, p.D - c, v);
    }
  } else {
    float most = 0.f;
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V) {
      float v[V];
      out_at(c, v);
#pragma unroll
      for (int e = 0; e < V; ++e) most = fmaxf(most, fabsf(v[e]));
    }
    const Quant q(row_join<AN_NT, true>(most, red));
    if (threadIdx.x == 0) p.q_scale[row] = q.scale();
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V) {
      float v[V];
      out_at(c, v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = q(v[e]);
      st_q8<V>(p.q + row * p.D + c, p.D - c, v);
    }
  }
}

// Gradient.  p.blocks workgroups walk the rows, each thread always on the same
// columns, and keep dw in registers: at most ADDNORM_ROWS rows a thread.  A workgroup's threads
// of one column are added in fp32, the workgroups' parts in 64 bits (join_parts_kernel).
template <class E, class RT, int TPR, int NV>
__global__ __launch_bounds__(AN_NT) void addnorm_bwd_kernel(AddNormParams p) {
  constexpr int V = kAV<E>, RPB = AN_NT / TPR;
  __shared__ float red[AN_NT / 64];
  __shared__ float cols[RPB > 1 ? RPB * TPR * V : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float dw[NV][V] = {};
  for (int64_t base = blockIdx.x * (int64_t)RPB; base < p.R; base += (int64_t)p.blocks * RPB) {
    const int64_t row = min(base + sub, p.R - 1);
    const bool live = base + sub < p.R;
    float n[NV][V], d[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      ld_part<V>(static_cast<const RT*>(p.s) + row * p.x_stride + c, p.D - c, n[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      ld_part<V>(static_cast<const E*>(p.dy) + row * p.D + c, p.D - c, d[i]);
    }
    float ss = 0.f, c1 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      float w[V];
      ld_part<V>(static_cast<const E*>(p.w) + c, p.D - c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ss += n[i][e] * n[i][e];
        c1 += d[i][e] * w[e] * n[i][e];
      }
    }
    const float rstd = 1.f / sqrtf(row_join<TPR, false>(ss, red) / p.D + p.eps);
    c1 = row_join<TPR, false>(c1, red) * rstd / p.D;
    if (!live) continue;  // (one row a workgroup: all threads live)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      float w[V], g[V] = {};
      ld_part<V>(static_cast<const E*>(p.w) + c, p.D - c, w);
      if (p.ds) ld_part<V>(static_cast<const RT*>(p.ds) + row * p.D + c, p.D - c, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float ne = n[i][e] * rstd;
        dw[i][e] += d[i][e] * ne;
        g[e] += (d[i][e] * w[e] - ne * c1) * rstd;
      }
      if (p.dx) st_part<V>(static_cast<E*>(p.dx) + row * p.D + c, p.D - c, g);
      if (p.dr) st_part<V>(static_cast<RT*>(p.dr) + row * p.D + c, p.D - c, g);
    }
  }
  if (!p.dw) return;
  float* part = p.part + blockIdx.x * (int64_t)p.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * V;
    if constexpr (RPB > 1) {  // over the workgroup's rows' threads
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) cols[(sub * V + e) * TPR + lane] = dw[i][e];
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = 0.f;
          for (int r = 0; r < RPB; ++r) s += cols[(r * V + e) * TPR + lane];
          dw[i][e] = s;
        }
      }
    }
    if (sub == 0) st_part<V>(part + c, p.D - c, dw[i]);
  }
}

template <class E, class RT>
__global__ __launch_bounds__(AN_NT) void addnorm_bwd_long_kernel(AddNormParams p) {
  constexpr int V = kAV<E>;
  __shared__ float red[AN_NT / 64];
  float* part = p.part + blockIdx.x * (int64_t)p.D;  // thread-owned columns
  if (p.dw)
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V)
      for (int e = 0; e < V && c + e < p.D; ++e) part[c + e] = 0.f;
  for (int64_t row = blockIdx.x; row < p.R; row += p.blocks) {
    const RT* sp = static_cast<const RT*>(p.s) + row * p.x_stride;
    const E* dp = static_cast<const E*>(p.dy) + row * p.D;
    const E* wp = static_cast<const E*>(p.w);
    float ss = 0.f, c1 = 0.f;
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V) {
      float n[V], d[V], w[V];
      ld_part<V>(sp + c, p.D - c, n);
      ld_part<V>(dp + c, p.D - c, d);
      ld_part<V>(wp + c, p.D - c, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ss += n[e] * n[e];
        c1 += d[e] * w[e] * n[e];
      }
    }
    const float rstd = 1.f / sqrtf(row_join<AN_NT, false>(ss, red) / p.D + p.eps);
    c1 = row_join<AN_NT, false>(c1, red) * rstd / p.D;
    for (int c = threadIdx.x * V; c < p.D; c += AN_NT * V) {
      float n[V], d[V], w[V], g[V] = {};
      ld_part<V>(sp + c, p.D - c, n);
      ld_part<V>(dp + c, p.D - c, d);
      ld_part<V>(wp + c, p.D - c, w);
      if (p.ds) ld_part<V>(static_cast<const RT*>(p.ds) + row * p.D + c, p.D - c, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float ne = n[e] * rstd;
        if (p.dw && c + e < p.D) part[c + e] += d[e] * ne;
        g[e] += (d[e] * w[e] - ne * c1) * rstd;
      }
      if (p.dx) st_part<V>(static_cast<E*>(p.dx) + row * p.D + c, p.D - c, g);
      if (p.dr) st_part<V>(static_cast<RT*>(p.dr) + row * p.D + c, p.D - c, g);
    }
  }
}

// 32 columns a workgroup, sixteen threads a column.
constexpr int JOIN_ROWS = 16;
template <class E>
__global__ __launch_bounds__(32 * JOIN_ROWS) void join_parts_kernel(const float* part, int64_t rows, int64_t cols, E* out) {
  __shared__ double red[JOIN_ROWS][33];
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t col = block_2d() * 32 + cl;
  double s = 0.;
  if (col < cols) {
#pragma unroll 8
    for (int64_t b = rl; b < rows; b += JOIN_ROWS) s += part[b * cols + col];
  }
  red[rl][cl] = s;
  __syncthreads();
  if (rl == 0 && col < cols) {
    s = 0.;
#pragma unroll
    for (int r = 0; r < JOIN_ROWS; ++r) s += red[r][cl];
    out[col] = to_e<E>((float)s);
  }
}

template <class E, int OUT, int TPR, int NV>
hipError_t an_fwd(const AddNormParams& p, int res_f32, hipStream_t st) {
  constexpr int RPB = AN_NT / TPR;
  hipLaunchKernelGGL((addnorm_fwd_kernel<E, TPR, NV, OUT>), blocks_2d((p.R + RPB - 1) / RPB), dim3(AN_NT), 0, st, p, res_f32);
  return hipGetLastError();
}
template <class E, int OUT>
hipError_t an_fwd_any(const AddNormParams& p, int res_f32, hipStream_t st) {
  const int nv = (p.D + kAV<E> - 1) / kAV<E>;
  if (nv <= 16) return an_fwd<E, OUT, 16, 1>(p, res_f32, st);
  if (nv <= 64) return an_fwd<E, OUT, 64, 1>(p, res_f32, st);
  if (p.R > 1024) {  // a wave a row: the chip is full without splitting rows
    if (nv <= 128) return an_fwd<E, OUT, 64, 2>(p, res_f32, st);
    if (nv <= 192) return an_fwd<E, OUT, 64, 3>(p, res_f32, st);
    if (nv <= 256) return an_fwd<E, OUT, 64, 4>(p, res_f32, st);
    if (nv <= 320) return an_fwd<E, OUT, 64, 5>(p, res_f32, st);
    if (nv <= 384) return an_fwd<E, OUT, 64, 6>(p, res_f32, st);
    if (nv <= 512) return an_fwd<E, OUT, 64, 8>(p, res_f32, st);
  }
  if (nv <= 256) return an_fwd<E, OUT, 256, 1>(p, res_f32, st);
  if (nv <= 512) return an_fwd<E, OUT, 256, 2>(p, res_f32, st);
  if (nv <= 768) return an_fwd<E, OUT, 256, 3>(p, res_f32, st);
  if (nv <= 1024) return an_fwd<E, OUT, 256, 4>(p, res_f32, st);
  if (nv <= 1536) return an_fwd<E, OUT, 256, 6>(p, res_f32, st);
  if (nv <= 2048) return an_fwd<E, OUT, 256, 8>(p, res_f32, st);
  hipLaunchKernelGGL((addnorm_fwd_long_kernel<E, OUT>), blocks_2d(p.R), dim3(AN_NT), 0, st, p, res_f32);
  return hipGetLastError();
}

template <class E, class RT, int TPR, int NV>
hipError_t an_bwd(const AddNormParams& p, hipStream_t st) {
  hipLaunchKernelGGL((addnorm_bwd_kernel<E, RT, TPR, NV>), dim3(p.blocks), dim3(AN_NT), 0, st, p);
  return hipGetLastError();
}
// Threads of a row in the gradient, for a row of nv vectors.
int an_bwd_tpr(int nv) { return nv <= 16 ? 16 : nv <= 256 ? 64 : nv <= 384 ? 128 : 256; }
template <class E, class RT>
hipError_t an_bwd_any(const AddNormParams& p, hipStream_t st) {
  const int nv = (p.D + kAV<E> - 1) / kAV<E>;
  if (nv <= 16) return an_bwd<E, RT, 16, 1>(p, st);
  if (nv <= 64) return an_bwd<E, RT, 64, 1>(p, st);
  if (nv <= 128) return an_bwd<E, RT, 64, 2>(p, st);
  if (nv <= 192) return an_bwd<E, RT, 64, 3>(p, st);
  if (nv <= 256) return an_bwd<E, RT, 64, 4>(p, st);
  if (nv <= 384) return an_bwd<E, RT, 128, 3>(p, st);
  if (nv <= 512) return an_bwd<E, RT, 256, 2>(p, st);
  if (nv <= 768) return an_bwd<E, RT, 256, 3>(p, st);
  if (nv <= 1024) return an_bwd<E, RT, 256, 4>(p, st);
  hipLaunchKernelGGL((addnorm_bwd_long_kernel<E, RT>), dim3(p.blocks), dim3(AN_NT), 0, st, p);
  return hipGetLastError();
}

}  // namespace

int addnorm_blocks(int64_t R, int D, int esize, int cus) {
  const int nv = (int)((D + 16ll / esize - 1) / (16 / esize));
  const int64_t rpb = nv <= 1024 ? AN_NT / an_bwd_tpr(nv) : 1;  // rows at a time
  const int64_t groups = (R + rpb - 1) / rpb;
  // as many as are resident at once, more where a thread would take too many rows
  return (int)std::max<int64_t>(1, std::max(std::min<int64_t>(groups, 3 * cus), (groups + ADDNORM_ROWS - 1) / ADDNORM_ROWS));
}

hipError_t launch_addnorm_fwd(int dtype, int res_dtype, const AddNormParams& p, hipStream_t st) {
  const int rf = res_dtype == GDN_F32;
  if (dtype == GDN_BF16) return p.q ? an_fwd_any<bf16, OUT_Q>(p, rf, st) : an_fwd_any<bf16, OUT_Y>(p, rf, st);
  return p.q ? an_fwd_any<float, OUT_Q>(p, rf, st) : an_fwd_any<float, OUT_Y>(p, rf, st);
}
hipError_t launch_quant_rows(int dtype, const AddNormParams& p, hipStream_t st) {
  return dtype == GDN_BF16 ? an_fwd_any<bf16, OUT_QUANT>(p, 0, st) : an_fwd_any<float, OUT_QUANT>(p, 0, st);
}
hipError_t launch_addnorm_bwd(int dtype, int res_dtype, const AddNormParams& p, hipStream_t st) {
  if (dtype == GDN_F32) return an_bwd_any<float, float>(p, st);
  return res_dtype == GDN_F32 ? an_bwd_any<bf16, float>(p, st) : an_bwd_any<bf16, bf16>(p, st);
}
hipError_t launch_join_parts(int dtype, const float* part, int64_t rows, int64_t cols, void* out, hipStream_t st) {
  const dim3 grid = blocks_2d((cols + 31) / 32);
  if (dtype == GDN_BF16)
    hipLaunchKernelGGL((join_parts_kernel<bf16>), grid, dim3(32 * JOIN_ROWS), 0, st, part, rows, cols, static_cast<bf16*>(out));
  else
    hipLaunchKernelGGL((join_parts_kernel<float>), grid, dim3(32 * JOIN_ROWS), 0, st, part, rows, cols, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace gdn
