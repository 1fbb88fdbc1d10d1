// gdn_scan_ops.hip -- the scan's smaller kernels: joins between segments, the
// gradients of step sizes and decays, the sums of dB and dC over a group's
// parts, and the single-token step.
#include "gdn_layer.h"
#include "gdn_scan_device.h"

namespace gdn {

namespace {

template <class E> __device__ __forceinline__ float ldE(const void* p, int64_t i) { return to_f(static_cast<const E*>(p)[i]); }

// Per (sequence, head): end states of the segments, each from a zero start,
// become the states entering them (in sweep order).  Four entries a thread; the
// states of JOIN_AHEAD segments are requested together, since the chain through
// them is only a multiply-add each.  Bound: the states, read and written (4 x 8
// segments of 16 heads of 128 x 128, 67 MB in 12 us), or the chain (128 segments of
// 4 heads, as many bytes, in 19; with one entry a thread, or the next eight requested
// ahead, within 2 us of that either way).
constexpr int JOIN_AHEAD = 8;
__global__ __launch_bounds__(256) void scan_join_kernel(ScanJoinParams p) {
  const int n = blockIdx.z, h = blockIdx.y;
  if (plan_invalid(p.seq, p.segs)) return;
  const int64_t ss = (int64_t)p.Dk * p.Dv, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int j0 = p.seq.cu ? p.seg_first[n] : n * p.seq.nseg_per_seq();
  const int ns = p.seq.nseg_of(p.seg_first, n);
  typedef f32x4 __attribute__((aligned(4))) f32x4_u;
  f32x4 carry = zero4();
  if (p.s0) carry = *reinterpret_cast<const f32x4_u*>(p.s0 + ((int64_t)n * p.H + h) * ss + e);
  for (int i0 = 0; i0 < ns; i0 += JOIN_AHEAD) {
    f32x4 loc[JOIN_AHEAD];
    float dec[JOIN_AHEAD];
    float* at[JOIN_AHEAD];
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k) {
      const int i = min(i0 + k, ns - 1);
      const int64_t j = j0 + (p.rev ? ns - 1 - i : i);
      at[k] = p.s_loc + (j * p.H + h) * ss + e;
      loc[k] = zero4();
      dec[k] = 0.f;
      if (i0 + k + 1 < ns) {  // the last segment's own end state is not formed
        loc[k] = *reinterpret_cast<const f32x4_u*>(at[k]);
        dec[k] = p.s_dec[j * p.H + h];
      }
    }
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k) {
      if (i0 + k >= ns) break;
      *reinterpret_cast<f32x4_u*>(at[k]) = carry;
      carry = carry * dec[k] + loc[k];
    }
  }
}

// ddt of every token and each chunk's sums for dA, dD and ddt_bias: a wave per
// (chunk, head), lane = token.  The recursion of da is a suffix sum of
// v_t = rt_t - D_t ct_t, undamped (a rounding stays in it to the chunk's start),
// so it and the sums over tokens are held in 64 bits, and what the sums miss the
// anchor at the chunk's start by is spread evenly over the tokens (a sequence's first
// chunk: zero without an h0; with one its product is not used).  Where a
// token's own decay is below fp32's unit round-off the recursion restarts with
// v_t = rt_t (cut): what is left of da_{t+1} - D_t ct_t = <., exp(a_t) h_{t-1}>
// there is below the rounding of its two parts, which |A| in ddt would multiply.
// 16,384 tokens of 16 heads: 9 us, and 4 for the sums (latency).
__global__ __launch_bounds__(64) void scan_grad_kernel(ScanGradParams p) {
  const int h = blockIdx.y, l = lane_id();
  const int64_t chunk = blockIdx.x;
  const int nsl = p.Dv / PS, g = h / (p.H / p.G);
  const int2 nc = p.seq.chunk_of(p.chunk_tab, (int)chunk);  // (sequence, chunk within it)
  if (nc.x < 0) return;  // the device cu_seqlens disagrees with the plan: nothing is written
  const int len = min(CH, p.seq.len(nc.x) - nc.y * CH);
  const int64_t row = p.seq.start(nc.x) + nc.y * CH + min(l, len - 1);
  const bool in = l < len;
  const float A = p.A[h];
  const float raw = scan_dt_raw(p.dt, p.dt_f32, row * p.dt_stride + h) + (p.dt_bias ? p.dt_bias[h] : 0.f);
  const float cb = p.cb[(int64_t)g * p.tokens + row];
  double v = 0., own = 0., ct = 0., cs = 0., xd = 0.;
  for (int s = 0; s < nsl; ++s) {
    const int64_t at = ((int64_t)h * nsl + s) * p.tokens + row;
    v += p.rt[at];
    own += p.rt2[at];  // of D_t ct_t the chunk's own pairs, and the rest
    cs += p.ct2[at];
    ct += p.ct[at];
    xd += p.xd[at];
  }
  // <h, dh> at the chunk's end, and at its start (the end of the chunk before; h = 0 before the first)
  double carry = 0., start = 0.;
  for (int s = 0; s < nsl; ++s) {
    carry += p.anchor[(chunk * p.H + h) * nsl + s];
    if (nc.y > 0) start += p.anchor[((chunk - 1) * p.H + h) * nsl + s];
  }
  const float d = p.softplus ? scan_softplus(raw) : raw;
  const bool cut = in && d * A < LN_EPS;
  if (!cut) v -= own + d * cs;
  if (!in) v = 0.;
  const double miss = __any(cut) || (nc.y == 0 && p.has_h0) ? 0. : (start - carry - wave_sum_d(v)) / len;
  double suf = v + (in ? miss : 0.);
  int ended = cut;  // a cut at or behind this token, within the chunk
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_down(suf, o, 64);
    const int f = __shfl_down(ended, o, 64);
    if (l + o < 64 && !ended) {
      suf += y;
      ended = f;
    }
  }
  const double da = ended ? suf : carry + suf;
  double dd = ct + cb * xd + A * da;
  if (p.softplus) dd *= 1.f / (1.f + expf(-raw));
  if (in) {
    if (p.dt_f32) static_cast<float*>(p.ddt)[row * p.H + h] = (float)dd;
    else static_cast<bf16*>(p.ddt)[row * p.H + h] = to_e<bf16>((float)dd);
  }
  const double sA = wave_sum_d(in ? d * da : 0.), sD = wave_sum_d(in ? xd : 0.), sb = wave_sum_d(in ? dd : 0.);
  if (l == 0) {
    double* o = p.part + (chunk * p.H + h) * 3;
    o[0] = sA;
    o[1] = sD;
    o[2] = sb;
  }
}
__global__ __launch_bounds__(64) void scan_grad_sum_kernel(ScanGradParams p, int nchunk) {
  const int h = blockIdx.x, l = lane_id();
  if (plan_invalid(p.seq, p.segs)) return;
  double s[3] = {0., 0., 0.};
  for (int j = l; j < nchunk; j += 64)
    for (int i = 0; i < 3; ++i) s[i] += p.part[((int64_t)j * p.H + h) * 3 + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    for (int i = 0; i < 3; ++i) s[i] += __shfl_xor(s[i], o, 64);
  if (l == 0) {
    p.dA[h] = (float)s[0];
    if (p.dD) p.dD[h] = (float)s[1];
    if (p.ddt_bias) p.ddt_bias[h] = (float)s[2];
  }
}

// dB or dC from the parts: four columns a thread.  Bound: the parts, read once
// (eight of 16,384 x 128: 67 MB in 12 us, 5.8 TB/s).
template <class E>
__global__ __launch_bounds__(256) void scan_reduce_kernel(ScanReduceParams p) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  const int q = p.Dk / 4;
  const int64_t row = i / (q * p.G);
  if (row >= p.tokens || plan_invalid(p.seq, p.segs)) return;
  const int rem = (int)(i - row * q * p.G), g = rem / q, c = (rem % q) * 4;
  f32x4 s = zero4();
  for (int v = 0; v < p.ppg; ++v)
    s += *reinterpret_cast<const f32x4*>(p.part + (((int64_t)g * p.ppg + v) * p.tokens + row) * p.Dk + c);
  st4f<E>(static_cast<E*>(p.out) + (row * p.G + g) * p.Dk + c, s);
}

// Single-token step: a workgroup owns 32 columns of one (sequence, head) state,
// its 256 threads 4 columns x Dk/32 rows each, as the delta rule's step does.
// Bound: the fp32 state, read and written once, non-temporal (64 sequences of 16
// heads of 128 x 128: 135 MB in 26 us, 5.2 TB/s).
constexpr int STEP_COLS = 32;
template <class E, int DK>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepParams p) {
  const int DV = p.Dv;
  constexpr int RPT = DK / 32;
  __shared__ float red[32][STEP_COLS + 1];
  const int tid = threadIdx.x, tc = tid & 7, tr = tid >> 3;
  const int nh = blockIdx.x, n = nh / p.H, h = nh - n * p.H, g = h / (p.H / p.G);
  const int slot = p.state_idx ? p.state_idx[n] : n;
  if (slot < 0 || slot >= p.num_slots) return;  // padding entry
  const int c0 = blockIdx.y * STEP_COLS + 4 * tc;
  float* hs = p.state + ((int64_t)slot * p.H + h) * DK * DV;
  f32x4 hv[RPT];
  float bv[RPT], cv[RPT];
#pragma unroll
  for (int m = 0; m < RPT; ++m) {
    const int i = tr + 32 * m;
    hv[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(hs + (int64_t)i * DV + c0));
    bv[m] = ldE<E>(p.b, n * p.b_stride + (int64_t)g * DK + i);
    cv[m] = ldE<E>(p.c, n * p.c_stride + (int64_t)g * DK + i);
  }
  const float d = scan_step_size(p, n, h), a = expf(d * p.A[h]);
  const f32x4 x4 = ld4f<E>(static_cast<const E*>(p.x) + n * p.x_stride + (int64_t)h * DV + c0);
  const f32x4 dx = x4 * d;
  f32x4 part = zero4();
#pragma unroll
  for (int m = 0; m < RPT; ++m) {
    const int i = tr + 32 * m;
    const f32x4 hn = hv[m] * a + dx * bv[m];
    __builtin_nontemporal_store(hn, reinterpret_cast<f32x4*>(hs + (int64_t)i * DV + c0));
    part += hn * cv[m];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[tr][4 * tc + e] = part[e];
  __syncthreads();
  if (tid < STEP_COLS) {
    float s = 0.f;
#pragma unroll 8
    for (int r = 0; r < 32; ++r) s += red[r][tid];
    const int j = blockIdx.y * STEP_COLS + tid;
    if (p.D) s += p.D[h] * ldE<E>(p.x, n * p.x_stride + (int64_t)h * DV + j);
    static_cast<E*>(p.y)[(int64_t)nh * DV + j] = to_e<E>(s);
  }
}

template <class E>
hipError_t step_any(int Dk, const ScanStepParams& p, hipStream_t st) {
  const dim3 g(p.N * p.H, p.Dv / STEP_COLS), b(256);
  if (Dk == 128) hipLaunchKernelGGL((scan_step_kernel<E, 128>), g, b, 0, st, p);
  else if (Dk == 64) hipLaunchKernelGGL((scan_step_kernel<E, 64>), g, b, 0, st, p);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_join(const ScanJoinParams& p, hipStream_t st) {
  hipLaunchKernelGGL(scan_join_kernel, dim3(p.Dk * p.Dv / 1024, p.H, p.N), dim3(256), 0, st, p);
  return hipGetLastError();
}
hipError_t launch_scan_grad(const ScanGradParams& p, int nchunk, hipStream_t st) {
  if (nchunk > 0) {
    hipLaunchKernelGGL(scan_grad_kernel, dim3(nchunk, p.H), dim3(64), 0, st, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(scan_grad_sum_kernel, dim3(p.H), dim3(64), 0, st, p, nchunk);
  return hipGetLastError();
}
hipError_t launch_scan_reduce(int dtype, const ScanReduceParams& p, hipStream_t st) {
  const int64_t n = p.tokens * p.G * (p.Dk / 4);
  if (n == 0) return hipSuccess;
  if (dtype == GDN_BF16) hipLaunchKernelGGL((scan_reduce_kernel<bf16>), dim3((n + 255) / 256), dim3(256), 0, st, p);
  else hipLaunchKernelGGL((scan_reduce_kernel<float>), dim3((n + 255) / 256), dim3(256), 0, st, p);
  return hipGetLastError();
}
hipError_t launch_scan_step(int dtype, int Dk, const ScanStepParams& p, hipStream_t st) {
  if (p.N * p.H == 0) return hipSuccess;
  return dtype == GDN_BF16 ? step_any<bf16>(Dk, p, st) : step_any<float>(Dk, p, st);
}

}  // namespace gdn
