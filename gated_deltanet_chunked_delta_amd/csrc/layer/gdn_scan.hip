// gdn_scan.hip -- selective state space scan on the vector unit: the token by
// token sweeps (fp32 inputs), the joins between segments, the gradients of the
// step sizes and decays, and the single-token step.
//
// Per sequence and head, with step D_t, decay a_t = D_t A (A <= 0):
//   h_t = exp(a_t) h_{t-1} + D_t B_t x_t^T     (Dk x Dv),      y_t = h_t^T C_t + D x_t
// and backwards in time, for the gradient dh of the states,
//   dh_t = exp(a_{t+1}) dh_{t+1} + C_t dy_t^T
//   dx_t = D_t dh_t^T B_t + D dy_t,   dB_t = D_t dh_t x_t,   dC_t = h_t dy_t
// (dB, dC summed over the heads that share them).  Both directions are one
// sweep, SweepParams, with the roles of B, C, x and dy exchanged.
//
// Gradient of the decays.  da_t = <dh_t, exp(a_t) h_{t-1}> obeys
//   da_t = da_{t+1} + rt_t - D_t ct_t,
//   rt_t = C_t . (exp(a_t) h_{t-1}) dy_t,   ct_t = B_t . (exp(a_{t+1}) dh_{t+1}) x_t
// (the terms of token t with itself cancel and are left out, so under strong
// decay both sides are as small as da itself), started at every segment's end
// from <h, dh> there.  Then dD_t = ct_t + (C_t . B_t)(x_t . dy_t) + A da_t.
//
// A sequence is cut into segments of chunks (the plan of the C ABI) that run
// side by side: sweeps without output form each segment's own end state, the
// join turns them into the states entering the segments.
#include "gdn_layer.h"

namespace gdn {

namespace {

constexpr int VT = 16;  // tokens staged together

struct SegRange {
  int n, s, ns;     // sequence, segment within it, segments of the sequence
  int64_t row0;     // first token of the segment (global row)
  int len;          // its tokens
};
__device__ __forceinline__ bool seg_range(const SeqInfo& seq, const SegDesc* segs, const int* seg_first, int j,
                                          SegRange& r) {
  const SegDesc d = seq.seg_of(segs, j);
  if (d.n < 0) return false;  // the device cu_seqlens disagrees with the plan: nothing is written
  r.n = d.n;
  r.s = d.s;
  r.ns = seq.nseg_of(seg_first, d.n);
  const int t0 = min(d.c_begin * CH, seq.len(d.n)), t1 = min(d.c_end * CH, seq.len(d.n));
  r.row0 = seq.start(d.n) + t0;
  r.len = t1 - t0;
  return true;
}

// The plan marks every segment when the device cu_seqlens disagrees with the
// host copy that sized the work.
__device__ __forceinline__ bool plan_invalid(const SeqInfo& seq, const SegDesc* segs) {
  return seq.cu && segs[0].n < 0;
}

template <class E> __device__ __forceinline__ float ldE(const void* p, int64_t i) { return to_f(static_cast<const E*>(p)[i]); }

// Value sweep (out1) and state sweep (no output).  256 threads per (segment,
// head, slice): thread column j = tid % 64, its wave one quarter of the state's
// Dk rows, in registers.  The keys of VT tokens are staged in LDS in fp32; a
// wave reads them as broadcasts.
template <class E, int DK, bool REV, bool OUT>
__global__ __launch_bounds__(256) void sweep_value_kernel(SweepParams p) {
  constexpr int NR = DK / 4;
  __shared__ __align__(16) float sk[VT][DK], sq[OUT ? VT : 1][DK];
  __shared__ float sv[VT][PS], red[OUT ? 4 : 1][VT][PS], sdec[VT], ssw[VT], stw[VT];
  const int tid = threadIdx.x, j = tid & 63, rg = tid >> 6;
  const int nsl = p.Dv / PS;
  const int vh = blockIdx.y, h = vh / nsl, sl = vh % nsl, g = h / (p.H / p.G);
  SegRange r;
  if (!seg_range(p.seq, p.segs, p.seg_first, blockIdx.x, r)) return;
  const bool first = REV ? r.s == r.ns - 1 : r.s == 0, last = REV ? r.s == 0 : r.s == r.ns - 1;
  if (!OUT && last) return;  // nothing follows this segment
  const int64_t st_off = (int64_t)DK * p.Dv, col = sl * PS + j;
  float st[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) st[i] = 0.f;
  if (OUT && p.s_in && (p.per_seg || first)) {
    const float* s0 = p.s_in + ((int64_t)(p.per_seg ? (int)blockIdx.x : r.n) * p.H + h) * st_off + col;
#pragma unroll
    for (int i = 0; i < NR; ++i) st[i] = s0[(int64_t)(rg * NR + i) * p.Dv];
  }
  const float A = p.A[h], Dh = p.D ? p.D[h] : 0.f;
  float pend = 1.f, total = 0.f;
  for (int b = 0; b < r.len; b += VT) {
    const int nt = min(VT, r.len - b);
    __syncthreads();
    for (int i = tid; i < nt * DK; i += 256) {
      const int t = i / DK, c = i % DK;
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - t : b + t);
      sk[t][c] = ldE<E>(p.k, row * p.k_stride + (int64_t)g * DK + c);
      if (OUT) sq[t][c] = ldE<E>(p.q, row * p.q_stride + (int64_t)g * DK + c);
    }
    for (int i = tid; i < nt * PS; i += 256) {
      const int t = i / PS, c = i % PS;
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - t : b + t);
      sv[t][c] = ldE<E>(p.v, row * p.v_stride + (int64_t)h * p.Dv + sl * PS + c);
    }
    if (tid < nt) {
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - tid : b + tid);
      const float d = scan_step_size(p, row, h);
      sdec[tid] = d * A;
      ssw[tid] = REV ? 1.f : d;
      stw[tid] = REV ? d : 1.f;
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float a = sdec[t], e = expf(a), f = REV ? pend : e;
      pend = e;
      if (!OUT) total += a;
      const float vw = sv[t][j] * ssw[t];
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        st[i] = f * st[i] + sk[t][rg * NR + i] * vw;
        if (OUT) acc += sq[t][rg * NR + i] * st[i];
      }
      if (OUT) red[rg][t][j] = acc;
    }
    if (OUT) {
      __syncthreads();
      for (int i = tid; i < nt * PS; i += 256) {
        const int t = i / PS, c = i % PS;
        const int64_t row = r.row0 + (REV ? r.len - 1 - b - t : b + t);
        const float o = stw[t] * (red[0][t][c] + red[1][t][c] + red[2][t][c] + red[3][t][c]) + Dh * sv[t][c];
        static_cast<E*>(p.out1)[(row * p.H + h) * p.Dv + sl * PS + c] = to_e<E>(o);
      }
    }
  }
  const float tail = REV ? pend : 1.f;  // backwards, the state before the segment's first token
  float* dst = OUT ? (last ? p.s_end : nullptr) : p.s_loc;
  if (!dst) return;
  dst += ((int64_t)(OUT ? r.n : (int)blockIdx.x) * p.H + h) * st_off + col;
#pragma unroll
  for (int i = 0; i < NR; ++i) dst[(int64_t)(rg * NR + i) * p.Dv] = tail * st[i];
  if (!OUT && tid == 0 && sl == 0) p.s_dec[(int64_t)blockIdx.x * p.H + h] = expf(total);
}

// Key sweep (out2 and the row terms): thread i holds row i of the state's
// slice, PS values in registers, and forms its entry of out2 alone.
template <class E, int DK, bool REV>
__global__ __launch_bounds__(DK) void sweep_key_kernel(SweepParams p) {
  __shared__ __align__(16) float sv[VT][PS], sw[VT][PS];
  __shared__ float sdec[VT], ssw[VT], stw[VT], sxd[VT], red[VT][DK / 64], redc[VT][DK / 64], anch[DK / 64];
  const int tid = threadIdx.x;
  const int nsl = p.Dv / PS;
  const int vh = blockIdx.y, h = vh / nsl, sl = vh % nsl, g = h / (p.H / p.G);
  SegRange r;
  if (!seg_range(p.seq, p.segs, p.seg_first, blockIdx.x, r)) return;
  const bool first = REV ? r.s == r.ns - 1 : r.s == 0;
  const int64_t st_off = (int64_t)DK * p.Dv;
  float st[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) st[i] = 0.f;
  if (p.s_in && (p.per_seg || first)) {
    const float* s0 = p.s_in + ((int64_t)(p.per_seg ? (int)blockIdx.x : r.n) * p.H + h) * st_off + (int64_t)tid * p.Dv + sl * PS;
#pragma unroll
    for (int i = 0; i < PS; ++i) st[i] = s0[i];
  }
  const float A = p.A[h];
  float pend = 1.f;
  const bool cb_mine = p.cb && h % (p.H / p.G) == 0 && sl == 0;
  for (int b = 0; b < r.len; b += VT) {
    const int nt = min(VT, r.len - b);
    __syncthreads();
    for (int i = tid; i < nt * PS; i += DK) {
      const int t = i / PS, c = i % PS;
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - t : b + t);
      sv[t][c] = ldE<E>(p.v, row * p.v_stride + (int64_t)h * p.Dv + sl * PS + c);
      sw[t][c] = ldE<E>(p.w, row * p.w_stride + (int64_t)h * p.Dv + sl * PS + c);
    }
    if (tid < nt) {
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - tid : b + tid);
      const float d = scan_step_size(p, row, h);
      sdec[tid] = expf(d * A);
      ssw[tid] = REV ? 1.f : d;
      stw[tid] = REV ? d : 1.f;
    }
    __syncthreads();
    if (tid < nt) {
      float s = 0.f;
      for (int c = 0; c < PS; ++c) s += sv[tid][c] * sw[tid][c];
      sxd[tid] = s;
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - t : b + t);
      const float kk = ldE<E>(p.k, row * p.k_stride + (int64_t)g * DK + tid);
      const float qq = ldE<E>(p.q, row * p.q_stride + (int64_t)g * DK + tid);
      const float e = sdec[t], f = REV ? pend : e, ks = kk * ssw[t];
      pend = e;
      float pre = 0.f;
#pragma unroll
      for (int i = 0; i < PS; ++i) {
        st[i] *= f;
        pre += st[i] * sw[t][i];
        st[i] += ks * sv[t][i];
      }
      p.out2[((int64_t)vh * p.tokens + row) * DK + tid] = stw[t] * (pre + ks * sxd[t]);
      const float rt = wave_sum(qq * pre);
      if (lane_id() == 0) red[t][wave_id()] = rt;
      if (cb_mine) {
        const float cb = wave_sum(qq * kk);
        if (lane_id() == 0) redc[t][wave_id()] = cb;
      }
    }
    __syncthreads();
    if (tid < nt) {
      const int64_t row = r.row0 + (REV ? r.len - 1 - b - tid : b + tid);
      float s = 0.f, c = 0.f;
#pragma unroll
      for (int w = 0; w < DK / 64; ++w) {
        s += red[tid][w];
        if (cb_mine) c += redc[tid][w];
      }
      p.rt[(int64_t)vh * p.tokens + row] = s;
      if (p.xd) p.xd[(int64_t)vh * p.tokens + row] = sxd[tid];
      if (cb_mine) p.cb[(int64_t)g * p.tokens + row] = c;
    }
  }
  if (p.anchor) {
    float s = 0.f;
    if (p.g_end && (p.g_per_seg || r.s == r.ns - 1)) {
      const float* ge = p.g_end + ((int64_t)(p.g_per_seg ? (int)blockIdx.x : r.n) * p.H + h) * st_off + (int64_t)tid * p.Dv + sl * PS;
#pragma unroll
      for (int i = 0; i < PS; ++i) s += st[i] * ge[i];
    }
    s = wave_sum(s);
    if (lane_id() == 0) anch[wave_id()] = s;
    __syncthreads();
    if (tid == 0) {
      s = 0.f;
      for (int w = 0; w < DK / 64; ++w) s += anch[w];
      p.anchor[(int64_t)blockIdx.x * p.H * nsl + vh] = s;
    }
  }
}

// Per (sequence, head): end states of the segments, each from a zero start,
// become the states entering them (in sweep order).
__global__ __launch_bounds__(256) void scan_join_kernel(ScanJoinParams p) {
  const int n = blockIdx.z, h = blockIdx.y;
  if (plan_invalid(p.seq, p.segs)) return;
  const int64_t ss = (int64_t)p.Dk * p.Dv, e = blockIdx.x * 256 + threadIdx.x;
  const int j0 = p.seq.cu ? p.seg_first[n] : n * p.seq.nseg_per_seq();
  const int ns = p.seq.nseg_of(p.seg_first, n);
  float carry = p.s0 ? p.s0[((int64_t)n * p.H + h) * ss + e] : 0.f;
  for (int i = 0; i < ns; ++i) {
    const int64_t j = j0 + (p.rev ? ns - 1 - i : i);
    float* s = p.s_loc + (j * p.H + h) * ss + e;
    const float loc = i + 1 < ns ? *s : 0.f;
    *s = carry;
    if (i + 1 < ns) carry = p.s_dec[j * p.H + h] * carry + loc;
  }
}

// ddt of every token and the segment's sums for dA, dD and ddt_bias: a wave
// per (segment, head) walks the segment's 64-token pieces backwards.
__global__ __launch_bounds__(64) void scan_grad_kernel(ScanGradParams p) {
  const int j = blockIdx.x, h = blockIdx.y, l = lane_id();
  const int nsl = p.Dv / PS, g = h / (p.H / p.G);
  SegRange r;
  const bool ok = seg_range(p.seq, p.segs, p.seg_first, j, r);
  float sA = 0.f, sD = 0.f, sb = 0.f;
  if (ok) {
    float carry = 0.f;
    if (p.anchor)
      for (int s = 0; s < nsl; ++s) carry += p.anchor[((int64_t)j * p.H + h) * nsl + s];
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    for (int b = (r.len - 1) / 64 * 64; b >= 0 && r.len > 0; b -= 64) {
      const int t = b + l;
      const bool in = t < r.len;
      const int64_t row = r.row0 + min(t, r.len - 1);
      const float raw = scan_dt_raw(p.dt, p.dt_f32, row * p.dt_stride + h) + bias;
      const float d = p.softplus ? scan_softplus(raw) : raw;
      float rt = 0.f, ct = 0.f, xd = 0.f;
      for (int s = 0; s < nsl; ++s) {
        const int64_t o = ((int64_t)h * nsl + s) * p.tokens + row;
        rt += p.rt[o];
        ct += p.ct[o];
        xd += p.xd[o];
      }
      const float diff = in ? rt - d * ct : 0.f;
      // suffix sum over the piece
      float suf = diff;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const float y = __shfl_down(suf, o, 64);
        if (l + o < 64) suf += y;
      }
      const float da = carry + suf;
      carry += __shfl(suf, 0, 64);
      float dd = ct + p.cb[(int64_t)g * p.tokens + row] * xd + A * da;
      if (p.softplus) dd *= sigmoid_f(raw);
      if (in) {
        if (p.dt_f32) static_cast<float*>(p.ddt)[row * p.H + h] = dd;
        else static_cast<bf16*>(p.ddt)[row * p.H + h] = to_e<bf16>(dd);
        sA += d * da;
        sD += xd;
        sb += dd;
      }
    }
  }
  sA = wave_sum(sA);
  sD = wave_sum(sD);
  sb = wave_sum(sb);
  if (l == 0) {
    float* o = p.part + ((int64_t)j * p.H + h) * 3;
    o[0] = sA;
    o[1] = sD;
    o[2] = sb;
  }
}
__global__ __launch_bounds__(64) void scan_grad_sum_kernel(ScanGradParams p, int nseg) {
  const int h = blockIdx.x, l = lane_id();
  if (plan_invalid(p.seq, p.segs)) return;
  double s[3] = {0., 0., 0.};
  for (int j = l; j < nseg; j += 64)
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

// dB or dC from the parts: four columns a thread.
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
// Bound: the fp32 state, read and written once, non-temporal.
constexpr int STEP_COLS = 32;
template <class E, int DK, int DV>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepParams p) {
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

template <class E, int DK, bool REV>
hipError_t sweep_vec(int mode, const SweepParams& p, int nseg, hipStream_t st) {
  const dim3 g(nseg, p.H * (p.Dv / PS));
  if (mode == SWEEP_VALUE) hipLaunchKernelGGL((sweep_value_kernel<E, DK, REV, true>), g, dim3(256), 0, st, p);
  else if (mode == SWEEP_STATE) hipLaunchKernelGGL((sweep_value_kernel<E, DK, REV, false>), g, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((sweep_key_kernel<E, DK, REV>), g, dim3(DK), 0, st, p);
  return hipGetLastError();
}
template <class E>
hipError_t sweep_vec_any(int rev, int mode, const SweepParams& p, int nseg, hipStream_t st) {
  if (p.Dk == 64) return rev ? sweep_vec<E, 64, true>(mode, p, nseg, st) : sweep_vec<E, 64, false>(mode, p, nseg, st);
  if (p.Dk == 128) return rev ? sweep_vec<E, 128, true>(mode, p, nseg, st) : sweep_vec<E, 128, false>(mode, p, nseg, st);
  return hipErrorInvalidValue;
}

template <class E>
hipError_t step_any(int Dk, int Dv, const ScanStepParams& p, hipStream_t st) {
  const dim3 g(p.N * p.H, Dv / STEP_COLS), b(256);
  if (Dk == 128 && Dv == 128) hipLaunchKernelGGL((scan_step_kernel<E, 128, 128>), g, b, 0, st, p);
  else if (Dk == 64 && Dv == 64) hipLaunchKernelGGL((scan_step_kernel<E, 64, 64>), g, b, 0, st, p);
  else if (Dk == 64 && Dv == 128) hipLaunchKernelGGL((scan_step_kernel<E, 64, 128>), g, b, 0, st, p);
  else if (Dk == 128 && Dv == 64) hipLaunchKernelGGL((scan_step_kernel<E, 128, 64>), g, b, 0, st, p);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sweep(int dtype, int rev, int mode, const SweepParams& p, int nseg, hipStream_t st) {
  return dtype == GDN_BF16 ? sweep_vec_any<bf16>(rev, mode, p, nseg, st) : sweep_vec_any<float>(rev, mode, p, nseg, st);
}
int sweep_parts_per_group(int, int H, int G, int Dv) { return H / G * (Dv / PS); }

hipError_t launch_scan_join(const ScanJoinParams& p, hipStream_t st) {
  hipLaunchKernelGGL(scan_join_kernel, dim3(p.Dk * p.Dv / 256, p.H, p.N), dim3(256), 0, st, p);
  return hipGetLastError();
}
hipError_t launch_scan_grad(const ScanGradParams& p, int nseg, hipStream_t st) {
  hipLaunchKernelGGL(scan_grad_kernel, dim3(nseg, p.H), dim3(64), 0, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(scan_grad_sum_kernel, dim3(p.H), dim3(64), 0, st, p, nseg);
  return hipGetLastError();
}
hipError_t launch_scan_reduce(int dtype, const ScanReduceParams& p, hipStream_t st) {
  const int64_t n = p.tokens * p.G * (p.Dk / 4);
  if (n == 0) return hipSuccess;
  if (dtype == GDN_BF16) hipLaunchKernelGGL((scan_reduce_kernel<bf16>), dim3((n + 255) / 256), dim3(256), 0, st, p);
  else hipLaunchKernelGGL((scan_reduce_kernel<float>), dim3((n + 255) / 256), dim3(256), 0, st, p);
  return hipGetLastError();
}
hipError_t launch_scan_step(int dtype, int Dk, int Dv, const ScanStepParams& p, hipStream_t st) {
  if (p.N * p.H == 0) return hipSuccess;
  return dtype == GDN_BF16 ? step_any<bf16>(Dk, Dv, p, st) : step_any<float>(Dk, Dv, p, st);
}

}  // namespace gdn
