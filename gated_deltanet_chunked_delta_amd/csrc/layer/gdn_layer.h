// gdn_layer.h -- parameter blocks and launchers of the operators around the
// recurrence: short causal convolution, selective state space scan, gated
// group norm (not part of the ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

// ---------------------------------------------------------------- vectors of V elements
template <class E, int V> struct VecIO;
template <class E> struct VecIO<E, 1> {
  typedef E raw;
  static __device__ __forceinline__ raw load(const E* p) { return *p; }
  static __device__ __forceinline__ raw zero() { return to_e<E>(0.f); }
  static __device__ __forceinline__ void get(raw r, float (&f)[1]) { f[0] = to_f(r); }
  static __device__ __forceinline__ raw pack(const float (&f)[1]) { return to_e<E>(f[0]); }
};
template <> struct VecIO<bf16, 8> {
  typedef bf16x8 raw;
  static __device__ __forceinline__ raw load(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }
  static __device__ __forceinline__ raw zero() { return raw{}; }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)r[i];
  }
  static __device__ __forceinline__ raw pack(const float (&f)[8]) {
    return bf16x8{(bf16)f[0], (bf16)f[1], (bf16)f[2], (bf16)f[3], (bf16)f[4], (bf16)f[5], (bf16)f[6], (bf16)f[7]};
  }
};
template <> struct VecIO<bf16, 4> {
  typedef bf16x4 raw;
  static __device__ __forceinline__ raw load(const bf16* p) { return *reinterpret_cast<const bf16x4*>(p); }
  static __device__ __forceinline__ raw zero() { return raw{}; }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)r[i];
  }
  static __device__ __forceinline__ raw pack(const float (&f)[4]) {
    return bf16x4{(bf16)f[0], (bf16)f[1], (bf16)f[2], (bf16)f[3]};
  }
};
template <> struct VecIO<float, 4> {
  typedef f32x4 raw;
  static __device__ __forceinline__ raw load(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
  static __device__ __forceinline__ raw zero() { return zero4(); }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = r[i];
  }
  static __device__ __forceinline__ raw pack(const float (&f)[4]) { return f32x4{f[0], f[1], f[2], f[3]}; }
};
template <class E, int V>
__device__ __forceinline__ void store_vec(E* p, const float (&f)[V]) {
  *reinterpret_cast<typename VecIO<E, V>::raw*>(p) = VecIO<E, V>::pack(f);
}
// A store past the L2, for outputs that stream through memory and are not read
// again by the kernel: the inputs' lines, which neighbouring workgroups do read
// again, stay (norm of 32,768 x 16 x 128: 81 -> 70 us; convolution gradient of
// 49,828 x 2,304: 180 -> 173 us).  The convolution's forward pass keeps ordinary
// stores: 92 us against 105 there.
template <class E, int V>
__device__ __forceinline__ void stream_vec(E* p, const float (&f)[V]) {
  typedef typename VecIO<E, V>::raw raw;
  __builtin_nontemporal_store(VecIO<E, V>::pack(f), reinterpret_cast<raw*>(p));
}
// Elements of one 16-byte access.
template <class E> constexpr int kVec = 16 / (int)sizeof(E);

// sigmoid(x) and the SiLU gate with the hardware's exponential and reciprocal,
// each within a unit in the last place: the exact division of sigmoid_f takes ten
// instructions, a third of what these memory-bound kernels spend on an element.
// exp overflow gives 1 / inf = 0.  The exponent -x log2(e) rounded to fp32 alone is
// off by |x| 2^-24, which is far below a bf16 result's step.  For fp32 tensors
// what 2^h misses exp(-x) by enters as a first-order factor, 1 + (-x - h ln 2) with ln 2
// in two parts: silu within 4 fp32 roundings (2^-24) of its value for x in -80 .. 80,
// 62 without it.  (x held to +-88 there, where the gate is 0 or 1; a NaN comes back in
// through the products with x itself.)
template <class E>
__device__ __forceinline__ float fast_sigmoid(float x) {
  if constexpr (sizeof(E) == 4) {
    const float c = __builtin_amdgcn_fmed3f(x, -88.f, 88.f), h = -1.44269504f * c;
    const float e = __builtin_amdgcn_exp2f(h);
    const float miss = fmaf(h, 1.90465430e-9f, fmaf(h, -0.69314718f, -c));
    return __builtin_amdgcn_rcpf(1.f + fmaf(e, miss, e));
  }
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}
template <class E>
__device__ __forceinline__ float silu_gate(float x) { return x * fast_sigmoid<E>(x); }
// its derivative, from x and sigmoid(x)
__device__ __forceinline__ float dsilu_gate(float x, float s) { return s + x * (s - s * s); }

// ---------------------------------------------------------------- short causal convolution
struct ConvParams {
  const void* x;             // [tokens][D], x_stride elements between tokens
  int64_t x_stride;
  const void* w;             // [D][W]
  const void* bias;          // nullable [D]
  const void* init;          // nullable [N][W-1][D]
  const int32_t* cu;         // nullable [N+1]
  int B, T, D, N, silu;
  int64_t tokens;            // B * T
  int run;                   // tokens per thread
  int64_t nruns;
  // forward
  void* y;                   // [tokens][D]
  void* fin;                 // nullable [N][W-1][D]
  // backward
  const void* dy;            // [tokens][D]
  const void* dfin;          // nullable [N][W-1][D]
  void* dx;                  // [tokens][D]
  void* dw;                  // [D][W]
  void* dbias;               // nullable [D]
  void* dinit;               // nullable [N][W-1][D]
  float* part;               // [nruns][W+1][D] partial sums of dw and dbias
};
struct ConvStepParams {
  const void* x;             // [N][D]
  int64_t x_stride;
  void* state;               // [slots][W-1][D], shifted in place
  const int32_t* state_idx;
  int num_slots;
  const void* w;
  const void* bias;
  void* y;
  int N, D, silu;
};
// vec: 16-byte accesses are possible (D, strides and pointers allow them)
hipError_t launch_conv_fwd(int dtype, int W, bool vec, const ConvParams& p, hipStream_t st);
hipError_t launch_conv_bwd(int dtype, int W, bool vec, const ConvParams& p, hipStream_t st);
hipError_t launch_conv_dw(int dtype, int W, const ConvParams& p, hipStream_t st);
hipError_t launch_conv_step(int dtype, int W, bool vec, const ConvStepParams& p, hipStream_t st);

// ---------------------------------------------------------------- gated group norm
struct NormParams {
  const void* x;             // [R][G][D], x_stride elements between tokens
  int64_t x_stride;
  const void* z;             // nullable gate, z_stride
  int64_t z_stride;
  const void* w;             // [G][D], or [D] with shared
  const void* bias;          // nullable, like w
  int64_t R;
  int G, D, shared, center, gate_first;
  float eps;
  void* y;                   // [R][G][D]
  const void* dy;            // [R][G][D]
  void* dx;
  void* dz;                  // nullable (no gate)
  void* dw;
  void* dbias;               // nullable
  float* part;               // [weight groups][blocks][1 or 2][D]
  int blocks;                // workgroups per weight group (backward); the launcher may take more
};
constexpr int NORM_ROWS = 64;  // rows whose weight gradients one fp32 sum takes, at most
hipError_t launch_norm_fwd(int dtype, bool vec, const NormParams& p, hipStream_t st);
hipError_t launch_norm_bwd(int dtype, bool vec, const NormParams& p, hipStream_t st);

// ---------------------------------------------------------------- selective state space scan
constexpr int PS = 64;       // value columns of one slice: a head of Dv columns is Dv / PS slices

// One sweep over the tokens of every segment, forwards or backwards in time,
// with a Dk x PS slice of the state per (segment, head, slice):
//   state <- decay * state + sw_t K_t V_t^T
//   out1_t = tw_t (state^T Q_t) + D_h V_t          (a value row)
//   out2_t = tw_t (state W_t)                      (a key row, one part per slice)
//   rt_t   = Q_t . (state before token t) W_t      (the decay gradient's row term)
// Forwards in time K = B, Q = C, V = x, W = dy, sw = step, tw = 1: out1 = y,
// out2 = dC.  Backwards K = C, Q = B, V = dy, W = x, sw = 1, tw = step:
// out1 = dx, out2 = dB.
struct SweepParams {
  const void* q;             // [tokens][G][Dk]
  const void* k;
  int64_t q_stride, k_stride;
  const void* v;             // [tokens][H][Dv]
  const void* w;
  int64_t v_stride, w_stride;
  const void* dt;            // [tokens][H]
  int64_t dt_stride;
  int dt_f32, softplus;
  const float* dt_bias;      // nullable [H]
  const float* A;            // [H]
  const float* D;            // nullable [H]
  int H, G, Dk, Dv;
  int64_t tokens;
  SeqInfo seq;
  const SegDesc* segs;
  const int* seg_first;
  const float* s_in;         // nullable: state entering each segment (by segment when per_seg, else by sequence)
  int per_seg;
  float* s_end;              // nullable: state leaving the last segment of each sequence in sweep order [N][H][Dk][Dv]
  float* s_loc;              // sweeps without output: each segment's own end state [nseg][H][Dk][Dv]
  float* s_dec;              // and its total decay [nseg][H]
  int round_once;            // bf16 out1: the chunk matrix and the state in two parts
  void* out1;                // [tokens][H][Dv]
  float* out2;               // [G * parts][tokens][Dk], where a group has more than one part
  void* out2_whole;          // [tokens][G][Dk], where it has one
  float* rt;                 // [H * Dv / PS][tokens]
  float* rt2;                // the same: of the chunk's own pairs, by source token (forwards); rt's part from the state (backwards)
  float* xd;                 // nullable [H * Dv / PS][tokens]: x_t . dy_t over the slice
  float* cb;                 // nullable [G][tokens]: C_t . B_t
  // anchors of the decay gradient: the forward key sweep leaves its state at the
  // end of every chunk, the backward one writes <it, its gradient>
  const int* chunk_first;    // first chunk of each sequence
  float* dump;               // [chunks][H * Dv / PS][Dk * PS] in the key sweep's own order
  double* anchor;            // [chunks][H * Dv / PS]
};

struct ScanJoinParams {      // end states of the segments -> states entering them
  float* s_loc;
  const float* s_dec;
  const float* s0;           // nullable [N][H][Dk][Dv]
  int H, Dk, Dv, rev;
  SeqInfo seq;
  const SegDesc* segs;
  const int* seg_first;
  int N;
};

struct ScanGradParams {      // ddt, dA, dD, ddt_bias from the row terms
  const void* dt;
  int64_t dt_stride;
  int dt_f32, softplus;
  const float* dt_bias;
  const float* A;
  int H, G, Dk, Dv;
  int64_t tokens;
  SeqInfo seq;
  const SegDesc* segs;
  const float* rt;           // forward sweep's row terms [slices][tokens]
  const float* rt2;
  const float* ct;           // backward sweep's
  const float* ct2;
  const float* xd;
  const float* cb;
  const int2* chunk_tab;
  const double* anchor;      // [chunks][H * Dv / PS]
  int has_h0;
  void* ddt;                 // [tokens][H], dtype of dt
  double* part;              // [chunks][H][3]
  float* dA;
  float* dD;                 // nullable
  float* ddt_bias;           // nullable
};

struct ScanReduceParams {    // parts of dB or dC -> sums over a group's slices
  const float* part;         // [G * parts per group][tokens][Dk]
  void* out;                 // [tokens][G][Dk]
  int G, ppg, Dk;
  int64_t tokens;
  SeqInfo seq;
  const SegDesc* segs;
};

struct ScanStepParams {
  const void* x;             // [N][H][Dv]
  const void* dt;            // [N][H]
  const void* b;             // [N][G][Dk]
  const void* c;
  int64_t x_stride, dt_stride, b_stride, c_stride;
  const float* A;
  const float* D;
  const float* dt_bias;
  int dt_f32, softplus;
  float* state;              // [slots][H][Dk][Dv]
  const int32_t* state_idx;
  int num_slots;
  void* y;                   // [N][H][Dv]
  int N, H, G, Dv;
};

// Outputs of a sweep.
enum { SWEEP_STATE = 0, SWEEP_VALUE = 1, SWEEP_KEY = 2 };
hipError_t launch_sweep(int dtype, int rev, int mode, const SweepParams& p, int nseg, hipStream_t st);
hipError_t launch_scan_join(const ScanJoinParams& p, hipStream_t st);
hipError_t launch_scan_grad(const ScanGradParams& p, int nchunk, hipStream_t st);
hipError_t launch_scan_reduce(int dtype, const ScanReduceParams& p, hipStream_t st);
hipError_t launch_scan_step(int dtype, int Dk, const ScanStepParams& p, hipStream_t st);
// Parts of out2 per group of heads that a key sweep writes.
int sweep_parts_per_group(int dtype, int H, int G, int Dv);
// Workgroups of a sweep per segment.
int sweep_workgroups(int dtype, int H, int G, int Dv);

// Step size and log decay of one token and head.
__device__ __forceinline__ float scan_dt_raw(const void* dt, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(dt)[i] : to_f(static_cast<const bf16*>(dt)[i]);
}
// softplus as max(x, 0) + log1p(exp(-|x|)); the accurate exp and log: a step of
// 1e-3 keeps its relative precision, and it is formed once per token and head.
__device__ __forceinline__ float scan_softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }
template <class P>
__device__ __forceinline__ float scan_step_size(const P& p, int64_t row, int h) {
  const float raw = scan_dt_raw(p.dt, p.dt_f32, row * p.dt_stride + h) + (p.dt_bias ? p.dt_bias[h] : 0.f);
  return p.softplus ? scan_softplus(raw) : raw;
}

}  // namespace gdn
