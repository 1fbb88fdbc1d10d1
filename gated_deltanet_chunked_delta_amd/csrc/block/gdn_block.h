// gdn_block.h -- parameter blocks and launchers of a block's operators: residual
// norm, rows in 8 bits, projections, gated linear recurrence (not part of the ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_device.h"
#include "gdn_internal.h"
#include "layer/gdn_layer.h"

namespace gdn {

// ---------------------------------------------------------------- rows of any width
// Vectors aligned to an element only: rows of odd widths and slices start anywhere.
// The memory takes such accesses (a line more for some of them), so one path of full
// width serves every width, with single elements at a row's end alone.
typedef bf16x8 bf16x8_any __attribute__((aligned(2)));
typedef bf16x4 bf16x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <int V> __device__ __forceinline__ void ld_full(const bf16* p, float (&f)[V]) {
  if constexpr (V == 8) {
    const bf16x8 v = *reinterpret_cast<const bf16x8_any*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
  } else {
    const bf16x4 v = *reinterpret_cast<const bf16x4_any*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)v[i];
  }
}
template <int V> __device__ __forceinline__ void ld_full(const float* p, float (&f)[V]) {
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    const f32x4 v = reinterpret_cast<const f32x4_any*>(p)[j];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * j + i] = v[i];
  }
}
// V elements at p of which n belong to the row (the rest: 0).
template <int V, class E>
__device__ __forceinline__ void ld_part(const E* p, int n, float (&f)[V]) {
  if (n >= V) {
    ld_full<V>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
  }
}
// Stored past the L2, as outputs that stream through memory (norm forward of 16,384 x
// 2,304 on an fp32 stream: 76 us, 90 with ordinary stores; of 2,303 channels, whose lines are
// shared, 77 and 100).
template <int V, class E>
__device__ __forceinline__ void st_part(E* p, int n, const float (&f)[V]) {
  if (n >= V) {
    if constexpr (sizeof(E) == 2) {
      if constexpr (V == 8)
        __builtin_nontemporal_store(VecIO<bf16, 8>::pack(f), reinterpret_cast<bf16x8_any*>(p));
      else
        __builtin_nontemporal_store(VecIO<bf16, 4>::pack(f), reinterpret_cast<bf16x4_any*>(p));
    } else {
#pragma unroll
      for (int j = 0; j < V / 4; ++j)
        __builtin_nontemporal_store(f32x4{f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]},
                                    reinterpret_cast<f32x4_any*>(p) + j);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = to_e<E>(f[i]);
  }
}

// A launch has fewer than 2^32 threads in x: more workgroups go on in y.
inline dim3 blocks_2d(int64_t n) {
  constexpr int64_t most = 1 << 22;
  return n <= most ? dim3((uint32_t)n) : dim3((uint32_t)most, (uint32_t)((n + most - 1) / most));
}
__device__ __forceinline__ int64_t block_2d() { return blockIdx.y * (int64_t)gridDim.x + blockIdx.x; }

// ---------------------------------------------------------------- residual norm, rows in 8 bits
struct AddNormParams {
  const void* x;             // [R][D], x_stride elements between rows
  int64_t x_stride;
  const void* r;             // nullable, r_stride
  int64_t r_stride;
  const void* w;             // [D]
  void* s;                   // [R][D], with r
  void* y;                   // nullable [R][D]
  uint8_t* q;                // nullable [R][D]
  float* q_scale;            // [R]
  int64_t R;
  int D;
  float eps;
  // backward
  const void* dy;
  const void* ds;            // nullable
  void* dx;                  // nullable
  void* dr;                  // nullable
  void* dw;                  // nullable
  float* part;               // [blocks][D]
  int blocks;
};
// A thread sums at most these many rows' terms of the weight's gradient in fp32; the sums of a
// workgroup's threads of one column (2 to 16 with short rows) are added in fp32 too, the
// workgroups' in 64 bits.
constexpr int ADDNORM_ROWS = 64;
// Workgroups (rows of parts) of the gradient.
int addnorm_blocks(int64_t R, int D, int esize, int cus);
hipError_t launch_addnorm_fwd(int dtype, int res_dtype, const AddNormParams& p, hipStream_t st);
hipError_t launch_addnorm_bwd(int dtype, int res_dtype, const AddNormParams& p, hipStream_t st);
hipError_t launch_quant_rows(int dtype, const AddNormParams& p, hipStream_t st);

// ---------------------------------------------------------------- gated linear recurrence
struct RecParams {
  const void* x;             // [tokens][D], *_stride elements between tokens
  const void* g;
  const void* i;             // nullable
  int64_t x_stride, g_stride, i_stride;
  int g_f32;
  const float* scale;        // nullable [D]
  const float* h0;           // nullable [N][D]
  const int32_t* cu;         // nullable [N+1]
  int T, D, N, tokens;
  int nchunk;                // chunks of REC_W REC_FS tokens (backward: REC_W REC_BS)
  uint64_t* words;           // rec_words(nchunk, D): counters, the chunks' pairs, the groups' ends; null for one chunk
  float* enter;              // [ceil(tokens / REC_STATE)][D]: the state before every REC_STATE tokens; nullable forwards
  // forward
  void* y;                   // nullable
  float* hT;                 // nullable [N][D]
  // backward
  const void* dy;
  const float* dhT;          // nullable
  void* dx;
  void* dg;
  void* di;                  // nullable
  float* dh0;                // nullable
  float* part;               // nullable [nchunk][D]: dscale's parts
};
struct RecStepParams {
  const void* x;
  const void* g;
  const void* i;
  int64_t x_stride, g_stride, i_stride;
  int g_f32;
  const float* scale;
  float* state;
  const int32_t* state_idx;
  int num_slots, N, D;
  void* y;
};
constexpr int REC_W = 8;                    // waves of a chunk
constexpr int REC_BYTES = 4;               // of a token's row that a thread takes
constexpr int REC_FS = 16, REC_BS = 8;      // tokens that a thread holds, forwards and backwards
constexpr int REC_STATE = REC_W * REC_BS;   // tokens between saved states: one a chunk backwards
static_assert(REC_STATE % REC_FS == 0 && REC_W * REC_FS % REC_STATE == 0, "a wave's first token is before a saved state or not");
int64_t rec_words(int nchunk, int D);
hipError_t launch_rec_fwd(int dtype, const RecParams& p, hipStream_t st);
hipError_t launch_rec_bwd(int dtype, const RecParams& p, hipStream_t st);
hipError_t launch_rec_step(int dtype, const RecStepParams& p, hipStream_t st);

// ---------------------------------------------------------------- products
// What a product's sums go through on their way out: v = sum (x_scale[m] w_scale[n]) +
// bias[n], out = act(v) + r.
struct Epilogue {
  const float* x_scale;      // nullable [M]
  const float* w_scale;      // nullable [N]
  const void* bias;          // nullable [N]
  const void* r;             // nullable [M][N], r_stride
  int64_t r_stride;
  int act;
  void* out;                 // [M][N]
  float* v_save;             // nullable [M][N]
};
// out[m][n] = sum over k of a[m][k] b[n][k]: both operands' rows contiguous along k, in
// 16-byte units (pointers, strides; zeros fill the last unit of a row).
struct GemmParams {
  const void* a;
  const void* b;
  int64_t lda, ldb;          // bytes between rows
  int64_t M;
  int N, kbytes;             // bytes of a row that take part
  int splits, steps;         // the sum over k in `splits` parts of `steps` steps of 128 bytes
  float* part;               // [splits][M][N], with splits > 1
  Epilogue e;
};
// How a product is divided: tiles of 256 x 256 or 128 x 128, splits along k.
struct GemmPlan { int tile, splits, steps; };
GemmPlan gemm_plan(int64_t M, int N, int64_t kbytes, int esize, int cus);
inline size_t gemm_part_bytes(const GemmPlan& g, int64_t M, int N) { return g.splits > 1 ? 4ull * g.splits * M * N : 0; }
hipError_t launch_gemm(int dtype, int out_dtype, const GemmParams& p, const GemmPlan& g, hipStream_t st);
// Few rows: a workgroup to 16 outputs (32 from 17 rows on), its waves along k.  Any strides and
// alignment.
constexpr int SKINNY_M = 64;
struct SkinnyParams {
  const void* x;
  const void* w;
  int64_t x_stride, w_stride;  // bytes
  int M, N, kbytes;
  Epilogue e;
};
hipError_t launch_skinny(int dtype, int out_dtype, const SkinnyParams& p, hipStream_t st);
// Rows re-laid for a product: in [R][C] (times act'(v) where v is given) to `rows`
// [R][ldo] and turned to `cols` [C][ldt], zeros behind the ends; sums[row / 64][C].
struct PackParams {
  const void* in;
  int64_t ld;                // elements
  int64_t R;
  int C;
  const float* v;            // nullable [R][C]
  int act;
  void* rows;                // nullable
  int64_t ldo;
  void* cols;                // nullable
  int64_t ldt;
  float* sums;               // nullable
};
// Several of them in one launch (8-bit rows: one).
struct PackJobs {
  PackParams job[3];
  int n = 0;
  __host__ __device__ int64_t blocks(int i) const { return (job[i].R + 63) / 64 * ((job[i].C + 63) / 64); }
};
hipError_t launch_pack(int dtype, const PackJobs& jobs, hipStream_t st);

// ---------------------------------------------------------------- sums of parts
// out[c] = sum over rows of part[row][c], in 64 bits and a fixed order, rounded once.
hipError_t launch_join_parts(int dtype, const float* part, int64_t rows, int64_t cols, void* out, hipStream_t st);

}  // namespace gdn
