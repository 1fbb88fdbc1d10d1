// gdn_linear.hip -- products with an epilogue: out = act(a b^T scales + bias) + r.
//
// Both operands' rows run along k.  A step of the main loop takes 128 bytes of every
// row of a tile -- 64 bf16, 32 fp32 or 128 8-bit values -- so one layout serves all types:
// a row's 128 bytes are eight pieces of 16, a lane's operand for one 16-row block is two of
// them.  Which k a piece stands for is the same for both operands, which is all that the
// sum asks for.
//
// The tiles are loaded straight into LDS (buffer loads with the lds bit), two buffers deep,
// one step ahead.  Such a load puts 64 lanes' pieces side by side, so the layout is made by
// which piece a lane asks for: piece j of row r lies in slot j ^ s(r), with s such that the
// 16 rows that a fragment read takes at once fall on all 64 banks.
//
// The products are formed turned (b's rows are the matrix core's rows), and the four 16-row
// blocks of a wave's 64 outputs take rows 32 (j / 2) + 8 q + 4 (j % 2) + i of b for block j: a
// lane (of group q) then holds twice eight outputs side by side, and a store of 16 bytes a
// lane fills 64 of a row by its four lanes (16 side by side, whose stores lie 32 bytes
// apart: 8 bits 413 us instead of 403, SiLU with v kept 470 instead of 435).
//
// Bound: the matrix cores, and between a tile's main loops its epilogue, which nothing
// hides (two buffers of a 256 x 256 tile take 128 of 160 KB of LDS: one workgroup a
// compute unit).  Measured: bf16 8,192^3 806-833 us (1,365-1,320 TFLOP/s; the library's
// product 1,267 on such a card); 16,384 x 2,048 -> 6,144 with SiLU 355-399 (1,160-1,030; the
// library without it 349), 432-449 with v kept in fp32 as well (402 MB more), its dx 324-339, its
// dw 391-410.  8 bits: 32,768 x 2,048 -> 6,144 382-412 us (2,160-2,000 TFLOP/s; the library 395),
// to fp32 (bf16 products) 658-670.  fp32 4,096^3 967-987 us (142-139 of the 157 TFLOP/s of its
// matrix instructions; the library 153).  Sums stay in the matrix cores' fp32: those of 2^20 like
// terms come out within 2e-6 (rms), of few rows within 7e-6.  No better: other groups of tile rows (4: 347 instead of 331
// in dx, 16: 869 in 8,192^3), a raised priority around the products, the next fragment requested
// by hand, requests between the products, non-temporal stores (481 instead of 413), a persistent
// workgroup that requests its next tile's first step with this one's last (its registers spill:
// 869 in 8,192^3).
#include <utility>

#include "gdn_block.h"

namespace gdn {

namespace {

typedef uint32_t u32x4 __attribute__((__vector_size__(16)));
typedef int i32x8 __attribute__((__vector_size__(32)));

template <int T> struct ElemOf;
template <> struct ElemOf<GDN_F32> { typedef float type; };
template <> struct ElemOf<GDN_BF16> { typedef bf16 type; };

// One lane's two pieces of a row, and the product of two 16-row blocks over one step.
struct Pieces { u32x4 lo, hi; };
// Sixteen 8-bit values as bf16, which holds each of them.
__device__ __forceinline__ void widen(u32x4 v, bf16x8& lo, bf16x8& hi) {
  typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 pair;
  pair t[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t[2 * j] = __builtin_bit_cast(pair, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j], 1.f, false));
    t[2 * j + 1] = __builtin_bit_cast(pair, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j], 1.f, true));
  }
  lo = bf16x8{t[0][0], t[0][1], t[1][0], t[1][1], t[2][0], t[2][1], t[3][0], t[3][1]};
  hi = bf16x8{t[4][0], t[4][1], t[5][0], t[5][1], t[6][0], t[6][1], t[7][0], t[7][1]};
}
// EXACT (8-bit rows with fp32 outputs): the 8-bit matrix instructions' sums carry about 17
// bits (measured 1.3e-5 of the result against 64 bits, of either instruction), enough for a
// bf16 result and not for an fp32 one; there the values are widened to bf16.
template <int T, bool EXACT = false>
__device__ __forceinline__ void mma_step(f32x4& acc, const Pieces& a, const Pieces& b) {
  if constexpr (T == GDN_BF16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.lo), __builtin_bit_cast(bf16x8, b.lo), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.hi), __builtin_bit_cast(bf16x8, b.hi), acc, 0, 0, 0);
  } else if constexpr (T == GDN_F32) {
    const f32x4 al = __builtin_bit_cast(f32x4, a.lo), bl = __builtin_bit_cast(f32x4, b.lo);
    const f32x4 ah = __builtin_bit_cast(f32x4, a.hi), bh = __builtin_bit_cast(f32x4, b.hi);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(al[j], bl[j], acc, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(ah[j], bh[j], acc, 0, 0, 0);
  } else if constexpr (EXACT) {
    bf16x8 al[4], bl[4];
    widen(a.lo, al[0], al[1]);
    widen(a.hi, al[2], al[3]);
    widen(b.lo, bl[0], bl[1]);
    widen(b.hi, bl[2], bl[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(al[j], bl[j], acc, 0, 0, 0);
  } else {  // e4m3: 128 values of k at the full 8-bit rate, block scales of 1 (2^(127 - 127))
    const i32x8 av = {(int)a.lo[0], (int)a.lo[1], (int)a.lo[2], (int)a.lo[3], (int)a.hi[0], (int)a.hi[1], (int)a.hi[2], (int)a.hi[3]};
    const i32x8 bv = {(int)b.lo[0], (int)b.lo[1], (int)b.lo[2], (int)b.lo[3], (int)b.hi[0], (int)b.hi[1], (int)b.hi[2], (int)b.hi[3]};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
  }
}

// sigmoid(u) for an activation of v: fp32's gate stops at sigmoid(-88), which a v near the
// type's lowest value would still turn into a result of order 1.
template <class E>
__device__ __forceinline__ float act_gate(float u) {
  const float s = fast_sigmoid<E>(u);
  return sizeof(E) == 4 && u < -87.f ? 0.f : s;
}
// act(v); derivative in d.  E: the type that the result is rounded to
template <class E, bool D>
__device__ __forceinline__ float act_of(int act, float v, float& d) {
  if (act == GDN_ACT_SILU) {
    const float s = act_gate<E>(v);
    if (D) d = dsilu_gate(v, s);
    return v * s;
  }
  if (act == GDN_ACT_GELU) {
    constexpr float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float s = act_gate<E>(c * fmaf(0.044715f * v * v, v, v));
    if (D) {  // (past +-16, where s is 0 or 1, the square may not grow until 0 times it is a NaN)
      const float t = __builtin_amdgcn_fmed3f(v, -16.f, 16.f);
      d = fmaf(v * (s - s * s), c * fmaf(3.f * 0.044715f * t, t, 1.f), s);
    }
    return v * s;
  }
  d = 1.f;
  return v;
}

// f xs ws of 8-bit rows' sums.  The scales' own product may leave fp32's range where the
// result does not (7e-22 each: a result of 1e-37 is off by 2^-10 of it), so f comes first: a
// sum is 0 or between 2^-18 and 2^42 and a scale at least 2^-109, so that f times a scale of 1 at
// most stays in range, and with xs above 1 f ws leaves it only where the result does too.
__device__ __forceinline__ float scaled(float f, float xs, float ws) { return xs <= 1.f ? f * xs * ws : f * ws * xs; }

// Four outputs side by side of row m, from column n on (c of them exist).  Q: there may be scales
template <class O, bool Q = true>
__device__ __forceinline__ void finish4(const Epilogue& e, int64_t m, int N, int n, f32x4 v) {
  const int c = N - n;
  if (c <= 0) return;
  float f[4] = {v[0], v[1], v[2], v[3]}, t[4];
  if (Q && e.x_scale) {
    const float xs = e.x_scale[m];
    ld_part<4>(e.w_scale + n, c, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = scaled(f[i], xs, t[i]);
  }
  if (e.bias) {
    ld_part<4>(static_cast<const O*>(e.bias) + n, c, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += t[i];
  }
  if (e.v_save) {
    float* p = e.v_save + m * N + n;
    if (c >= 4) *reinterpret_cast<f32x4_any*>(p) = f32x4{f[0], f[1], f[2], f[3]};
    else
      for (int i = 0; i < c; ++i) p[i] = f[i];
  }
  if (e.act) {
    float d;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = act_of<O, false>(e.act, f[i], d);
  }
  if (e.r) {
    ld_part<4>(static_cast<const O*>(e.r) + m * e.r_stride + n, c, t);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += t[i];
  }
  O* p = static_cast<O*>(e.out) + m * N + n;
  if (c >= 4) {
    if constexpr (sizeof(O) == 2) *reinterpret_cast<bf16x4_any*>(p) = bf16x4{(bf16)f[0], (bf16)f[1], (bf16)f[2], (bf16)f[3]};
    else *reinterpret_cast<f32x4_any*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  } else {
    for (int i = 0; i < c; ++i) p[i] = to_e<O>(f[i]);
  }
}

// Block j's first row of b among a wave's 64, which is its outputs' first column too.
__device__ __forceinline__ constexpr int blk_b(int j) { return 32 * (j >> 1) + 4 * (j & 1); }

// A lane's sixteen outputs of each of its rows, eight at column n and eight at n + 32:
// what belongs to the columns is loaded once, and one branch decides for all sixteen (a
// tile's epilogue runs while its compute unit's matrix cores wait).
template <class O, bool Q>
struct Columns {
  float b[16], ws[16];
  int n;
  bool whole;  // all sixteen exist
  static constexpr __device__ __forceinline__ int col(int j) { return j < 8 ? j : j + 24; }
  __device__ __forceinline__ Columns(const Epilogue& e, int N, int n_) : n(n_), whole(N - n_ >= 40) {
    if (!whole) return;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      float t[4] = {};
      if (e.bias) ld_full<4>(static_cast<const O*>(e.bias) + n + col(j), t);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[j + i] = t[i];
      if (Q) ld_full<4>(e.w_scale + n + col(j), t);
#pragma unroll
      for (int i = 0; i < 4; ++i) ws[j + i] = t[i];
    }
  }
  __device__ __forceinline__ void finish(const Epilogue& e, int64_t m, int N, const f32x4 (&v)[4]) const {
    // (the branch for scales above 1, which are rare, is a wave's: one for every entry took 1.9 % of
    // 32,768 x 2,048 -> 6,144 in 8 bits)
    const float xs = Q ? e.x_scale[m] : 1.f;
    if (!whole || (Q && !__all(xs <= 1.f))) {
#pragma unroll
      for (int j = 0; j < 4; ++j) finish4<O, Q>(e, m, N, n + blk_b(j), v[j]);
      return;
    }
    float f[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = v[j / 4][j % 4];
    if (Q) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = f[j] * xs * ws[j];
    }
    if (e.bias) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] += b[j];
    }
    const int64_t at = m * N + n;
    if (e.v_save) {
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<f32x4_any*>(e.v_save + at + col(j)) = f32x4{f[j], f[j + 1], f[j + 2], f[j + 3]};
    }
    float d;
    if (e.act == GDN_ACT_SILU) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = act_of<O, false>(GDN_ACT_SILU, f[j], d);
    } else if (e.act == GDN_ACT_GELU) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = act_of<O, false>(GDN_ACT_GELU, f[j], d);
    }
    constexpr int V = 16 / (int)sizeof(O);
    if (e.r) {
#pragma unroll
      for (int j = 0; j < 16; j += V) {
        float t[V];
        ld_full<V>(static_cast<const O*>(e.r) + m * e.r_stride + n + col(j), t);
#pragma unroll
        for (int i = 0; i < V; ++i) f[j + i] += t[i];
      }
    }
    O* p = static_cast<O*>(e.out) + at;
#pragma unroll
    for (int j = 0; j < 16; j += V) {
      if constexpr (V == 8) {
        const float t[8] = {f[j], f[j + 1], f[j + 2], f[j + 3], f[j + 4], f[j + 5], f[j + 6], f[j + 7]};
        *reinterpret_cast<bf16x8_any*>(p + col(j)) = VecIO<bf16, 8>::pack(t);
      } else {
        *reinterpret_cast<f32x4_any*>(p + col(j)) = f32x4{f[j], f[j + 1], f[j + 2], f[j + 3]};
      }
    }
  }
};

// A tile's operand: where its rows start, how far they reach (below 2^31 bytes).
constexpr uint32_t PAST_END = 0x80000000u;
__device__ __forceinline__ u32x4 make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, bytes, 0x00027000u};
}
// 16 bytes a lane from rsrc + off to LDS at `lds` + 16 * lane; past the buffer's end: zeros.
// The compiler does not see these loads: what reads their target waits by hand (lds_wait). It
// sets m0, an input, itself: m0 is not to be written behind its back. The s_nop is the wait
// state between that and the load; descriptors_ready() is theirs for the descriptors.
__device__ __forceinline__ void load_lds(u32x4 rsrc, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" :: "{m0}"(lds), "v"(off), "s"(rsrc) : "memory");
}
// A memory access may read scalars that vector instructions wrote (v_readfirstlane) five
// wait states later.
__device__ __forceinline__ void descriptors_ready(u32x4 a, u32x4 b) { asm volatile("s_nop 4" :: "s"(a), "s"(b)); }
__device__ __forceinline__ void lds_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ int swz_a(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_b(int row) { return ((row >> 1) & 1) | ((row >> 3) & 3) << 1; }

// f(0) .. f(N - 1), each with its number as a constant: past a size of its body a loop is not
// unrolled, and the accumulators that it indexes lie in memory (fp32 4,096^3: 1,670 us, not 980).
template <int... I, class F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) { (f(std::integral_constant<int, I>{}), ...); }
template <int N, class F>
__device__ __forceinline__ void each(F f) { each_of(std::make_integer_sequence<int, N>{}, f); }

// BM x BN tile, WM x WN waves, each TM 16-row blocks of a and 64 rows of b.
template <int T, class O, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void gemm_kernel(GemmParams p) {
  constexpr int W = WM * WN, TM = BM / WM / 16, TN = 4;
  static_assert(BN / WN == 64, "a wave takes 64 rows of b");
  constexpr int NA = BM / 8 / W, NB = BN / 8 / W;  // loads of a wave and step
  constexpr int BUF = (BM + BN) * 128;
  __shared__ __attribute__((aligned(1024))) char smem[2 * BUF];
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
  // Workgroups go round the eight dies: each die takes a run of tiles of its own, in
  // groups of eight tile rows, so that its L2 sees the same rows of a and b again.
  const int tn_n = (p.N + BN - 1) / BN;
  const int64_t tm_n = (p.M + BM - 1) / BM, tiles = tm_n * tn_n;
  int64_t id = block_2d();
  const int split = (int)(id / tiles);
  if (split >= p.splits) return;
  id -= split * tiles;
  {
    const int64_t per = tiles / 8, more = tiles % 8, die = id % 8;
    id = id / 8 + die * per + min(die, more);
  }
  constexpr int GROUP = 8;
  const int64_t g0 = id / (GROUP * (int64_t)tn_n) * GROUP, rows_g = min((int64_t)GROUP, tm_n - g0), in_g = id - g0 * tn_n;
  const int64_t m0 = (g0 + in_g % rows_g) * BM;
  const int n0 = (int)(in_g / rows_g) * BN;

  const int64_t am = min((int64_t)BM, p.M - m0);
  const int bn = min(BN, p.N - n0);
  const u32x4 ra = make_rsrc(static_cast<const char*>(p.a) + m0 * p.lda, (uint32_t)((am - 1) * p.lda + p.kbytes));
  const u32x4 rb = make_rsrc(static_cast<const char*>(p.b) + (int64_t)n0 * p.ldb, (uint32_t)((bn - 1) * p.ldb + p.kbytes));
  const int k0 = split * p.steps * 128, k1 = min(p.kbytes, k0 + p.steps * 128);
  const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem);
  uint32_t oa[NA], ob[NB], ca[NA], cb[NB];  // byte offsets of the lane's pieces; their place along k
#pragma unroll
  for (int j = 0; j < NA; ++j) {
    const int row = (w * NA + j) * 8 + (lane >> 3);
    ca[j] = ((lane & 7) ^ swz_a(row)) * 16;
    oa[j] = (uint32_t)(row * p.lda) + k0 + ca[j];
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int row = (w * NB + j) * 8 + (lane >> 3);
    cb[j] = ((lane & 7) ^ swz_b(row)) * 16;
    ob[j] = (uint32_t)(row * p.ldb) + k0 + cb[j];
  }
  auto request = [&](int k, int buf) {
    const uint32_t at = base + buf * BUF + w * (NA * 1024);
    const uint32_t left = k1 - k;  // pieces past the end of k ask past the buffer's end
#pragma unroll
    for (int j = 0; j < NA; ++j) load_lds(ra, ca[j] < left ? oa[j] : PAST_END, at + j * 1024);
    const uint32_t bt = base + buf * BUF + BM * 128 + w * (NB * 1024);
#pragma unroll
    for (int j = 0; j < NB; ++j) load_lds(rb, cb[j] < left ? ob[j] : PAST_END, bt + j * 1024);
#pragma unroll
    for (int j = 0; j < NA; ++j) oa[j] += 128;
#pragma unroll
    for (int j = 0; j < NB; ++j) ob[j] += 128;
  };
  const int wm = w / WN, wn = w % WN, q = lane >> 4, r16 = lane & 15;
  // fragment addresses: a's block i, row 16 i + r16; b's block j, row blk_b(j) + 8 (r16 / 4) + r16 % 4
  const char* fa = smem + (wm * TM * 16 + r16) * 128;
  const int sa = swz_a(r16);  // (the same for every block: they lie 16 rows apart)
  const int rb0 = 8 * (r16 >> 2) + (r16 & 3);
  const char* fb = smem + BM * 128 + (wn * 64 + rb0) * 128;
  const int sb = swz_b(rb0);  // (blk_b leaves it as it is)
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = zero4();
  descriptors_ready(ra, rb);
  if (k0 < k1) request(k0, 0);
  lds_wait();
  __syncthreads();
  int buf = 0;
  for (int k = k0; k < k1; k += 128) {
    if (k + 128 < k1) request(k + 128, buf ^ 1);
    const char *pa = fa + buf * BUF, *pb = fb + buf * BUF;
    Pieces b[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      b[j].lo = *reinterpret_cast<const u32x4*>(pb + blk_b(j) * 128 + ((q ^ sb) << 4));
      b[j].hi = *reinterpret_cast<const u32x4*>(pb + blk_b(j) * 128 + (((q + 4) ^ sb) << 4));
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      Pieces a;
      a.lo = *reinterpret_cast<const u32x4*>(pa + i * 2048 + ((q ^ sa) << 4));
      a.hi = *reinterpret_cast<const u32x4*>(pa + i * 2048 + (((q + 4) ^ sa) << 4));
#pragma unroll
      for (int j = 0; j < TN; ++j) mma_step<T, sizeof(O) == 4>(acc[i][j], b[j], a);
    }
    lds_wait();
    __syncthreads();
    buf ^= 1;
  }
  const int n = n0 + wn * 64 + 8 * q;
  if (n >= p.N) return;
  if (p.splits > 1) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + (wm * TM + i) * 16 + r16;
      if (m >= p.M) break;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        float* t = p.part + (split * p.M + m) * p.N + n + blk_b(j);
        const int c = p.N - n - blk_b(j);
        if (c >= 4) *reinterpret_cast<f32x4_any*>(t) = acc[i][j];
        else
          for (int x = 0; x < c; ++x) t[x] = acc[i][j][x];
      }
    }
    return;
  }
  const Columns<O, T == GDN_E4M3> cols(p.e, p.N, n);
  each<TM>([&](auto i) {
    const int64_t m = m0 + (wm * TM + i) * 16 + r16;
    if (m < p.M) cols.finish(p.e, m, p.N, acc[i]);
  });
}

// The splits' sums, in order, and the epilogue: four outputs a thread.
template <class O>
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmParams p) {
  const int per = (p.N + 3) / 4;
  const int64_t i = block_2d() * 256 + threadIdx.x, m = i / per;
  if (m >= p.M) return;
  const int n = (int)(i - m * per) * 4, c = p.N - n;
  f32x4 s = zero4();
  for (int k = 0; k < p.splits; ++k) {
    float f[4];
    ld_part<4>(p.part + (k * p.M + m) * p.N + n, c, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += f[e];
  }
  finish4<O>(p.e, m, p.N, n, s);
}

// Up to 16 MT rows of x by 16 outputs: eight waves take every eighth 128 bytes of k.
// Bound: the weight's bytes, and latency: 16 x 2,048 -> 6,144 in 10.5 us (25 MB; 5.2 at the
// rate of a copy), 16 x 8,192 -> 8,192 in 34 (28).
typedef u32x4 u32x4_any __attribute__((aligned(1)));
__device__ __forceinline__ u32x4 ld_piece(const char* row, int k, int kbytes) {
  if (k + 16 <= kbytes) return *reinterpret_cast<const u32x4_any*>(row + k);
  u32x4 v = {};
  for (int i = 0; i < 16 && k + i < kbytes; ++i) v[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
  return v;
}
// With more rows a workgroup takes 16 NT outputs, so that the rows of x, which every
// workgroup reads whole, are read less often (32 and 64 rows
// of 2,048 to 6,144: 10.3 and 13.4 us with 32 outputs, 12.8 and 20.3 with 16).
template <int T, class O, int MT, int NT>
__global__ __launch_bounds__(512) void skinny_kernel(SkinnyParams p) {
  constexpr int W = 8;
  __shared__ f32x4 red[W][NT * MT][64];
  const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), q = lane >> 4, r16 = lane & 15;
  const int64_t first = block_2d() * (16 * NT);
  if (first >= p.N) return;
  const int n0 = (int)first;
  const char *wr[NT], *xr[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) wr[j] = static_cast<const char*>(p.w) + min(first + j * 16 + r16, (int64_t)p.N - 1) * p.w_stride;
#pragma unroll
  for (int i = 0; i < MT; ++i) xr[i] = static_cast<const char*>(p.x) + (int64_t)min(i * 16 + r16, p.M - 1) * p.x_stride;
  f32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = zero4();
  constexpr int U = MT <= 2 ? 4 : 2;  // steps requested together
  auto steps = [&](int k, auto piece) {
    Pieces b[U][NT], a[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ku = k + u * W * 128 + q * 16;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        b[u][j].lo = piece(wr[j], ku);
        b[u][j].hi = piece(wr[j], ku + 64);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        a[u][i].lo = piece(xr[i], ku);
        a[u][i].hi = piece(xr[i], ku + 64);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) mma_step<T, sizeof(O) == 4>(acc[j][i], b[u][j], a[u][i]);
  };
  int k = w * 128;
  // whole steps without a test in front of each load, which would keep them apart
  for (; k + (U - 1) * W * 128 + 128 <= p.kbytes; k += U * W * 128)
    steps(k, [](const char* row, int at) { return *reinterpret_cast<const u32x4_any*>(row + at); });
  for (; k < p.kbytes; k += U * W * 128) steps(k, [&](const char* row, int at) { return ld_piece(row, at, p.kbytes); });
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) red[w][j * MT + i][lane] = acc[j][i];
  __syncthreads();
  // four outputs of a row a thread: entry (j MT + i, lane) holds columns 16 j + 4 (lane / 16) of row 16 i + lane % 16
  for (int t = threadIdx.x; t < NT * MT * 64; t += 512) {
    const int ji = t / 64, l = t % 64;
    f32x4 s = red[0][ji][l];
#pragma unroll
    for (int v = 1; v < W; ++v) s += red[v][ji][l];
    const int m = ji % MT * 16 + (l & 15);
    if (m < p.M) finish4<O>(p.e, m, p.N, n0 + ji / MT * 16 + 4 * (l >> 4), s);
  }
}

// Eight elements at p, which is aligned to four of them or more; rows of copies hold whole
// 16 bytes, so only fp32's may end after four.
__device__ __forceinline__ void put8(float* p, const float (&f)[8], bool both) {
  *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  if (both) *reinterpret_cast<f32x4*>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
}
__device__ __forceinline__ void put8(bf16* p, const float (&f)[8], bool) { store_vec<bf16, 8>(p, f); }

// 64 x 64 elements a workgroup, eight side by side a thread and access in either
// direction: eight threads fill 128 bytes of a row, and of a turned row.  Stride 65 puts
// the 64 values that a wave touches at once on 64 banks both ways.  Bound: memory (16,384 x
// 6,144 with v, both copies: 1.0 GB in 219 us, 4.6 TB/s).
template <class E>
__global__ __launch_bounds__(256) void pack_kernel(PackJobs jobs) {
  __shared__ float tile[64][65];
  int64_t blk = block_2d();
  int job = 0;
  while (job < jobs.n - 1 && blk >= jobs.blocks(job)) blk -= jobs.blocks(job++);
  const PackParams& p = jobs.job[job];
  const int cols_n = (p.C + 63) / 64;
  const int64_t br = blk / cols_n, r0 = br * 64;
  const int c0 = (int)(blk - br * cols_n) * 64;
  if (r0 >= p.R) return;
  const int ti = threadIdx.x / 8, tj = threadIdx.x % 8 * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = r0 + ti + 32 * h;
    const int c = c0 + tj;
    float f[8] = {};
    if (r < p.R && c < p.C) {
      ld_part<8>(static_cast<const E*>(p.in) + r * p.ld + c, p.C - c, f);
      if (p.v) {
        float v[8];
        ld_part<8>(p.v + r * p.C + c, p.C - c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float d;
          act_of<E, true>(p.act, v[e], d);
          f[e] *= d;
        }
      }
    }
    if (p.rows && r < p.R && c < p.ldo) put8(static_cast<E*>(p.rows) + r * p.ldo + c, f, c + 8 <= p.ldo);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[ti + 32 * h][tj + e] = f[e];
  }
  if (!p.cols && !p.sums) return;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = c0 + ti + 32 * h;
    float g[8], s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      g[e] = tile[tj + e][ti + 32 * h];
      s += g[e];
    }
    if (p.cols && c < p.C && r0 + tj < p.ldt) put8(static_cast<E*>(p.cols) + c * p.ldt + r0 + tj, g, r0 + tj + 8 <= p.ldt);
    if (p.sums) {
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) s += __shfl_xor(s, o, 64);
      if (c < p.C && tj == 0) p.sums[br * p.C + c] = s;
    }
  }
}
// Bytes copied row by row (8-bit rows).
__global__ __launch_bounds__(256) void pack_bytes_kernel(PackParams p) {
  const int64_t i = block_2d() * 256 + threadIdx.x, per = p.ldo / 16, r = i / per;
  if (r >= p.R) return;
  const int c = (int)(i - r * per) * 16;
  const u32x4 v = ld_piece(static_cast<const char*>(p.in) + r * p.ld, c, p.C);
  *reinterpret_cast<u32x4*>(static_cast<char*>(p.rows) + r * p.ldo + c) = v;
}

template <int T, class O>
hipError_t gemm_any(const GemmParams& p, const GemmPlan& g, hipStream_t st) {
  const int64_t tiles = (p.M + g.tile - 1) / g.tile * ((p.N + g.tile - 1) / g.tile);
  const dim3 grid = blocks_2d(tiles * g.splits);
  if (g.tile == 256) hipLaunchKernelGGL((gemm_kernel<T, O, 256, 256, 2, 4>), grid, dim3(512), 0, st, p);
  else hipLaunchKernelGGL((gemm_kernel<T, O, 128, 128, 2, 2>), grid, dim3(256), 0, st, p);
  if (hipError_t e = hipGetLastError(); e != hipSuccess || g.splits == 1) return e;
  hipLaunchKernelGGL((gemm_join_kernel<O>), blocks_2d((p.M * ((p.N + 3) / 4) + 255) / 256), dim3(256), 0, st, p);
  return hipGetLastError();
}
template <int T, class O>
hipError_t skinny_any(const SkinnyParams& p, hipStream_t st) {
  auto grid = [&](int nt) { return blocks_2d(((int64_t)p.N + 16 * nt - 1) / (16 * nt)); };
  if (p.M <= 16) hipLaunchKernelGGL((skinny_kernel<T, O, 1, 1>), grid(1), dim3(512), 0, st, p);
  else if (p.M <= 32) hipLaunchKernelGGL((skinny_kernel<T, O, 2, 2>), grid(2), dim3(512), 0, st, p);
  else hipLaunchKernelGGL((skinny_kernel<T, O, 4, 2>), grid(2), dim3(512), 0, st, p);
  return hipGetLastError();
}

}  // namespace

// The cheapest of both tiles and a few splits of k, by a model of their times in us that
// was fitted to bf16 products of 64 to 16,384 rows (a step: 128 bytes of k).  A round of
// 256 x 256 tiles, one a compute unit, takes 1.55 a step and 11 to start and end; 128 x
// 128 tiles take 0.69 and 5 one a compute unit, 1 and 5 two.  Splits add a join: its bytes
// (mostly from cache), and a launch.  Measured against the other choice: 4,096 x 2,048 ->
// 2,048 in tiles of 128 37 us, of 256 60; 8,192 rows 72 and 61; 128 rows -> 6,144 in 4 parts
// 20, whole 25; sums over 8,192 to 2,048 x 2,048 of 128 in 2 parts 80, whole 89, of 256 in 4
// parts 93; over 32,768 of 256 in 4 parts 276, whole 652, of 128 in 2 parts 310.
GemmPlan gemm_plan(int64_t M, int N, int64_t kbytes, int esize, int cus) {
  const int steps = (int)((kbytes + 127) / 128);
  const double slow = esize == 4 ? 8. : 1.;  // fp32's matrix instructions against bf16's
  GemmPlan best{256, 1, steps};
  double least = 0.;
  for (int tile : {256, 128}) {
    const int64_t tiles = (M + tile - 1) / tile * ((N + tile - 1) / tile);
    for (int s = 1; s <= 16 && (s == 1 || (s <= steps / 8 && tiles * s <= 4 * (int64_t)cus)); s *= 2) {
      const double k = (steps + s - 1) / s * slow;
      const int64_t n = tiles * s;
      double t;
      if (tile == 256) {
        t = (double)((n + cus - 1) / cus) * (1.55 * k + 11.);
      } else {
        const int64_t rest = n % (2 * cus);
        t = (double)(n / (2 * cus)) * (k + 5.) + (rest == 0 ? 0. : rest <= cus ? 0.69 * k + 5. : k + 5.);
      }
      if (s > 1) t += 4. + (double)M * N * (8. * s + 2.) / 5e6;
      if (least == 0. || t < least) {
        least = t;
        best = GemmPlan{tile, s, (steps + s - 1) / s};
      }
    }
  }
  if (best.steps > 0) best.splits = std::max(1, (steps + best.steps - 1) / best.steps);  // none of them empty
  return best;
}
hipError_t launch_gemm(int dtype, int out_dtype, const GemmParams& p, const GemmPlan& g, hipStream_t st) {
  if (dtype == GDN_BF16) return gemm_any<GDN_BF16, bf16>(p, g, st);
  if (dtype == GDN_F32) return gemm_any<GDN_F32, float>(p, g, st);
  return out_dtype == GDN_BF16 ? gemm_any<GDN_E4M3, bf16>(p, g, st) : gemm_any<GDN_E4M3, float>(p, g, st);
}
hipError_t launch_skinny(int dtype, int out_dtype, const SkinnyParams& p, hipStream_t st) {
  if (dtype == GDN_BF16) return skinny_any<GDN_BF16, bf16>(p, st);
  if (dtype == GDN_F32) return skinny_any<GDN_F32, float>(p, st);
  return out_dtype == GDN_BF16 ? skinny_any<GDN_E4M3, bf16>(p, st) : skinny_any<GDN_E4M3, float>(p, st);
}
hipError_t launch_pack(int dtype, const PackJobs& jobs, hipStream_t st) {
  if (dtype == GDN_E4M3) {
    const PackParams& p = jobs.job[0];
    hipLaunchKernelGGL(pack_bytes_kernel, blocks_2d((p.R * (p.ldo / 16) + 255) / 256), dim3(256), 0, st, p);
  } else {
    int64_t blocks = 0;
    for (int i = 0; i < jobs.n; ++i) blocks += jobs.blocks(i);
    if (dtype == GDN_BF16) hipLaunchKernelGGL((pack_kernel<bf16>), blocks_2d(blocks), dim3(256), 0, st, jobs);
    else hipLaunchKernelGGL((pack_kernel<float>), blocks_2d(blocks), dim3(256), 0, st, jobs);
  }
  return hipGetLastError();
}

}  // namespace gdn
