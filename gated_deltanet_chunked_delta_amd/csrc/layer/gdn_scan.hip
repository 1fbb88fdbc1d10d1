// gdn_scan.hip -- the sweeps of the selective state space scan on the matrix
// cores.
//
// Per sequence and head, with step D_t and decay a_t = D_t A (A <= 0):
//   h_t = exp(a_t) h_{t-1} + D_t B_t x_t^T     (Dk x Dv),      y_t = h_t^T C_t + D x_t
// and backwards in time, for the gradient dh of the states,
//   dh_t = exp(a_{t+1}) dh_{t+1} + C_t dy_t^T
//   dx_t = D_t dh_t^T B_t + D dy_t,   dB_t = D_t dh_t x_t,   dC_t = h_t dy_t
// (dB, dC summed over the heads that share them).  Both directions are one
// sweep (SweepParams) with the roles of B, C, x and dy exchanged; backwards the
// rows of a chunk are taken in reverse, so that every chunk matrix stays lower
// triangular.  A chunk of 64 tokens with keys K, queries Q, values V, the state
// S before it and cum_r the decay from the chunk's start to row r:
//   out1 = (L o Q K^T o sw) V + exp(cum) Q S                  value sweep
//   out2 = (L o W V^T o sw) K + exp(cum) W S^T                key sweep
//   S'   = exp(tot) S + sum_s exp(tot - cum_s) sw_s K_s V_s^T
// with L[t][s] = exp(cum_t - cum_s), s <= t.
//
// Gradient of the decays.  da_t = <dh_t, exp(a_t) h_{t-1}> obeys
//   da_t = da_{t+1} + rt_t - D_t ct_t,
//   rt_t = C_t . (exp(a_t) h_{t-1}) dy_t,   ct_t = B_t . (exp(a_{t+1}) dh_{t+1}) x_t
// (the terms of a token with itself cancel and are left out, so under strong
// decay both sides are as small as da itself).  The recursion is undamped, so
// it restarts at every chunk's end from <h, dh> there: the forward key sweep
// leaves its states and the backward one takes the products, in 64 bits; what a chunk's
// sums miss the product at its start by is spread over its tokens (but in a first
// chunk with an h0, where <h0, dh0> is of larger terms than those sums).  A pair of
// tokens of one chunk enters rt_t of the later and D_t ct_t of the earlier one and
// cancels before both: so the forward key sweep takes both sums from the same
// products (rt; rt2 by the earlier token), and of the backward one's ct only the part
// that comes from the state (rt2) enters the recursion.  Error of dA in fp32 roundings of
// its terms (16 heads of 128 x 128, 4,096 tokens fp32 and 8,192 bf16; 4 of 64 x 64, 3,392
// fp32 with h0): 5.2, 3.9, 5.5; with the pairs from two sweeps, products in 32 bits and
// the spread in every chunk 8.0, 7.1, 8.7 (and 2 % less time of a training pass).  Then
// dD_t = ct_t + (C_t . B_t)(x_t . dy_t) + A da_t.
//
// Precision.  Products of bf16 inputs are exact and summed in fp32.  An fp32
// factor (the state, keys or values times their decay) enters a product as
// three bf16 parts, 24 bits in all, wherever its rounding would reach an fp32
// result: the states, and the row terms rt, ct behind dA and ddt.  Where only a
// bf16 output depends on it it enters in two parts, each rounded (2^-18 of it): the
// chunk matrix in out2, and the values' decays in a segment whose state does not
// leave.  In out1 the chunk matrix and the state are rounded to bf16 once, together
// an error like the output's own rounding, unless the caller asks for outputs that
// are rounded only once (round_once): then they too enter in two parts.  Rms error of
// y against 64 bits, 4,096 tokens of 2 heads of 128 x 128: 2.04e-3, with round_once
// 1.65e-3, which is the final rounding's alone; time with it: 333
// tokens 24.0 us instead of 23.5, 8,192 81.9 (79.2), 65,536 132 (120), a training
// pass of 4 x 4,096 609 (589).
// fp32 inputs take the fp32 matrix instructions throughout.
//
// Decay factors are products of factors <= 1 over 16-row blocks (a power of a
// sum inside a block, a factor for the blocks between), so that no difference
// of long sums is formed and only the four diagonal blocks need one per entry.
//
// Bound: neither memory nor the matrix cores alone.  A workgroup fills a compute
// unit (tiles and states: LDS, and up to 256 registers a lane at two waves a SIMD),
// and a chunk's phases wait for each other.  Measured, bf16, 16 heads of 128 x 128
// with one B and C: 8,192 tokens forward, states 29 us, join 14, outputs 44 (74 MB:
// 15 us at the memory's rate); 4 x 4,096 tokens, states 43, y 71, dx 69, dC 171, dB
// 157 us.  A value sweep's chunk takes about 14,000 cycles, a key sweep's about
// 36,000 for four slices, of which its matrix instructions would fill 8,000; its
// share of a chunk's state out (or in) and its parts of dC (dB) are 60 MB over the
// chip, 12 us at the memory's rate.  fp32 (tiles of twice the bytes wait in registers):
// 8,192 tokens of 16 heads of 128 x 128 forward 268 us, backward 666 us.
// Registers: value sweeps with outputs spill in fp32 (bytes a lane: Dk = 64, two waves 128
// forwards and 28 backwards; Dk = 128, four waves 248 and 148, two waves 564 and 412)
// and in bf16 where a group has one head of 64 columns and Dk = 128 (104 and 44);
// the dC sweep <bf16, 128, 4> spills 8.  Key sweeps of Dk = 64 with four slices, with two in
// fp32, and with two backwards in bf16 hold 266 to 343 registers: one wave a SIMD.
#include "gdn_layer.h"
#include "gdn_scan_device.h"

namespace gdn {

namespace {

// ---------------------------------------------------------------- operand parts
// An fp32 operand as bf16 parts whose sum is exact (24 bits, cut, not rounded:
// 8 + 8 + 8), or as itself.
template <class E> struct Parts;
template <> struct Parts<bf16> {
  static constexpr int N = 3;
  Frag<bf16> p[3];
};
template <> struct Parts<float> {
  static constexpr int N = 1;
  Frag<float> p[1];
};
__device__ __forceinline__ void split(Parts<float>& o, const f32x4& lo, const f32x4& hi) { pack_frag(o.p[0], lo, hi); }
__device__ __forceinline__ void split(Parts<bf16>& o, const f32x4& lo, const f32x4& hi) {
  typedef uint32_t u32x4 __attribute__((__vector_size__(16)));
  float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __builtin_bit_cast(uint32_t, x[2 * i]), b = __builtin_bit_cast(uint32_t, x[2 * i + 1]);
      v[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // the two high halves
      if (part < 2) {
        x[2 * i] -= __builtin_bit_cast(float, a & 0xFFFF0000u);
        x[2 * i + 1] -= __builtin_bit_cast(float, b & 0xFFFF0000u);
      }
    }
    o.p[part].v = __builtin_bit_cast(bf16x8, v);
  }
}
// The first two parts rounded instead of cut: off by at most 2^-18 of the
// operand to either side (two cut ones fall short by up to 2^-16).
__device__ __forceinline__ void split2(Parts<float>& o, const f32x4& lo, const f32x4& hi) { pack_frag(o.p[0], lo, hi); }
__device__ __forceinline__ void split2(Parts<bf16>& o, const f32x4& lo, const f32x4& hi) {
  const PFrag<bf16> f(Frag<float>{lo, hi});
  o.p[0] = f.hi;
  o.p[1] = f.lo;
}

// Fragment whose k-slots walk down a column of a row-major LDS matrix (rows
// k0 + 4g .. + 3 and k0 + 16 + 4g .. + 3, the order of two stacked accumulator
// tiles).  Lane 4a + b of a group takes column c0 + 8a + 4h + b: the pair of
// tiles h = 0, 1 then covers 32 columns such that lane group g's rows of the
// two tiles, stacked, are the columns c0 + 8g .. c0 + 8g + 7 in order -- a
// state tile pair pairs with 16-byte row fragments (ld_frag8), and a lane
// stores eight consecutive results.
__device__ __forceinline__ Frag<bf16> ld_col(const bf16* base, int ld, int k0, int c0, int h) {
  const int l = lane_id();
  const bf16* p = base + (k0 + (l >> 2)) * ld + c0 + 8 * (l & 3) + 4 * h;
  const bf16x4 a = ds_read_tr16(p), b = ds_read_tr16(p + 16 * ld);
  Frag<bf16> f;
  f.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return f;
}
__device__ __forceinline__ Frag<float> ld_col(const float* base, int ld, int k0, int c0, int h) {
  const int l = lane_id(), g = l >> 4, q = (l >> 2) & 3, b = l & 3;
  const float* p = base + (k0 + 4 * g + b) * ld + c0 + 8 * q + 4 * h;
  Frag<float> f;
  f.lo = quad_transpose(*reinterpret_cast<const f32x4*>(p));
  f.hi = quad_transpose(*reinterpret_cast<const f32x4*>(p + 16 * ld));
  return f;
}
__device__ __forceinline__ void frag_f32(const Frag<bf16>& f, f32x4& lo, f32x4& hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = (float)f.v[i];
    hi[i] = (float)f.v[4 + i];
  }
}
__device__ __forceinline__ void frag_f32(const Frag<float>& f, f32x4& lo, f32x4& hi) {
  lo = f.lo;
  hi = f.hi;
}

// The matrix cores' sums come out low by a fraction of a unit in the last place
// on average, whatever their sign.  A state gathers such errors chunk by chunk,
// and dA and the bias's gradient add products of two states over all tokens.  So a
// state is kept with its sign turned over from chunk to chunk of its sequence
// (sign_of chunk boundary b) and the errors of neighbouring chunks cancel: over 48 heads
// of 16,384 tokens the error of dA has a mean of 0.5 fp32 roundings of its terms, and
// of -12 with states of one sign.
__device__ __forceinline__ float sign_of(int b) { return b & 1 ? -1.f : 1.f; }

// Keeps the instruction scheduler from moving work across: without it the reads
// of every unrolled step are hoisted to the front and registers spill.
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// a times a value held in two parts (about 16 bits of it).
__device__ __forceinline__ void mma_hi_lo(f32x4& acc, const Frag<bf16>& a, const PFrag<bf16>& b) {
  mma(acc, a, b.lo);
  mma(acc, a, b.hi);
}
__device__ __forceinline__ void mma_hi_lo(f32x4& acc, const Frag<float>& a, const PFrag<float>& b) { mma(acc, a, b.f); }
__device__ __forceinline__ void mma_hi_lo(f32x4& acc, const PFrag<bf16>& a, const Frag<bf16>& b) {
  mma(acc, a.lo, b);
  mma(acc, a.hi, b);
}

// Tile of the lower triangle, tile (tb, sb) at index tb (tb + 1) / 2 + sb.
__device__ __forceinline__ void tri_tile(int idx, int& tb, int& sb) {
  tb = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
  sb = idx - tb * (tb + 1) / 2;
}

// LDS row lengths: 16-byte rows, staggered over the banks.
template <class E> constexpr int row_ld(int n) { return n + 16 / (int)sizeof(E); }

// ---------------------------------------------------------------- a chunk's rows and decays
struct ChunkRows {
  int64_t base;  // first token (global row)
  int nt;        // tokens, 1 .. CH
};
// Token of row r relative to the chunk's first.
template <bool REV>
__device__ __forceinline__ int tok_of(const ChunkRows& c, int r) { return REV ? c.nt - 1 - r : r; }
template <bool REV>
__device__ __forceinline__ int64_t row_of(const ChunkRows& c, int r) { return c.base + tok_of<REV>(c, r); }
// Chunk i of a segment in sweep order.
template <bool REV>
__device__ __forceinline__ ChunkRows chunk_rows(const SegRange& s, int i) {
  const int nch = (s.len + CH - 1) / CH, c = REV ? nch - 1 - i : i;
  ChunkRows r;
  r.base = s.row0 + (int64_t)c * CH;
  r.nt = min(CH, s.len - c * CH);
  return r;
}
// The chunk boundary (within the sequence) that a sweep's state stands at before
// its chunk i of nch.
template <bool REV>
__device__ __forceinline__ int boundary(const SegRange& s, int nch, int i) { return REV ? s.c0 + nch - i : s.c0 + i; }
// The segment, its fields known to be the same in every lane.
__device__ __forceinline__ void make_uniform(SegRange& r) {
  r.n = __builtin_amdgcn_readfirstlane(r.n);
  r.s = __builtin_amdgcn_readfirstlane(r.s);
  r.ns = __builtin_amdgcn_readfirstlane(r.ns);
  r.len = __builtin_amdgcn_readfirstlane(r.len);
  r.c0 = __builtin_amdgcn_readfirstlane(r.c0);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)r.row0);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(r.row0 >> 32));
  r.row0 = (int64_t)((uint64_t)hi << 32 | lo);
}

// DPP moves of 64-bit values (rows of 16 lanes; lanes without a source get 0).
template <int CTRL>
__device__ __forceinline__ double dpp_mov_d(double x) {
  typedef int i32x2 __attribute__((__vector_size__(8)));
  i32x2 v = __builtin_bit_cast(i32x2, x);
  v[0] = dpp_mov<CTRL>(v[0]);
  v[1] = dpp_mov<CTRL>(v[1]);
  return __builtin_bit_cast(double, v);
}
__device__ __forceinline__ double readlane_d(double x, int lane) {
  typedef int i32x2 __attribute__((__vector_size__(8)));
  i32x2 v = __builtin_bit_cast(i32x2, x);
  v[0] = __builtin_amdgcn_readlane(v[0], lane);
  v[1] = __builtin_amdgcn_readlane(v[1], lane);
  return __builtin_bit_cast(double, v);
}
// Sum over the 16 lanes of each row, in every lane.
__device__ __forceinline__ double row16_sum_d(double x) {
  x += dpp_mov_d<0xB1>(x);   // lane ^ 1
  x += dpp_mov_d<0x4E>(x);   // lane ^ 2
  x += dpp_mov_d<0x141>(x);  // half-row mirror
  x += dpp_mov_d<0x140>(x);  // row mirror
  return x;
}
// Sums over the 16 lanes of each row of four values at once: lane t gets that of
// x[t % 4].
__device__ __forceinline__ float row16_sum4(const f32x4& x) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  const float a = (odd ? x[1] : x[0]) + quad_xor<1>(odd ? x[0] : x[1]);
  const float b = (odd ? x[3] : x[2]) + quad_xor<1>(odd ? x[2] : x[3]);
  float c = (high ? b : a) + quad_xor<2>(high ? a : b);
  c += dpp_mov<0x128>(c);  // row rotated by 8
  return c + dpp_mov<0x124>(c);
}
// Sums over the four 16-lane groups of four values at once: lane 16 g + t gets
// the sum of x[g] over lanes t, 16 + t, 32 + t, 48 + t.  Exchanging odd with even
// lane rows of two values puts the halves of both sums side by side.
__device__ __forceinline__ float sum_groups4(const float (&x)[4]) {
  auto add = [](unsigned a, unsigned b) { return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b); };
  auto add16 = [&](float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
    return add(r[0], r[1]);
  };
  const float ab = add16(x[0], x[1]), cd = add16(x[2], x[3]);
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, ab), __builtin_bit_cast(unsigned, cd), false, false);
  return add(r[0], r[1]);
}

// Decay factors of one head's chunk, in LDS.
struct ChunkDecay {
  double p16[CH];  // sum of log2 decays from the row's 16-row block's start (its first row's own step included)
  float sw[CH];    // weight of a source row (0 past the end)
  float tw[CH];    // weight of a target row
  float tf[CH];    // decay from the chunk's start
  float row[CH];   // decay from the block's start (2^p16)
  float col[CH];   // decay from the row to its block's end, times sw
  float end[CH];   // decay from the row to the chunk's end, times sw
  float btw[4];    // decay over blocks 1, 2, and both; over the chunk
  __device__ __forceinline__ float between(int tb, int sb) const {
    return tb - sb < 2 ? 1.f : tb - sb == 3 ? btw[2] : btw[tb - 2];
  }
};
// 2^x of a 64-bit sum to fp32 precision: the instruction's exponent rounded to
// 24 bits, and the remainder's first-order factor (an exponent of -8 rounded
// alone would cost four bits of the result).
__device__ __forceinline__ float exp2_sum(double x) {
  const float hi = (float)x;
  const float e = __builtin_amdgcn_exp2f(hi);
  return hi < -126.f ? e : e + e * ((float)(x - hi) * 0.69314718f);
}
// Filled by one wave, lane = row, from the row's dt (requested a chunk ahead)
// and the head's constants.  Forwards the step onto a row is its own decay;
// backwards it is the previous (later) token's, and the state that leaves the
// chunk takes the last row's decay as well.  Sums of log decays are held in 64
// bits: both directions then weigh a pair of tokens alike, to fp32 rounding,
// which the decay gradient's differences of them need.
struct HeadConst {
  float A, bias;
  template <class P>
  __device__ __forceinline__ void load(const P& p, int h) {
    A = p.A[h];
    bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  }
};
// The bits of a row's dt, converted only where they are used (a conversion here
// would wait for the load).
template <bool REV, class P>
__device__ __forceinline__ uint32_t load_dt(const P& p, const ChunkRows& c, int h) {
  const int r = lane_id(), t = tok_of<REV>(c, r);
  const int64_t at = c.base * p.dt_stride + h;
  const uint32_t off = r < c.nt ? (uint32_t)(t * (int)p.dt_stride) : 0u;
  return p.dt_f32 ? (static_cast<const uint32_t*>(p.dt) + at)[off] : (static_cast<const uint16_t*>(p.dt) + at)[off];
}
template <class P>
__device__ __forceinline__ float dt_value(const P& p, uint32_t bits) {
  return __builtin_bit_cast(float, p.dt_f32 ? bits : bits << 16);
}
template <bool REV, class P>
__device__ __forceinline__ void fill_decay(ChunkDecay& o, const P& p, const HeadConst& hc, uint32_t bits, int nt) {
  const int r = lane_id();
  const float raw = dt_value(p, bits) + hc.bias;
  const float d = r < nt ? (p.softplus ? scan_softplus(raw) : raw) : 0.f;
  const double A2 = (double)hc.A * 1.4426950408889634;
  double step = d * A2, fin = 0.;
  if (REV) {
    fin = readlane_d(step, 63);
    const float dp = __shfl_up(d, 1, 64);
    step = r == 0 ? 0. : dp * A2;
  }
  // inclusive prefix and exclusive suffix sums in 16-row blocks
  double pre = step;
  pre += dpp_mov_d<0x111>(pre);
  pre += dpp_mov_d<0x112>(pre);
  pre += dpp_mov_d<0x114>(pre);
  pre += dpp_mov_d<0x118>(pre);
  double after = dpp_mov_d<0x101>(step);
  after += dpp_mov_d<0x101>(after);
  after += dpp_mov_d<0x102>(after);
  after += dpp_mov_d<0x104>(after);
  after += dpp_mov_d<0x108>(after);
  const double b0 = readlane_d(pre, 15), b1 = readlane_d(pre, 31), b2 = readlane_d(pre, 47), b3 = readlane_d(pre, 63);
  const int blk = r >> 4;
  const double before = blk == 0 ? 0. : blk == 1 ? b0 : blk == 2 ? b0 + b1 : b0 + b1 + b2;
  const double later = (blk == 0 ? b1 + b2 + b3 : blk == 1 ? b2 + b3 : blk == 2 ? b3 : 0.) + fin;
  const float w = r < nt ? 1.f : 0.f, sw = REV ? w : d;
  const float row = exp2_sum(pre), col = exp2_sum(after) * sw;
  o.p16[r] = pre;
  o.sw[r] = sw;
  o.tw[r] = REV ? d : w;
  o.tf[r] = exp2_sum(before) * row;
  o.row[r] = row;
  o.col[r] = col;
  o.end[r] = exp2_sum(later) * col;
  if (r < 4) {
    const double t = r == 0 ? b1 : r == 1 ? b2 : r == 2 ? b1 + b2 : b0 + b1 + b2 + b3 + fin;
    o.btw[r] = exp2_sum(t);
  }
}
// The factors L o sw of tile (tb, sb) for this lane's entries (s = 4g + i, t = lane % 16).
template <bool PRECISE>
__device__ __forceinline__ f32x4 tile_decay(const ChunkDecay& d, int tb, int sb) {
  const int l = lane_id(), t = l & 15, g = l >> 4;
  f32x4 f;
  if (sb < tb) {
    f = *reinterpret_cast<const f32x4*>(&d.col[16 * sb + 4 * g]) * (d.row[16 * tb + t] * d.between(tb, sb));
  } else {
    const double pt = d.p16[16 * tb + t];
    const double* ps = &d.p16[16 * sb + 4 * g];
    const f32x4 sw = *reinterpret_cast<const f32x4*>(&d.sw[16 * sb + 4 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double x = pt - ps[i];
      f[i] = 4 * g + i <= t ? (PRECISE ? exp2_sum(x) : __builtin_amdgcn_exp2f((float)x)) * sw[i] : 0.f;
    }
  }
  return f;
}

// ---------------------------------------------------------------- a chunk's rows in memory
// The rows of a chunk as a buffer: base at the chunk's first token, its length
// the chunk's own tokens.  Lane offsets are 32 bits; a row past the end lies
// past the buffer, and backwards, where rows run down from the last token, at a
// negative (huge unsigned) offset: loads give 0 there and stores do nothing, so
// ragged chunks need no branch.  64 rows of a legal stride are below 2^31 bytes.
typedef uint32_t u32x4 __attribute__((__vector_size__(16)));
struct RowBuf {
  __amdgpu_buffer_rsrc_t rsrc;
  int shift;  // bytes that the offsets of a full chunk run past this one's (backwards)
};
template <bool REV, class E>
__device__ __forceinline__ RowBuf row_buf(const E* base, int64_t stride, int width, int nt, bool live = true) {
  RowBuf b;
  const int bytes = live ? ((nt - 1) * (int)stride + width) * (int)sizeof(E) : 0;
  b.rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(base), 0, bytes, 0x00027000);
  b.shift = REV ? (CH - nt) * (int)stride * (int)sizeof(E) : 0;
  return b;
}
// Offset of row r (of a full chunk), entry e.
template <bool REV, class E>
__device__ __forceinline__ int row_off(int r, int64_t stride, int e) {
  return ((REV ? CH - 1 - r : r) * (int)stride + e) * (int)sizeof(E);
}
__device__ __forceinline__ u32x4 ld16(const RowBuf& b, int off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b.rsrc, off - b.shift, 0, 0));
}
template <class V>
__device__ __forceinline__ void st16(const RowBuf& b, int off, const V& v) {
  static_assert(sizeof(V) == 16, "one 16-byte store");
  typedef unsigned u4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), b.rsrc, off - b.shift, 0, 0);
}

// Four results as entries of a row.
__device__ __forceinline__ void st_row4(const RowBuf& b, int off, const f32x4& v, float*) { st16(b, off, v); }
__device__ __forceinline__ void st_row4(const RowBuf& b, int off, const f32x4& v, bf16*) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  const bf16x4 o = {(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, o), b.rsrc, off - b.shift, 0, 0);
}

// A chunk's [CH][C] tile into registers, then into LDS, by NT threads.
template <class E, int C, int NT, bool REV>
struct TileStage {
  static constexpr int PPR = C * (int)sizeof(E) / 16, PIECES = CH * PPR, PER = PIECES / NT, RPS = NT / PPR;
  static_assert(PIECES % NT == 0 && NT % PPR == 0, "whole rows a step");
  u32x4 v[PER];
  // base: the chunk's first token; off: row_off of this thread's first piece
  __device__ __forceinline__ void load(const E* base, int64_t stride, int nt, int off) {
    const RowBuf b = row_buf<REV>(base, stride, C, nt);
    const int step = (REV ? -1 : 1) * RPS * (int)stride * (int)sizeof(E);
#pragma unroll
    for (int k = 0; k < PER; ++k) v[k] = ld16(b, off + k * step);
  }
  static __device__ __forceinline__ int first_off(int64_t stride, int tid) {
    return row_off<REV, E>(tid / PPR, stride, tid % PPR * (16 / (int)sizeof(E)));
  }
  __device__ __forceinline__ void store(E* base, int ld, int tid) const {
    E* d = base + tid / PPR * ld + tid % PPR * (16 / (int)sizeof(E));
#pragma unroll
    for (int k = 0; k < PER; ++k) *reinterpret_cast<u32x4*>(d + k * RPS * ld) = v[k];
  }
};

// Workgroups go to the eight XCDs round-robin; this numbering gives each XCD a
// contiguous run of work items, so that the workgroups of one segment and group,
// which read the same K and Q, find them in one L2.
__device__ __forceinline__ int xcd_item() {
  const int n = gridDim.x, b = blockIdx.x, x = b & 7, per = n >> 3, rem = n & 7;
  return x * per + min(x, rem) + (b >> 3);
}

// ---------------------------------------------------------------- value sweep
// A workgroup of NW waves takes NW units of one group of heads in one segment;
// a unit is VC = 32 value columns of one head, its state Dk x 32 in the wave's
// accumulators for the whole segment.  K and Q are staged once for all waves;
// the waves of one head (a team: two, or four where a head has 128 or 256
// columns) share its decays and its chunk matrix, the tiles of which, Q K^T
// included, they form between them.  OUT = false: the state sweep (no Q, no
// output).
constexpr int VC = 32;

// Four floats at a 4-byte aligned address (a caller's state).
typedef f32x4 __attribute__((aligned(4))) f32x4_u;
__device__ __forceinline__ f32x4 ld_f32x4(const float* p) { return *reinterpret_cast<const f32x4_u*>(p); }
__device__ __forceinline__ void st_f32x4(float* p, const f32x4& v) { *reinterpret_cast<f32x4_u*>(p) = v; }

// bf16: the next chunk's K has a place of its own, so that it (and Q and V,
// whose last reads come earlier) is staged during a chunk and one barrier
// stands between chunks; in fp32 LDS does not hold it.
template <class E> constexpr int kKeyBufs = sizeof(E) == 2 ? 2 : 1;

// MP: parts of the chunk matrix and of the state in out1 (bf16; see above)
template <class E, int DK, int NW, int MP>
struct ValueLds {
  E k[kKeyBufs<E>][CH * row_ld<E>(DK)];
  E q[CH * row_ld<E>(DK)];
  E v[NW][CH * row_ld<E>(VC)];
  E m[NW / 2][10][MP][64][4];  // by team, tile, part
  ChunkDecay dec[2][NW / 2];   // of this chunk and the next
};

// Tile IDX of the head's chunk matrix: Q K^T, then the decays; in MP parts.
template <int IDX, class E, int DK, int NW, int MP>
__device__ __forceinline__ void chunk_matrix_tile(ValueLds<E, DK, NW, MP>& sh, const E* k, const ChunkDecay& dec, int team) {
  constexpr int tb = IDX >= 6 ? 3 : IDX >= 3 ? 2 : IDX >= 1 ? 1 : 0, sb = IDX - tb * (tb + 1) / 2, LDK = row_ld<E>(DK);
  const int l = lane_id(), t16 = l & 15;
  f32x4 a = zero4();
#pragma unroll
  for (int kb = 0; kb < DK / 32; ++kb)
    mma(a, ld_frag8(k, LDK, 16 * sb + t16, 32 * kb), ld_frag8(sh.q, LDK, 16 * tb + t16, 32 * kb));
  a *= tile_decay<sizeof(E) == 4>(dec, tb, sb);
#pragma unroll
  for (int q = 0; q < MP; ++q) {
    st4f<E>(sh.m[team][IDX][q][l], a);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] -= to_f(to_e<E>(a[i]));
  }
}

template <class E, int DK, int NW, bool REV, bool OUT, int MP>
__global__ __launch_bounds__(NW * 64, 2) void sweep_value_kernel(SweepParams p, int parts) {
  extern __shared__ __align__(16) char smem[];
  typedef ValueLds<E, DK, NW, MP> Lds;
  Lds* const sh0 = reinterpret_cast<Lds*>(smem);
  constexpr int LDK = row_ld<E>(DK), LDV = row_ld<E>(VC), NT = DK / 16, NTH = NW * 64;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), t16 = l & 15, g4 = l >> 4;
  const int item = xcd_item(), part = item % parts, grp = item / parts % p.G, j = item / parts / p.G;
  SegRange r;
  if (!seg_range(p.seq, p.segs, p.seg_first, j, r)) return;
  make_uniform(r);
  const bool first = REV ? r.s == r.ns - 1 : r.s == 0, last = REV ? r.s == 0 : r.s == r.ns - 1;
  if (!OUT && last) return;  // nothing follows this segment
  const int rep = p.H / p.G, upg = rep * (p.Dv / VC);
  const int unit = min(part * NW + w, upg - 1);
  const bool active = part * NW + w < upg;  // a wave without a unit repeats the last one and stores nothing
  const int h = grp * rep + unit / (p.Dv / VC), col = unit % (p.Dv / VC) * VC;
  const int team_size = NW >= 4 && p.Dv % 128 == 0 ? 4 : 2, team = w / team_size, sub = w % team_size;
  const int64_t st_off = (int64_t)DK * p.Dv;
  const float Dh = OUT && p.D ? p.D[h] : 0.f;

  // The state leaves as fp32 from the state sweep and from a sequence's last
  // segment; elsewhere only bf16 outputs read it, and two parts of the values
  // are enough.
  const int np = !OUT || (last && p.s_end) ? Parts<E>::N : min(Parts<E>::N, 2);
  const int nch = (r.len + CH - 1) / CH;
  TileStage<E, DK, NTH, REV> tk, tq;
  TileStage<E, VC, 64, REV> tv;
  const int ko = tk.first_off(p.k_stride, tid), qo = OUT ? tq.first_off(p.q_stride, tid) : 0;
  const int vo = tv.first_off(p.v_stride, l), oo = row_off<REV, E>(t16, p.H * p.Dv, 8 * g4);
  HeadConst hc;
  hc.load(p, h);
  uint32_t dt = 0;  // of the next chunk
  auto request = [&](int i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    tk.load(static_cast<const E*>(p.k) + c.base * p.k_stride + (int64_t)grp * DK, p.k_stride, c.nt, ko);
    if (OUT) tq.load(static_cast<const E*>(p.q) + c.base * p.q_stride + (int64_t)grp * DK, p.q_stride, c.nt, qo);
    tv.load(static_cast<const E*>(p.v) + c.base * p.v_stride + (int64_t)h * p.Dv + col, p.v_stride, c.nt, vo);
  };
  constexpr bool AHEAD = kKeyBufs<E> == 2;
  auto stage_q = [&] { if (OUT) tq.store(lds_opaque(sh0)->q, LDK, tid); };
  auto stage_k = [&](int i) { tk.store(lds_opaque(sh0)->k[AHEAD ? i & 1 : 0], LDK, tid); };
  auto stage_v = [&] { tv.store(lds_opaque(sh0)->v[w], LDV, l); };
  uint32_t dt0 = 0;
  if (nch > 0) {  // the first chunk's requests before the state's
    if (sub == 0) dt0 = load_dt<REV>(p, chunk_rows<REV>(r, 0), h);
    request(0);
  }
  // state tile (nt, pt), entry i: key 32 (nt / 2) + 8 g + 4 (nt % 2) + i, value
  // col + 8 a + 4 pt + b (lane 16 g + 4 a + b); in memory a lane moves four
  // values of key + b, turned over within the four lanes.
  f32x4 S[NT][2];
  const int64_t srow = (int64_t)(8 * g4 + (l & 3)) * p.Dv + col + 8 * (t16 >> 2);
  auto key0 = [&](int nt) { return 32 * (nt >> 1) + 4 * (nt & 1); };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) S[nt][pt] = zero4();
  if (OUT && p.s_in && (p.per_seg || first)) {
    const float* s0 = p.s_in + ((int64_t)(p.per_seg ? j : r.n) * p.H + h) * st_off + srow;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) S[nt][pt] = ld_f32x4(s0 + key0(nt) * p.Dv + 4 * pt);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) S[nt][pt] = quad_transpose(S[nt][pt]) * sign_of(boundary<REV>(r, nch, 0));
  }
  if (nch > 0) {
    if (sub == 0) {
      fill_decay<REV>(sh0->dec[0][team], p, hc, dt0, chunk_rows<REV>(r, 0).nt);
      if (nch > 1) dt = load_dt<REV>(p, chunk_rows<REV>(r, 1), h);
    }
    stage_k(0);
    stage_q();
    stage_v();
    if (nch > 1) request(1);
  }
  float total = 1.f;
  for (int i = 0; i < nch; ++i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    __syncthreads();  // this chunk's tiles are in place, the previous one's are read
    if (!AHEAD && i > 0) {
      stage_k(i);
      stage_q();
      stage_v();
      if (i + 1 < nch) request(i + 1);
      __syncthreads();
    }
    const int kb_ = AHEAD ? i & 1 : 0;
    const float sg = sign_of(boundary<REV>(r, nch, i));
    const uint32_t dt1 = dt;
    if (i + 2 < nch && sub == 0) dt = load_dt<REV>(p, chunk_rows<REV>(r, i + 2), h);
    // a team's first wave, once a chunk: the next chunk's decays
    auto next_decay = [&] {
      if (i + 1 < nch) fill_decay<REV>(lds_opaque(sh0)->dec[(i + 1) & 1][team], p, hc, dt1, chunk_rows<REV>(r, i + 1).nt);
    };
    Frag<E> vf[2][2];  // V down its columns: rows 32 kb.., columns of tile pt
    if (OUT) {
      {
        Lds& sh = *lds_opaque(sh0);
        const ChunkDecay& dec = sh.dec[i & 1][team];
        const E* k = sh.k[kb_];
        if (team_size == 4) {
          if (sub == 0) {
            chunk_matrix_tile<1>(sh, k, dec, team);
            next_decay();
          } else if (sub == 1) {
            chunk_matrix_tile<0>(sh, k, dec, team);
            chunk_matrix_tile<2>(sh, k, dec, team);
            chunk_matrix_tile<4>(sh, k, dec, team);
          } else if (sub == 2) {
            chunk_matrix_tile<5>(sh, k, dec, team);
            chunk_matrix_tile<9>(sh, k, dec, team);
            chunk_matrix_tile<3>(sh, k, dec, team);
          } else {
            chunk_matrix_tile<6>(sh, k, dec, team);
            chunk_matrix_tile<7>(sh, k, dec, team);
            chunk_matrix_tile<8>(sh, k, dec, team);
          }
        } else if (sub == 0) {
          chunk_matrix_tile<1>(sh, k, dec, team);
          chunk_matrix_tile<3>(sh, k, dec, team);
          chunk_matrix_tile<4>(sh, k, dec, team);
          chunk_matrix_tile<6>(sh, k, dec, team);
          next_decay();
        } else {
          chunk_matrix_tile<7>(sh, k, dec, team);
          chunk_matrix_tile<8>(sh, k, dec, team);
          chunk_matrix_tile<0>(sh, k, dec, team);
          chunk_matrix_tile<2>(sh, k, dec, team);
          chunk_matrix_tile<5>(sh, k, dec, team);
          chunk_matrix_tile<9>(sh, k, dec, team);
        }
      }
      f32x4 o[4][2];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) o[tb][0] = o[tb][1] = zero4();
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb) {
        sched_fence();
        Lds& sh = *lds_opaque(sh0);
        PFrag<E> sf[2];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) sf[pt] = PFrag<E>(Frag<float>{S[2 * kb][pt], S[2 * kb + 1][pt]});
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const Frag<E> q = ld_frag8(sh.q, LDK, 16 * tb + t16, 32 * kb);
          if constexpr (MP == 2) {
            mma_hi_lo(o[tb][0], sf[0], q);
            mma_hi_lo(o[tb][1], sf[1], q);
          } else {
            mma(o[tb][0], e_part(sf[0]), q);
            mma(o[tb][1], e_part(sf[1]), q);
          }
        }
      }
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) vf[kb][pt] = ld_col(lds_opaque(sh0)->v[w], LDV, 32 * kb, 0, pt);
      __syncthreads();
      if (AHEAD && i + 1 < nch) {  // Q has been read, the other K buffer is free
        stage_q();
        stage_k(i + 1);
      }
      const RowBuf out = row_buf<REV>(static_cast<const E*>(p.out1) + c.base * p.H * p.Dv + (int64_t)h * p.Dv + col,
                                      p.H * p.Dv, VC, c.nt, active);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        sched_fence();
        Lds& sh = *lds_opaque(sh0);
        const ChunkDecay& dec = sh.dec[i & 1][team];
        const float tf = dec.tf[16 * tb + t16] * sg;
        o[tb][0] *= tf;
        o[tb][1] *= tf;
#pragma unroll
        for (int kb = 0; kb <= tb / 2; ++kb) {
          const int i0 = tb * (tb + 1) / 2 + 2 * kb;
#pragma unroll
          for (int q = MP - 1; q >= 0; --q) {
            Frag<E> m;
            if constexpr (sizeof(E) == 2) {
              const bf16x4 x = *reinterpret_cast<const bf16x4*>(sh.m[team][i0][q][l]);
              bf16x4 y = bf16x4{};
              if (2 * kb + 1 <= tb) y = *reinterpret_cast<const bf16x4*>(sh.m[team][i0 + (2 * kb + 1 <= tb)][q][l]);
              m.v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
              m.lo = *reinterpret_cast<const f32x4*>(sh.m[team][i0][q][l]);
              m.hi = 2 * kb + 1 <= tb ? *reinterpret_cast<const f32x4*>(sh.m[team][i0 + (2 * kb + 1 <= tb)][q][l]) : zero4();
            }
            mma(o[tb][0], vf[kb][0], m);
            mma(o[tb][1], vf[kb][1], m);
          }
        }
        const int row = 16 * tb + t16;
        const E* vr = sh.v[w] + row * LDV + 8 * g4;
        f32x4 y0 = o[tb][0], y1 = o[tb][1];
        if (REV) {  // forwards the target weight is 1
          const float tw = dec.tw[row];
          y0 *= tw;
          y1 *= tw;
        }
        y0 += ld4f<E>(vr) * Dh;
        y1 += ld4f<E>(vr + 4) * Dh;
        const int off = oo + (REV ? -tb : tb) * 16 * p.H * p.Dv * (int)sizeof(E);
        if constexpr (sizeof(E) == 2) {
          Frag<bf16> f;
          pack_frag(f, y0, y1);
          st16(out, off, f.v);
        } else {
          st16(out, off, y0);
          st16(out, off + 16, y1);
        }
      }
    } else {
      if (sub == 0) next_decay();
      if (AHEAD && i + 1 < nch) stage_k(i + 1);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) vf[kb][pt] = ld_col(lds_opaque(sh0)->v[w], LDV, 32 * kb, 0, pt);
    }
    if (AHEAD && i + 1 < nch) {
      stage_v();  // (the wave's own)
      if (i + 2 < nch) request(i + 2);
    }
    sched_fence();
    // S' = exp(tot) S + K^T (end V)
    const ChunkDecay& dec = lds_opaque(sh0)->dec[i & 1][team];
    const float tot = -dec.btw[3];
    if (!OUT) total *= -tot;
    Parts<E> vp[2][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const f32x4 e0 = *reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 4 * g4]) * -sg;
      const f32x4 e1 = *reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 16 + 4 * g4]) * -sg;
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) {
        f32x4 lo, hi;
        frag_f32(vf[kb][pt], lo, hi);
        if (np == Parts<E>::N) split(vp[kb][pt], lo * e0, hi * e1);
        else split2(vp[kb][pt], lo * e0, hi * e1);
      }
    }
#pragma unroll
    for (int n2 = 0; n2 < NT; n2 += 2) {  // four accumulator chains at a time
      sched_fence();
      Lds& sh = *lds_opaque(sh0);
      Frag<E> kf[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        S[n2 + e][0] *= tot;
        S[n2 + e][1] *= tot;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) kf[e][kb] = ld_col(sh.k[kb_], LDK, 32 * kb, 16 * n2, e);
      }
#pragma unroll
      for (int q = Parts<E>::N - 1; q >= 0; --q) {
        if (q >= np) continue;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mma(S[n2 + e][0], kf[e][kb], vp[kb][0].p[q]);
            mma(S[n2 + e][1], kf[e][kb], vp[kb][1].p[q]);
          }
      }
    }
  }
  float* dst = OUT ? (last ? p.s_end : nullptr) : p.s_loc;
  if (!dst || !active) return;
  dst += ((int64_t)(OUT ? r.n : j) * p.H + h) * st_off + srow;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) st_f32x4(dst + key0(nt) * p.Dv + 4 * pt, quad_transpose(S[nt][pt] * sign_of(boundary<REV>(r, nch, nch))));
  if (!OUT && l == 0 && col == 0) p.s_dec[(int64_t)j * p.H + h] = total;
}

// ---------------------------------------------------------------- key sweep
// A workgroup of Dk / 16 waves takes HS slices of PS = 64 value columns of one
// group of heads in one segment.  Wave nt owns 16 keys of all slices' states
// (transposed: values down, keys across), so that the sum of out2 over the
// slices stays in its accumulators; a slice's chunk matrix W V^T is formed tile
// by tile over the waves, decayed and summed over the slices in LDS before the
// one product with K.  out2 leaves as one fp32 part per workgroup, or, where one
// workgroup has all of a group's slices, as dC (dB) itself (two launches fewer:
// 3,392 tokens of 4 heads of 64 x 64 with a B and C each, fp32, both ways: 155 -> 143 us of kernels).
template <class E, int DK, int HS>
struct KeyLds {
  E k[CH * row_ld<E>(DK)];
  E q[CH * row_ld<E>(DK)];
  E v[HS][CH * row_ld<E>(PS)];
  E w[HS][CH * row_ld<E>(PS)];
  f32x4 z[10][64];               // sum over slices of the decayed chunk matrix, by tile and lane
  float rti[10][HS][16];         // row terms of the chunk itself, by tile and target row
  float cti[10][HS][16];         // forwards: the same pairs' sums by source row
  float rtx[DK / 16][HS][CH];    // row terms of the state, by key tile
  double anc[DK / 16][4][HS];    // <state, its gradient>, by key tile and lane group
  ChunkDecay dec[2][HS];         // of this chunk and the next
};

template <class E, int DK, int HS, bool REV>
__global__ __launch_bounds__(DK * 4) void sweep_key_kernel(SweepParams p, int parts) {
  extern __shared__ __align__(16) char smem[];
  typedef KeyLds<E, DK, HS> Lds;
  Lds* const sh0 = reinterpret_cast<Lds*>(smem);
  constexpr int LDK = row_ld<E>(DK), LDV = row_ld<E>(PS), NW = DK / 16, NTH = DK * 4;
  const int tid = threadIdx.x, nt = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), t16 = l & 15, g4 = l >> 4;
  const int item = xcd_item(), part = item % parts, grp = item / parts % p.G, j = item / parts / p.G;
  SegRange r;
  if (!seg_range(p.seq, p.segs, p.seg_first, j, r)) return;
  make_uniform(r);
  const bool first = REV ? r.s == r.ns - 1 : r.s == 0;
  const int rep = p.H / p.G, spg = rep * (p.Dv / PS), spv = p.Dv / PS;
  const int64_t st_off = (int64_t)DK * p.Dv;
  const int ns = min(HS, spg - part * HS);       // slices of this workgroup
  auto slice_of = [&](int s) { return grp * spg + part * HS + min(s, ns - 1); };  // over all heads
  // key of a lane's column (as the state's column) and of its rows (as out2's)
  const int kcol = 32 * (nt >> 1) + 8 * (t16 >> 2) + 4 * (nt & 1) + (t16 & 3);
  const int krow = 32 * (nt >> 1) + 8 * g4 + 4 * (nt & 1);

  const int nch = (r.len + CH - 1) / CH;
  const int nsl = p.H * spv;  // slices of all heads
  const int64_t chunk0 = p.seq.first_chunk(p.chunk_first, r.n) + r.c0;  // the segment's first, over all sequences
  // the state at the end of the segment's chunk ci: [tile of 16 keys][pt][lane] per slice
  auto dump_of = [&](int ci, int s) {
    return reinterpret_cast<f32x4*>(p.dump) + (((chunk0 + ci) * nsl + slice_of(s)) * NW + nt) * 256 + l;
  };
  TileStage<E, DK, NTH, REV> tk, tq;
  TileStage<E, PS, NTH, REV> tv[HS], tw[HS];
  static_assert(HS <= NW, "one wave a slice forms its decays");
  const int ko = tk.first_off(p.k_stride, tid), qo = tq.first_off(p.q_stride, tid);
  const int vo = tv[0].first_off(p.v_stride, tid), wo = tw[0].first_off(p.w_stride, tid);
  const int oo = row_off<REV, float>(t16, DK, krow);
  // heads of the slices: their decays are formed by one wave each, of eight waves
  // first the last two, which have the least of the chunk matrix
  const int head0 = slice_of(0) / spv, nheads = slice_of(ns - 1) / spv - head0 + 1;
  auto head_of = [&](int s) { return slice_of(s) / spv - head0; };
  const int dw = NW == 8 ? (nt >= 6 ? nt - 6 : nt >= 4 ? HS : 5 - nt) : nt;
  const int ds = dw < nheads ? dw : -1, dh = head0 + max(ds, 0);
  HeadConst hc;
  hc.load(p, dh);
  uint32_t dt = 0;  // of the next chunk
  auto request = [&](int i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    tk.load(static_cast<const E*>(p.k) + c.base * p.k_stride + (int64_t)grp * DK, p.k_stride, c.nt, ko);
    tq.load(static_cast<const E*>(p.q) + c.base * p.q_stride + (int64_t)grp * DK, p.q_stride, c.nt, qo);
#pragma unroll
    for (int s = 0; s < HS; ++s) {
      tv[s].load(static_cast<const E*>(p.v) + c.base * p.v_stride + (int64_t)slice_of(s) * PS, p.v_stride, c.nt, vo);
      tw[s].load(static_cast<const E*>(p.w) + c.base * p.w_stride + (int64_t)slice_of(s) * PS, p.w_stride, c.nt, wo);
    }
  };
  auto stage = [&] {
    Lds& sh = *lds_opaque(sh0);
    tk.store(sh.k, LDK, tid);
    tq.store(sh.q, LDK, tid);
#pragma unroll
    for (int s = 0; s < HS; ++s) {
      tv[s].store(sh.v[s], LDV, tid);
      tw[s].store(sh.w[s], LDV, tid);
    }
  };
  uint32_t dt0 = 0;
  if (nch > 0) {  // the first chunk's requests before the state's
    if (ds >= 0) dt0 = load_dt<REV>(p, chunk_rows<REV>(r, 0), dh);
    request(0);
  }
  // state tile pt of slice s, entry i: value 32 (pt / 2) + 8 g + 4 (pt % 2) + i, key kcol
  f32x4 T[HS][4];
#pragma unroll
  for (int s = 0; s < HS; ++s) {
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) T[s][pt] = zero4();
    if (s < ns && p.s_in && (p.per_seg || first)) {
      const int sl = slice_of(s);
      const float* s0 = p.s_in + ((int64_t)(p.per_seg ? j : r.n) * p.H + sl / spv) * st_off + (int64_t)kcol * p.Dv + sl % spv * PS;
#pragma unroll
      for (int pt = 0; pt < 4; ++pt)
        T[s][pt] = ld_f32x4(s0 + 32 * (pt >> 1) + 8 * g4 + 4 * (pt & 1)) * sign_of(boundary<REV>(r, nch, 0));
    }
  }
  if (nch > 0) {
    if (ds >= 0) {
      fill_decay<REV>(sh0->dec[0][ds], p, hc, dt0, chunk_rows<REV>(r, 0).nt);
      if (nch > 1) dt = load_dt<REV>(p, chunk_rows<REV>(r, 1), dh);
    }
    stage();
    if (nch > 1) request(1);
  }
  for (int i = 0; i < nch; ++i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    const int ci = REV ? nch - 1 - i : i;  // chunk within the segment
    const float sg = sign_of(boundary<REV>(r, nch, i));
    // backwards: the state entering the chunk is the gradient of the state at its end
    f32x4 dump[4];  // of the next slice
    auto request_dump = [&](int s) {
      const f32x4* d = dump_of(ci, s);
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) dump[pt] = __builtin_nontemporal_load(d + pt * 64);
    };
    if (REV) request_dump(0);
    __syncthreads();  // this chunk's tiles and decays are in place
    // the chunk's own part: tiles of (rows s, columns t), the diagonal ones, which
    // cost more, on the first four waves; of eight waves the others take the rest
    // and the next chunk's decays
    for (int n = nt; n < 10; n += NW == 8 && n < 4 ? 10 : 4) {
      Lds& sh = *lds_opaque(sh0);
      const int idx = n == 0 ? 0 : n == 1 ? 2 : n == 2 ? 5 : n == 3 ? 9 : n == 4 ? 1 : n < 7 ? n - 2 : n - 1;
      int tb, sb;
      tri_tile(idx, tb, sb);
      f32x4 cb = zero4(), zs = zero4(), f = zero4();  // f: the decays of the current slice's head
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb)
        mma(cb, ld_frag8(sh.k, LDK, 16 * sb + t16, 32 * kb), ld_frag8(sh.q, LDK, 16 * tb + t16, 32 * kb));
      const int row = 16 * tb + t16;
      const bool live = row < c.nt;
      const int64_t grow = live ? row_of<REV>(c, row) : 0;
      if (p.cb && tb == sb && part == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * g4 + e == t16 && live) p.cb[(int64_t)grp * p.tokens + grow] = cb[e];
      }
      float rts[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < HS; ++s) {
        if (s == 2) sched_fence();
        Lds& sh = *lds_opaque(sh0);
        f32x4 x = zero4();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
          mma(x, ld_frag8(sh.v[s], LDV, 16 * sb + t16, 32 * kb), ld_frag8(sh.w[s], LDV, 16 * tb + t16, 32 * kb));
        if (p.xd && tb == sb && s < ns) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (4 * g4 + e == t16 && live) p.xd[(int64_t)slice_of(s) * p.tokens + grow] = x[e];
        }
        if (s == 0 || slice_of(s) % spv == 0) f = tile_decay<true>(sh.dec[i & 1][head_of(s)], tb, sb);
        const f32x4 z = x * f;
        f32x4 pair = z * cb;  // of source row 4g + e and target row t16, other than itself
        if (sb == tb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) pair[e] = 4 * g4 + e < t16 ? pair[e] : 0.f;
        }
        rts[s] = (pair[0] + pair[1]) + (pair[2] + pair[3]);
        if (!REV) {
          const float own = row16_sum4(pair);  // source row 4g + t16 % 4
          if (t16 < 4) sh.cti[idx][s][4 * g4 + t16] = own;
        }
        if (s < ns) zs += z * sh.dec[i & 1][head_of(s)].tw[row];
      }
      const float rt = sum_groups4(rts);  // slice g
      if (g4 < HS) sh.rti[idx][g4][t16] = rt;
      sh.z[idx][l] = zs;
    }
    if (ds >= 0 && i + 1 < nch)
      fill_decay<REV>(lds_opaque(sh0)->dec[(i + 1) & 1][ds], p, hc, dt, chunk_rows<REV>(r, i + 1).nt);
    __syncthreads();
    Frag<E> kf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) kf[kb] = ld_col(lds_opaque(sh0)->k, LDK, 32 * kb, 32 * (nt >> 1), nt & 1);
    // K times its decay to the chunk's end, of the current slice's head (backwards,
    // with the anchors' registers, formed for every slice instead of held)
    Parts<E> kp[2];
    f32x4 o[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      if (tb > 1) sched_fence();
      Lds& sh = *lds_opaque(sh0);
      o[tb] = zero4();
#pragma unroll
      for (int kb = 0; kb <= tb / 2; ++kb) {
        const int i0 = tb * (tb + 1) / 2 + 2 * kb;
        PFrag<E> z(Frag<float>{sh.z[i0][l], 2 * kb + 1 <= tb ? sh.z[2 * kb + 1 <= tb ? i0 + 1 : i0][l] : zero4()});
        mma_hi_lo(o[tb], kf[kb], z);
      }
    }
#pragma unroll
    for (int s = 0; s < HS; ++s) {
      if (s >= ns) break;
      sched_fence();
      if (REV) {  // <state at the chunk's end, its gradient>, this lane's part
        double a = 0.;
#pragma unroll
        for (int pt = 0; pt < 4; ++pt)
#pragma unroll
          for (int e = 0; e < 4; ++e) a += (double)dump[pt][e] * T[s][pt][e];
        a = row16_sum_d(a);
        if (t16 == 0) lds_opaque(sh0)->anc[nt][g4][s] = sg * a;
        if (s + 1 < ns) request_dump(s + 1);
      }
      // u = W T^T of the state before the chunk, four row blocks side by side
      f32x4 u[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) u[tb] = zero4();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Lds& sh = *lds_opaque(sh0);
        Frag<E> wf[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) wf[tb] = ld_frag8(sh.w[s], LDV, 16 * tb + t16, 32 * kb);
        Parts<E> tp;
        split(tp, T[s][2 * kb], T[s][2 * kb + 1]);
#pragma unroll
        for (int q = Parts<E>::N - 1; q >= 0; --q)
#pragma unroll
          for (int tb = 0; tb < 4; ++tb) mma(u[tb], tp.p[q], wf[tb]);
      }
      sched_fence();
      Lds& sh = *lds_opaque(sh0);
      const ChunkDecay& dec = sh.dec[i & 1][head_of(s)];
      float rts[4];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int row = 16 * tb + t16;
        const float tf = dec.tf[row];
        const f32x4 q4 = ld4f<E>(sh.q + row * LDK + krow);
        rts[tb] = (sg * tf) * ((u[tb][0] * q4[0] + u[tb][1] * q4[1]) + (u[tb][2] * q4[2] + u[tb][3] * q4[3]));
        o[tb] += u[tb] * (sg * (REV ? tf * dec.tw[row] : tf));  // forwards the target weight is 1
      }
      sh.rtx[nt][s][l] = sum_groups4(rts);  // block g: row l
      // T' = exp(tot) T + V^T (end K)
      if (REV || s == 0 || slice_of(s) % spv == 0) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          f32x4 lo, hi;
          frag_f32(ld_col(sh.k, LDK, 32 * kb, 32 * (nt >> 1), nt & 1), lo, hi);
          split(kp[kb], lo * (*reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 4 * g4]) * -sg),
                hi * (*reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 16 + 4 * g4]) * -sg));
        }
      }
      const float tot = -dec.btw[3];
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) T[s][pt] *= tot;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        Frag<E> vf[4];
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) vf[pt] = ld_col(sh.v[s], LDV, 32 * kb, 32 * (pt >> 1), pt & 1);
#pragma unroll
        for (int q = Parts<E>::N - 1; q >= 0; --q)
#pragma unroll
          for (int pt = 0; pt < 4; ++pt) mma(T[s][pt], vf[pt], kp[kb].p[q]);
      }
    }
    __syncthreads();  // the chunk's tiles are read, its row terms are in place
    // The next chunk's tiles into LDS and the requests of the one after it come
    // before this chunk's stores: the wait for a requested tile covers every
    // older store.
    if (i + 1 < nch) stage();
    if (i + 2 < nch) {
      if (ds >= 0) dt = load_dt<REV>(p, chunk_rows<REV>(r, i + 2), dh);
      request(i + 2);
    }
    if (parts == 1) {  // the whole group's sum: dC or dB itself
      const int64_t gs = (int64_t)p.G * DK;
      const RowBuf out = row_buf<REV>(static_cast<E*>(p.out2_whole) + c.base * gs + grp * DK, gs, DK, c.nt);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) st_row4(out, row_off<REV, E>(16 * tb + t16, gs, krow), o[tb], (E*)nullptr);
    } else {
      const RowBuf out = row_buf<REV>(p.out2 + ((int64_t)(grp * parts + part) * p.tokens + c.base) * DK, DK, DK, c.nt);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) st16(out, oo + (REV ? -tb : tb) * 16 * DK * 4, o[tb]);
    }
    if (!REV) {
#pragma unroll
      for (int s = 0; s < HS; ++s)
        if (s < ns) {
          f32x4* d = dump_of(ci, s);
#pragma unroll
          for (int pt = 0; pt < 4; ++pt) __builtin_nontemporal_store(T[s][pt] * -sg, d + pt * 64);
        }
    }
    Lds& sh = *lds_opaque(sh0);
    if (REV && tid < ns) {
      double a = 0.;
      for (int n = 0; n < NW; ++n)
        for (int g = 0; g < 4; ++g) a += sh.anc[n][g][tid];
      p.anchor[(chunk0 + ci) * nsl + slice_of(tid)] = a;
    }
    for (int k = tid; k < ns * CH; k += NTH) {
      const int s = k / CH, row = k % CH;
      const int blk = row / 16, r16 = row % 16;
      double own = 0., state = 0.;
#pragma unroll
      for (int sb = 0; sb < 4; ++sb) {
        const float v = sh.rti[blk * (blk + 1) / 2 + min(sb, blk)][s][r16];
        own += sb <= blk ? v : 0.f;
      }
#pragma unroll
      for (int n = 0; n < NW; ++n) state += sh.rtx[n][s][row];
      if (row < c.nt) {
        const int64_t at = (int64_t)slice_of(s) * p.tokens + row_of<REV>(c, row);
        p.rt[at] = (float)(own + state);
        if (!REV) {
          state = 0.;
#pragma unroll
          for (int tb = 0; tb < 4; ++tb) {
            const int hi = max(tb, blk);
            const float v = sh.cti[hi * (hi + 1) / 2 + blk][s][r16];
            state += tb >= blk ? v : 0.f;
          }
        }
        p.rt2[at] = (float)state;
      }
    }
  }
}

template <class E, int DK, int NW, bool REV, bool OUT, int MP>
hipError_t value_launch_parts(const SweepParams& p, int nseg, hipStream_t st) {
  const int upg = p.H / p.G * (p.Dv / VC), parts = (upg + NW - 1) / NW;
  constexpr size_t lds = sizeof(ValueLds<E, DK, NW, MP>);
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&sweep_value_kernel<E, DK, NW, REV, OUT, MP>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sweep_value_kernel<E, DK, NW, REV, OUT, MP>), dim3(nseg * p.G * parts), dim3(NW * 64), lds, st, p, parts);
  return hipGetLastError();
}
template <class E, int DK, int NW, bool REV, bool OUT>
hipError_t value_launch(const SweepParams& p, int nseg, hipStream_t st) {
  if constexpr (OUT && sizeof(E) == 2)
    if (p.round_once) return value_launch_parts<E, DK, NW, REV, OUT, 2>(p, nseg, st);
  return value_launch_parts<E, DK, NW, REV, OUT, 1>(p, nseg, st);
}
// Waves of a value sweep's workgroup: as many units as the group has, up to
// eight (fp32: four, by LDS).
int value_waves(int dtype, int upg) { return upg >= 8 && dtype == GDN_BF16 ? 8 : upg >= 4 ? 4 : 2; }
template <class E, int DK, bool REV, bool OUT>
hipError_t value_nw(const SweepParams& p, int nseg, hipStream_t st) {
  const int nw = value_waves(sizeof(E) == 2 ? GDN_BF16 : GDN_F32, p.H / p.G * (p.Dv / VC));
  if (nw == 8) return value_launch<E, DK, sizeof(E) == 2 ? 8 : 4, REV, OUT>(p, nseg, st);
  if (nw == 4) return value_launch<E, DK, 4, REV, OUT>(p, nseg, st);
  return value_launch<E, DK, 2, REV, OUT>(p, nseg, st);
}

template <class E, int DK, int HS, bool REV>
hipError_t key_launch(const SweepParams& p, int nseg, hipStream_t st) {
  const int spg = p.H / p.G * (p.Dv / PS), parts = (spg + HS - 1) / HS;
  constexpr size_t lds = sizeof(KeyLds<E, DK, HS>);
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&sweep_key_kernel<E, DK, HS, REV>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sweep_key_kernel<E, DK, HS, REV>), dim3(nseg * p.G * parts), dim3(DK * 4), lds, st, p, parts);
  return hipGetLastError();
}
// Slices of a key sweep's workgroup: as many as the group has, up to what LDS holds.
int key_slices(int dtype, int spg) { return spg >= 3 && dtype == GDN_BF16 ? 4 : spg >= 2 ? 2 : 1; }

template <class E, int DK, bool REV>
hipError_t sweep_any(int mode, const SweepParams& p, int nseg, hipStream_t st) {
  if (mode == SWEEP_VALUE) return value_nw<E, DK, REV, true>(p, nseg, st);
  if (mode == SWEEP_STATE) return value_nw<E, DK, REV, false>(p, nseg, st);
  const int hs = key_slices(sizeof(E) == 2 ? GDN_BF16 : GDN_F32, p.H / p.G * (p.Dv / PS));
  if (hs == 4) return key_launch<E, DK, sizeof(E) == 2 ? 4 : 2, REV>(p, nseg, st);
  if (hs == 2) return key_launch<E, DK, 2, REV>(p, nseg, st);
  return key_launch<E, DK, 1, REV>(p, nseg, st);
}
template <class E>
hipError_t sweep_e(int rev, int mode, const SweepParams& p, int nseg, hipStream_t st) {
  if (p.Dk == 64) return rev ? sweep_any<E, 64, true>(mode, p, nseg, st) : sweep_any<E, 64, false>(mode, p, nseg, st);
  if (p.Dk == 128) return rev ? sweep_any<E, 128, true>(mode, p, nseg, st) : sweep_any<E, 128, false>(mode, p, nseg, st);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_sweep(int dtype, int rev, int mode, const SweepParams& p, int nseg, hipStream_t st) {
  return dtype == GDN_BF16 ? sweep_e<bf16>(rev, mode, p, nseg, st) : sweep_e<float>(rev, mode, p, nseg, st);
}
int sweep_parts_per_group(int dtype, int H, int G, int Dv) {
  const int spg = H / G * (Dv / PS), hs = key_slices(dtype, spg);
  return (spg + hs - 1) / hs;
}
int sweep_workgroups(int dtype, int H, int G, int Dv) {
  const int upg = H / G * (Dv / VC), nw = value_waves(dtype, upg);
  return G * max((upg + nw - 1) / nw, sweep_parts_per_group(dtype, H, G, Dv));
}

}  // namespace gdn
