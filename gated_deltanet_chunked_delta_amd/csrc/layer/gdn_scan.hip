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
// it restarts every AB chunks from <h, dh> there: the forward key sweep leaves
// its state at those places and the backward one takes the product; what the
// sums miss the next place's product by is spread over the tokens between.  Then
// dD_t = ct_t + (C_t . B_t)(x_t . dy_t) + A da_t.
//
// Precision.  Products of bf16 inputs are exact and summed in fp32.  An fp32
// factor (the state, keys or values times their decay) enters a product as
// three bf16 parts, 24 bits in all, wherever its rounding would reach an fp32
// result: the states, and the row terms rt, ct behind dA and ddt.  Where only a
// bf16 output depends on it, it is rounded to bf16 once in out1 (the chunk matrix
// and the state: together an error like the output's own rounding) and enters
// out2 in two parts (the chunk matrix; a few products a wave).  fp32 inputs take the fp32 matrix instructions throughout.
//
// Decay factors are products of factors <= 1 over 16-row blocks (a power of a
// sum inside a block, a factor for the blocks between), so that no difference
// of long sums is formed and only the four diagonal blocks need one per entry.
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

// a times a value held in two parts (about 16 bits of it).
__device__ __forceinline__ void mma_hi_lo(f32x4& acc, const Frag<bf16>& a, const PFrag<bf16>& b) {
  mma(acc, a, b.lo);
  mma(acc, a, b.hi);
}
__device__ __forceinline__ void mma_hi_lo(f32x4& acc, const Frag<float>& a, const PFrag<float>& b) { mma(acc, a, b.f); }

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
template <bool REV>
__device__ __forceinline__ int64_t row_of(const ChunkRows& c, int r) { return c.base + (REV ? c.nt - 1 - r : r); }
// Chunk i of a segment in sweep order.
template <bool REV>
__device__ __forceinline__ ChunkRows chunk_rows(const SegRange& s, int i) {
  const int nch = (s.len + CH - 1) / CH, c = REV ? nch - 1 - i : i;
  ChunkRows r;
  r.base = s.row0 + (int64_t)c * CH;
  r.nt = min(CH, s.len - c * CH);
  return r;
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
template <bool REV, class P>
__device__ __forceinline__ float load_dt(const P& p, const ChunkRows& c, int h) {
  const int r = lane_id();
  return r < c.nt ? scan_dt_raw(p.dt, p.dt_f32, row_of<REV>(c, r) * p.dt_stride + h) : 0.f;
}
template <bool REV, class P>
__device__ __forceinline__ void fill_decay(ChunkDecay& o, const P& p, const HeadConst& hc, float raw, int nt) {
  const int r = lane_id();
  raw += hc.bias;
  const float d = r < nt ? (p.softplus ? scan_softplus(raw) : raw) : 0.f;
  const double a = (double)d * hc.A * 1.4426950408889634;
  double step = a;
  if (REV) {
    step = __shfl_up(a, 1, 64);
    if (r == 0) step = 0.;
  }
  const int q = r & 15;
  double pre = step;   // inclusive prefix in the 16-row block
  double suf = step;   // inclusive suffix
#pragma unroll
  for (int o2 = 1; o2 < 16; o2 <<= 1) {
    const double y = __shfl_up(pre, o2, 16), z = __shfl_down(suf, o2, 16);
    if (q >= o2) pre += y;
    if (q + o2 < 16) suf += z;
  }
  double after = __shfl_down(suf, 1, 16);
  if (q == 15) after = 0.;
  const double b0 = __shfl(pre, 15, 64), b1 = __shfl(pre, 31, 64), b2 = __shfl(pre, 47, 64), b3 = __shfl(pre, 63, 64);
  const double fin = REV ? __shfl(a, 63, 64) : 0.;
  const int blk = r >> 4;
  const double before = blk == 0 ? 0. : blk == 1 ? b0 : blk == 2 ? b0 + b1 : b0 + b1 + b2;
  const double later = (blk == 0 ? b1 + b2 + b3 : blk == 1 ? b2 + b3 : blk == 2 ? b3 : 0.) + fin;
  const float w = r < nt ? 1.f : 0.f;
  o.p16[r] = pre;
  o.sw[r] = REV ? w : d;
  o.tw[r] = REV ? d : w;
  o.tf[r] = exp2_sum(before + pre);
  o.row[r] = exp2_sum(pre);
  o.col[r] = exp2_sum(after) * (REV ? w : d);
  o.end[r] = exp2_sum(after + later) * (REV ? w : d);
  if (r < 4) {
    const double t = r == 0 ? b1 : r == 1 ? b2 : r == 2 ? b1 + b2 : b0 + b1 + b2 + b3 + fin;
    o.btw[r] = exp2_sum(t);
  }
}
// The factors L o sw of tile (tb, sb) for this lane's entries (s = 4g + i, t = lane % 16).
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
    for (int i = 0; i < 4; ++i) f[i] = 4 * g + i <= t ? exp2_sum(pt - ps[i]) * sw[i] : 0.f;
  }
  return f;
}

// ---------------------------------------------------------------- staging
// A chunk's [CH][C] tile from global rows into registers, then into LDS, by NT
// threads; rows past the end are zero.
template <class E, int C, int NT>
struct TileStage {
  typedef uint32_t u32x4 __attribute__((__vector_size__(16)));
  static constexpr int PPR = C * (int)sizeof(E) / 16, PIECES = CH * PPR, PER = (PIECES + NT - 1) / NT;
  u32x4 v[PER];
  template <bool REV>
  __device__ __forceinline__ void load(const E* base, int64_t stride, const ChunkRows& c, int tid) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = tid + k * NT, r = i / PPR, pc = i % PPR;
      v[k] = u32x4{0, 0, 0, 0};
      if (r < c.nt) v[k] = *reinterpret_cast<const u32x4*>(base + row_of<REV>(c, r) * stride + pc * (16 / (int)sizeof(E)));
    }
  }
  __device__ __forceinline__ void store(E* lds, int ld, int tid) const {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = tid + k * NT, r = i / PPR, pc = i % PPR;
      if (PIECES % NT == 0 || i < PIECES) *reinterpret_cast<u32x4*>(lds + r * ld + pc * (16 / (int)sizeof(E))) = v[k];
    }
  }
};

// ---------------------------------------------------------------- value sweep
// A workgroup of NW waves takes NW units of one group of heads in one segment;
// a unit is VC = 32 value columns of one head, its state Dk x 32 in the wave's
// accumulators for the whole segment.  K and Q are staged once for all waves,
// and Q K^T, which has no head in it, is formed once by all waves together.
// OUT = false: the state sweep (no Q, no output).
constexpr int VC = 32;

template <class E, int DK, int NW>
struct ValueLds {
  E k[CH * row_ld<E>(DK)];
  E q[CH * row_ld<E>(DK)];
  E v[NW][CH * row_ld<E>(VC)];
  f32x4 cb[10][64];
  ChunkDecay dec[NW];
};

template <class E, int DK, int NW, bool REV, bool OUT>
__global__ __launch_bounds__(NW * 64) void sweep_value_kernel(SweepParams p, int parts) {
  extern __shared__ __align__(16) char smem[];
  typedef ValueLds<E, DK, NW> Lds;
  Lds* const sh0 = reinterpret_cast<Lds*>(smem);
  constexpr int LDK = row_ld<E>(DK), LDV = row_ld<E>(VC), NT = DK / 16, NTH = NW * 64;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), t16 = l & 15, g4 = l >> 4;
  const int part = blockIdx.x % parts, grp = blockIdx.x / parts % p.G, j = blockIdx.x / parts / p.G;
  SegRange r;
  if (!seg_range(p.seq, p.segs, p.seg_first, j, r)) return;
  const bool first = REV ? r.s == r.ns - 1 : r.s == 0, last = REV ? r.s == 0 : r.s == r.ns - 1;
  if (!OUT && last) return;  // nothing follows this segment
  const int rep = p.H / p.G, upg = rep * (p.Dv / VC);
  const int unit = min(part * NW + w, upg - 1);
  const bool active = part * NW + w < upg;  // a wave without a unit repeats the last one and stores nothing
  const int h = grp * rep + unit / (p.Dv / VC), col = unit % (p.Dv / VC) * VC;
  const int64_t st_off = (int64_t)DK * p.Dv;
  const float Dh = OUT && p.D ? p.D[h] : 0.f;

  // state tile (nt, pt), entry i: key 32 (nt / 2) + 8 g + 4 (nt % 2) + i, value col + 8 a + 4 pt + b (lane 16 g + 4 a + b)
  f32x4 S[NT][2];
  const int vcol = col + 8 * (t16 >> 2) + (t16 & 3);
  auto key_of = [&](int nt) { return 32 * (nt >> 1) + 8 * g4 + 4 * (nt & 1); };
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt) S[nt][pt] = zero4();
  if (OUT && p.s_in && (p.per_seg || first)) {
    const float* s0 = p.s_in + ((int64_t)(p.per_seg ? j : r.n) * p.H + h) * st_off + vcol;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[nt][pt][i] = s0[(int64_t)(key_of(nt) + i) * p.Dv + 4 * pt];
  }
  const int nch = (r.len + CH - 1) / CH;
  TileStage<E, DK, NTH> tk, tq;
  TileStage<E, VC, 64> tv;
  HeadConst hc;
  hc.load(p, h);
  float dt = 0.f;
  auto request = [&](int i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    dt = load_dt<REV>(p, c, h);
    tk.template load<REV>(static_cast<const E*>(p.k) + (int64_t)grp * DK, p.k_stride, c, tid);
    if (OUT) tq.template load<REV>(static_cast<const E*>(p.q) + (int64_t)grp * DK, p.q_stride, c, tid);
    tv.template load<REV>(static_cast<const E*>(p.v) + (int64_t)h * p.Dv + col, p.v_stride, c, l);
  };
  if (nch > 0) request(0);
  float total = 1.f;
  for (int i = 0; i < nch; ++i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    __syncthreads();  // the previous chunk's reads are done
    {
      Lds& sh = *lds_opaque(sh0);
      tk.store(sh.k, LDK, tid);
      if (OUT) tq.store(sh.q, LDK, tid);
      tv.store(sh.v[w], LDV, l);
    }
    const float raw = dt;
    if (i + 1 < nch) request(i + 1);
    fill_decay<REV>(lds_opaque(sh0)->dec[w], p, hc, raw, c.nt);
    __syncthreads();
    if (OUT) {
      Lds& sh = *lds_opaque(sh0);
      for (int idx = w; idx < 10; idx += NW) {
        int tb, sb;
        tri_tile(idx, tb, sb);
        f32x4 a = zero4();
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb)
          mma(a, ld_frag8(sh.k, LDK, 16 * sb + t16, 32 * kb), ld_frag8(sh.q, LDK, 16 * tb + t16, 32 * kb));
        sh.cb[idx][l] = a;
      }
    }
    Frag<E> vf[2][2];  // V down its columns: rows 32 kb.., columns of tile pt
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) vf[kb][pt] = ld_col(lds_opaque(sh0)->v[w], LDV, 32 * kb, 0, pt);
    if (OUT) {
      f32x4 o[4][2];
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) o[tb][0] = o[tb][1] = zero4();
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb) {
        Lds& sh = *lds_opaque(sh0);
        Frag<E> sf[2];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) pack_frag(sf[pt], S[2 * kb][pt], S[2 * kb + 1][pt]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const Frag<E> q = ld_frag8(sh.q, LDK, 16 * tb + t16, 32 * kb);
          mma(o[tb][0], sf[0], q);
          mma(o[tb][1], sf[1], q);
        }
      }
      __syncthreads();  // Q K^T of all waves
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        Lds& sh = *lds_opaque(sh0);
        const ChunkDecay& dec = sh.dec[w];
        const float tf = dec.tf[16 * tb + t16];
        o[tb][0] *= tf;
        o[tb][1] *= tf;
#pragma unroll
        for (int kb = 0; kb <= tb / 2; ++kb) {
          const f32x4 m0 = sh.cb[tb * (tb + 1) / 2 + 2 * kb][l] * tile_decay(dec, tb, 2 * kb);
          f32x4 m1 = zero4();
          if (2 * kb + 1 <= tb) m1 = sh.cb[tb * (tb + 1) / 2 + 2 * kb + 1][l] * tile_decay(dec, tb, 2 * kb + 1);
          Frag<E> m;
          pack_frag(m, m0, m1);
          mma(o[tb][0], vf[kb][0], m);
          mma(o[tb][1], vf[kb][1], m);
        }
        const int row = 16 * tb + t16;
        if (active && row < c.nt) {
          const float tw = dec.tw[row];
          const E* vr = sh.v[w] + row * LDV + 8 * g4;
          const f32x4 y0 = o[tb][0] * tw + ld4f<E>(vr) * Dh, y1 = o[tb][1] * tw + ld4f<E>(vr + 4) * Dh;
          E* dst = static_cast<E*>(p.out1) + (row_of<REV>(c, row) * p.H + h) * p.Dv + col + 8 * g4;
          if constexpr (sizeof(E) == 2) {
            Frag<bf16> f;
            pack_frag(f, y0, y1);
            *reinterpret_cast<bf16x8*>(dst) = f.v;
          } else {
            st4f<E>(dst, y0);
            st4f<E>(dst + 4, y1);
          }
        }
      }
    }
    // S' = exp(tot) S + K^T (end V)
    const ChunkDecay& dec = lds_opaque(sh0)->dec[w];
    const float tot = dec.btw[3];
    if (!OUT) total *= tot;
    Parts<E> vp[2][2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const f32x4 e0 = *reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 4 * g4]);
      const f32x4 e1 = *reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 16 + 4 * g4]);
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) {
        f32x4 lo, hi;
        frag_f32(vf[kb][pt], lo, hi);
        split(vp[kb][pt], lo * e0, hi * e1);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      Lds& sh = *lds_opaque(sh0);
      S[nt][0] *= tot;
      S[nt][1] *= tot;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const Frag<E> kf = ld_col(sh.k, LDK, 32 * kb, 32 * (nt >> 1), nt & 1);
#pragma unroll
        for (int q = Parts<E>::N - 1; q >= 0; --q) {
          mma(S[nt][0], kf, vp[kb][0].p[q]);
          mma(S[nt][1], kf, vp[kb][1].p[q]);
        }
      }
    }
  }
  float* dst = OUT ? (last ? p.s_end : nullptr) : p.s_loc;
  if (!dst || !active) return;
  dst += ((int64_t)(OUT ? r.n : j) * p.H + h) * st_off + vcol;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[(int64_t)(key_of(nt) + i) * p.Dv + 4 * pt] = S[nt][pt][i];
  if (!OUT && l == 0 && col == 0) p.s_dec[(int64_t)j * p.H + h] = total;
}

// ---------------------------------------------------------------- key sweep
// A workgroup of Dk / 16 waves takes HS slices of PS = 64 value columns of one
// group of heads in one segment.  Wave nt owns 16 keys of all slices' states
// (transposed: values down, keys across), so that the sum of out2 over the
// slices stays in its accumulators; a slice's chunk matrix W V^T is formed tile
// by tile over the waves, decayed and summed over the slices in LDS before the
// one product with K.  out2 leaves as one fp32 part per workgroup.
template <class E, int DK, int HS>
struct KeyLds {
  E k[CH * row_ld<E>(DK)];
  E q[CH * row_ld<E>(DK)];
  E v[HS][CH * row_ld<E>(PS)];
  E w[HS][CH * row_ld<E>(PS)];
  f32x4 z[10][64];               // sum over slices of the decayed chunk matrix, by tile and lane
  float rti[4][HS][CH];          // row terms of the chunk itself, by source block
  float rtx[DK / 16][HS][CH];    // row terms of the state, by key tile
  double anc[DK / 16][HS];
  ChunkDecay dec[HS];
};

template <class E, int DK, int HS, bool REV>
__global__ __launch_bounds__(DK * 4) void sweep_key_kernel(SweepParams p, int parts) {
  extern __shared__ __align__(16) char smem[];
  typedef KeyLds<E, DK, HS> Lds;
  Lds* const sh0 = reinterpret_cast<Lds*>(smem);
  constexpr int LDK = row_ld<E>(DK), LDV = row_ld<E>(PS), NW = DK / 16, NTH = DK * 4;
  const int tid = threadIdx.x, nt = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), t16 = l & 15, g4 = l >> 4;
  const int part = blockIdx.x % parts, grp = blockIdx.x / parts % p.G, j = blockIdx.x / parts / p.G;
  SegRange r;
  if (!seg_range(p.seq, p.segs, p.seg_first, j, r)) return;
  const bool first = REV ? r.s == r.ns - 1 : r.s == 0;
  const int rep = p.H / p.G, spg = rep * (p.Dv / PS), spv = p.Dv / PS;
  const int64_t st_off = (int64_t)DK * p.Dv;
  const int ns = min(HS, spg - part * HS);       // slices of this workgroup
  auto slice_of = [&](int s) { return grp * spg + part * HS + min(s, ns - 1); };  // over all heads
  // key of a lane's column (as the state's column) and of its rows (as out2's)
  const int kcol = 32 * (nt >> 1) + 8 * (t16 >> 2) + 4 * (nt & 1) + (t16 & 3);
  const int krow = 32 * (nt >> 1) + 8 * g4 + 4 * (nt & 1);

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
#pragma unroll
        for (int i = 0; i < 4; ++i) T[s][pt][i] = s0[32 * (pt >> 1) + 8 * g4 + 4 * (pt & 1) + i];
    }
  }
  const int nch = (r.len + CH - 1) / CH, nab = (p.seq.segc + AB - 1) / AB;
  const int nsl = p.H * spv;  // slices of all heads
  // the state at anchor block b of this segment: [tile of 16 keys][pt][lane] per slice
  auto dump_of = [&](int b, int s) {
    return reinterpret_cast<f32x4*>(p.dump) + ((((int64_t)j * nab + b) * nsl + slice_of(s)) * NW + nt) * 256 + l;
  };
  TileStage<E, DK, NTH> tk, tq;
  TileStage<E, PS, NTH> tv[HS], tw[HS];
  static_assert(HS <= NW, "one wave a slice forms its decays");
  HeadConst hc;
  hc.load(p, slice_of(nt) / spv);
  float dt = 0.f;
  auto request = [&](int i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    dt = load_dt<REV>(p, c, slice_of(nt) / spv);
    tk.template load<REV>(static_cast<const E*>(p.k) + (int64_t)grp * DK, p.k_stride, c, tid);
    tq.template load<REV>(static_cast<const E*>(p.q) + (int64_t)grp * DK, p.q_stride, c, tid);
#pragma unroll
    for (int s = 0; s < HS; ++s) {
      tv[s].template load<REV>(static_cast<const E*>(p.v) + (int64_t)slice_of(s) * PS, p.v_stride, c, tid);
      tw[s].template load<REV>(static_cast<const E*>(p.w) + (int64_t)slice_of(s) * PS, p.w_stride, c, tid);
    }
  };
  if (nch > 0) request(0);
  for (int i = 0; i < nch; ++i) {
    const ChunkRows c = chunk_rows<REV>(r, i);
    const int ci = REV ? nch - 1 - i : i;  // chunk within the segment
    if (REV && ((ci + 1) % AB == 0 || i == 0)) {
      Lds& sh = *lds_opaque(sh0);
      // the state entering the chunk is the gradient of the state at its end
#pragma unroll
      for (int s = 0; s < HS; ++s) {
        double a = 0.;
        if (s < ns) {
          const f32x4* d = dump_of(ci / AB, s);
#pragma unroll
          for (int pt = 0; pt < 4; ++pt) {
            const f32x4 x = d[pt * 64];
#pragma unroll
            for (int e = 0; e < 4; ++e) a += (double)x[e] * T[s][pt][e];
          }
        }
        a = wave_sum_d(a);
        if (l == 0) sh.anc[nt][s] = a;
      }
      __syncthreads();
      if (tid < ns) {
        double a = 0.;
        for (int n = 0; n < NW; ++n) a += sh.anc[n][tid];
        p.anchor[((int64_t)j * nab + ci / AB) * nsl + slice_of(tid)] = a;
      }
    }
    __syncthreads();  // the previous chunk's reads are done
    {
      Lds& sh = *lds_opaque(sh0);
      tk.store(sh.k, LDK, tid);
      tq.store(sh.q, LDK, tid);
#pragma unroll
      for (int s = 0; s < HS; ++s) {
        tv[s].store(sh.v[s], LDV, tid);
        tw[s].store(sh.w[s], LDV, tid);
      }
    }
    const float raw = dt;
    if (i + 1 < nch) request(i + 1);
    if (nt < HS) fill_decay<REV>(lds_opaque(sh0)->dec[nt], p, hc, raw, c.nt);
    __syncthreads();
    // the chunk's own part: tiles of (rows s, columns t)
    for (int idx = nt; idx < 10; idx += NW) {
      Lds& sh = *lds_opaque(sh0);
      int tb, sb;
      tri_tile(idx, tb, sb);
      f32x4 cb = zero4(), zs = zero4();
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
#pragma unroll
      for (int s = 0; s < HS; ++s) {
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
        const f32x4 z = x * tile_decay(sh.dec[s], tb, sb);
        float rt = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (sb < tb || 4 * g4 + e < t16) rt += z[e] * cb[e];
        rt += __shfl_xor(rt, 16, 64);
        rt += __shfl_xor(rt, 32, 64);
        if (g4 == 0) sh.rti[sb][s][row] = rt;
        if (s < ns) zs += z * sh.dec[s].tw[row];
      }
      sh.z[idx][l] = zs;
    }
    __syncthreads();
    Frag<E> kf[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) kf[kb] = ld_col(lds_opaque(sh0)->k, LDK, 32 * kb, 32 * (nt >> 1), nt & 1);
    f32x4 o[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
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
      Parts<E> tp[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) split(tp[kb], T[s][2 * kb], T[s][2 * kb + 1]);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        Lds& sh = *lds_opaque(sh0);
        const ChunkDecay& dec = sh.dec[s];
        f32x4 u = zero4();
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const Frag<E> wf = ld_frag8(sh.w[s], LDV, 16 * tb + t16, 32 * kb);
#pragma unroll
          for (int q = Parts<E>::N - 1; q >= 0; --q) mma(u, tp[kb].p[q], wf);
        }
        const int row = 16 * tb + t16;
        const float tf = dec.tf[row];
        const f32x4 q4 = ld4f<E>(sh.q + row * LDK + krow);
        float rt = (u[0] * q4[0] + u[1] * q4[1]) + (u[2] * q4[2] + u[3] * q4[3]);
        rt += __shfl_xor(rt, 16, 64);
        rt += __shfl_xor(rt, 32, 64);
        if (g4 == 0) sh.rtx[nt][s][row] = rt * tf;
        o[tb] += u * (tf * dec.tw[row]);
      }
      // T' = exp(tot) T + V^T (end K)
      Lds& sh = *lds_opaque(sh0);
      const ChunkDecay& dec = sh.dec[s];
      Parts<E> kp[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        f32x4 lo, hi;
        frag_f32(kf[kb], lo, hi);
        split(kp[kb], lo * *reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 4 * g4]),
              hi * *reinterpret_cast<const f32x4*>(&dec.end[32 * kb + 16 + 4 * g4]));
      }
      const float tot = dec.btw[3];
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) {
        T[s][pt] *= tot;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          const Frag<E> vf = ld_col(sh.v[s], LDV, 32 * kb, 32 * (pt >> 1), pt & 1);
#pragma unroll
          for (int q = Parts<E>::N - 1; q >= 0; --q) mma(T[s][pt], vf, kp[kb].p[q]);
        }
      }
    }
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      const int row = 16 * tb + t16;
      if (row < c.nt)
        *reinterpret_cast<f32x4*>(p.out2 + ((int64_t)(grp * parts + part) * p.tokens + row_of<REV>(c, row)) * DK + krow) = o[tb];
    }
    if (!REV && ((ci + 1) % AB == 0 || ci + 1 == nch)) {
#pragma unroll
      for (int s = 0; s < HS; ++s)
        if (s < ns) {
          f32x4* d = dump_of(ci / AB, s);
#pragma unroll
          for (int pt = 0; pt < 4; ++pt) d[pt * 64] = T[s][pt];
        }
    }
    __syncthreads();
    Lds& sh = *lds_opaque(sh0);
    for (int k = tid; k < ns * CH; k += NTH) {
      const int s = k / CH, row = k % CH;
      if (row < c.nt) {
        float a = 0.f;
        for (int sb = 0; sb <= row / 16; ++sb) a += sh.rti[sb][s][row];
#pragma unroll
        for (int n = 0; n < NW; ++n) a += sh.rtx[n][s][row];
        p.rt[(int64_t)slice_of(s) * p.tokens + row_of<REV>(c, row)] = a;
      }
    }
  }
  if (REV && p.h0 && r.s == 0) {
    Lds& sh = *sh0;
    // <h0, its gradient>: the anchor at the sequence's start
#pragma unroll
    for (int s = 0; s < HS; ++s) {
      double a = 0.;
      if (s < ns) {
        const int sl = slice_of(s);
        const float* s0 = p.h0 + ((int64_t)r.n * p.H + sl / spv) * st_off + (int64_t)kcol * p.Dv + sl % spv * PS;
#pragma unroll
        for (int pt = 0; pt < 4; ++pt)
#pragma unroll
          for (int i = 0; i < 4; ++i) a += (double)T[s][pt][i] * s0[32 * (pt >> 1) + 8 * g4 + 4 * (pt & 1) + i];
      }
      a = wave_sum_d(a);
      if (l == 0) sh.anc[nt][s] = a;
    }
    __syncthreads();
    if (tid < ns) {
      double a = 0.;
      for (int n = 0; n < NW; ++n) a += sh.anc[n][tid];
      p.anchor0[(int64_t)r.n * nsl + slice_of(tid)] = a;
    }
  }
}

template <class E, int DK, int NW, bool REV, bool OUT>
hipError_t value_launch(const SweepParams& p, int nseg, hipStream_t st) {
  const int upg = p.H / p.G * (p.Dv / VC), parts = (upg + NW - 1) / NW;
  constexpr size_t lds = sizeof(ValueLds<E, DK, NW>);
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&sweep_value_kernel<E, DK, NW, REV, OUT>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((sweep_value_kernel<E, DK, NW, REV, OUT>), dim3(nseg * p.G * parts), dim3(NW * 64), lds, st, p, parts);
  return hipGetLastError();
}
template <class E, int DK, bool REV, bool OUT>
hipError_t value_nw(const SweepParams& p, int nseg, hipStream_t st) {
  const int upg = p.H / p.G * (p.Dv / VC);
  if (upg >= 8 && sizeof(E) == 2) return value_launch<E, DK, sizeof(E) == 2 ? 8 : 4, REV, OUT>(p, nseg, st);
  if (upg >= 4) return value_launch<E, DK, 4, REV, OUT>(p, nseg, st);
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

}  // namespace gdn
