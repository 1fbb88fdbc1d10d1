// gdn_layer_api.hip -- host side of the operators around the recurrence:
// argument checks, work division, workspaces and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "gdn_host.h"
#include "gdn_layer.h"

namespace {

using namespace gdn_host;

bool known_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }
size_t esize(int d) { return d == GDN_BF16 ? 2 : 4; }

// A launch has fewer than 2^32 threads (in x; blocks of up to 512).
bool launchable(double threads) { return threads < 4294967296. - 512.; }

// ---------------------------------------------------------------- convolution
gdn_status check_conv(const gdn_conv_args& a) {
  if (!known_dtype(a.dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", a.dtype);
  if (a.B < 1 || a.T < 0 || a.D < 1) return fail(GDN_E_INVALID, "bad sizes B=%d T=%d D=%d", a.B, a.T, a.D);
  if (a.W < 2 || a.W > 4) return fail(GDN_E_UNSUPPORTED, "unsupported convolution width %d (2 to 4)", a.W);
  if (a.silu != 0 && a.silu != 1) return fail(GDN_E_INVALID, "silu must be 0 or 1");
  const size_t es = esize(a.dtype);
  // (token indices plus a run and its halo stay below 2^31)
  if ((long long)a.B * a.T >= std::min((1LL << 40) / a.D, (1LL << 31) - 1024)) return fail(GDN_E_INVALID, "problem too large");
  if (a.cu_seqlens) {
    if (a.B != 1) return fail(GDN_E_INVALID, "cu_seqlens requires B == 1 (got %d)", a.B);
    if (a.num_seqs < 1) return fail(GDN_E_INVALID, "num_seqs must be >= 1 with cu_seqlens");
    if (!aligned(a.cu_seqlens, 4)) return fail(GDN_E_INVALID, "cu_seqlens misaligned");
  } else if (a.num_seqs != a.B) {
    return fail(GDN_E_INVALID, "num_seqs (%d) must equal B (%d) without cu_seqlens", a.num_seqs, a.B);
  }
  if (!a.w) return fail(GDN_E_INVALID, "null weight");
  if ((long long)a.B * a.T > 0 && !a.x) return fail(GDN_E_INVALID, "null input x");
  if (a.x_stride < a.D) return fail(GDN_E_INVALID, "x_stride %lld below D = %d", (long long)a.x_stride, a.D);
  if (!aligned(a.x, es) || !aligned(a.w, es) || !aligned(a.bias, es) || !aligned(a.init, es))
    return fail(GDN_E_INVALID, "x, w, bias or init misaligned");
  return GDN_OK;
}

// Whether every row of D (or stride) elements at p can be accessed 16 bytes at a time.
bool vec_row(const void* p, int64_t width, int dtype) {
  return aligned(p, 16) && width % (16 / (int64_t)esize(dtype)) == 0;
}

gdn::ConvParams conv_params(const gdn_conv_args& a) {
  gdn::ConvParams p{};
  p.x = a.x; p.x_stride = a.x_stride; p.w = a.w; p.bias = a.bias; p.init = a.init; p.cu = a.cu_seqlens;
  p.B = a.B; p.T = a.T; p.D = a.D; p.N = a.num_seqs; p.silu = a.silu;
  p.tokens = (int64_t)a.B * a.T;
  return p;
}

// Tokens a thread walks: long runs re-read and recompute less at their ends
// (W-1 rows a run; the gradient also writes a row of W+1 fp32 parts a run),
// short runs give more threads.  The longest run that still leaves
// `waves_per_cu` waves for every compute unit, within [lo, hi].
int conv_run(const gdn_conv_args& a, bool vec, int lo, int hi, int waves_per_cu) {
  const int64_t tokens = (int64_t)a.B * a.T, cv = vec ? a.D * (int64_t)esize(a.dtype) / 16 : a.D;
  const int64_t want = (int64_t)cu_count() * waves_per_cu * 64;
  int run = lo;
  while (run < hi && (tokens + 2 * run - 1) / (2 * run) * cv >= want) run *= 2;
  return run;
}
bool conv_vec(const gdn_conv_args& a) {
  return vec_row(a.x, a.D, a.dtype) && vec_row(a.x, a.x_stride, a.dtype) && aligned(a.init, 16) && aligned(a.w, 16) &&
         aligned(a.bias, 16);
}
int64_t runs_of(const gdn_conv_args& a, int run) { return ((int64_t)a.B * a.T + run - 1) / run; }

// The threads of a pass with V channels each: the runs, and W-1 rows of each
// sequence's state where those are written.
bool conv_launchable(const gdn_conv_args& a, int run, int V, bool states) {
  return launchable((double)(runs_of(a, run) + (states ? (int64_t)a.num_seqs * (a.W - 1) : 0)) * (a.D / V));
}

// The gradient's run length does not depend on pointers, so that the workspace
// size is known before they are.
int conv_bwd_run(const gdn_conv_args& a) { return conv_run(a, a.D % (16 / (int)esize(a.dtype)) == 0, 16, 128, 4); }

// ---------------------------------------------------------------- scan
struct ScanPlan {
  int nseg = 0, nchunk = 0, segc = 1;
  bool multi = false;  // some sequence has more than one segment
  size_t o_chunk_first = 0, o_seg_first = 0, o_segs = 0, o_chunk_tab = 0;
  size_t o_state = 0, o_dec = 0, o_grad = 0, o_rt = 0, o_rt2 = 0, o_ct = 0, o_ct2 = 0, o_xd = 0, o_cb = 0, o_anchor = 0, o_dump = 0, o_sums = 0,
         o_part = 0, total = 0;
};

int seq_len(const gdn_scan_args& a, int n) {
  return a.cu_seqlens ? a.cu_seqlens_host[n + 1] - a.cu_seqlens_host[n] : a.T;
}
int64_t state_elems(const gdn_scan_args& a) { return (int64_t)a.H * a.Dk * a.Dv; }

// Chunks per segment.  A sweep runs one workgroup a compute unit at a time, so
// its time goes as the larger of its work's share and its longest segment, in
// chunks (of segments alike: rounds x chunks per segment), and a round takes a
// chunk's time to start.  Cutting adds a sweep for the segments' states (0.6 of an
// output chunk per chunk, measured) and a join, about two and a half chunks' time
// in all.  Among the shortest segments of a few round counts, and no cut at all,
// the cheapest.  Measured, forward, 16 heads of 128 x 128: 1,024 tokens in segments
// of 1 chunk 38 us, 4 62 us, uncut 106 us; 8,192 tokens in 4 chunks (one round)
// 84 us, 2 118 us, 8 106 us; 32,768 tokens in 16 (one round) 206 us, 8 236 us,
// 32 340 us; 128 tokens uncut 21 us, cut 31 us.
int auto_segment(const gdn_scan_args& a, int maxc, long long chunks) {
  if (maxc <= 1) return 1;
  const long long cus = cu_count(), per = gdn::sweep_workgroups(a.dtype, a.H, a.G, a.Dv);
  auto rounds = [&](int sc) {
    long long w = 0;
    if (!a.cu_seqlens) w = (long long)a.B * ((maxc + sc - 1) / sc);
    else
      for (int n = 0; n < a.num_seqs; ++n) w += std::max(1, ((seq_len(a, n) + gdn::CH - 1) / gdn::CH + sc - 1) / sc);
    return (w * per + cus - 1) / cus;
  };
  const double share = (double)chunks * per / cus;
  auto sweep = [&](long long r, int sc) { return std::min((double)r * sc, share + sc); };
  int best = maxc;
  const long long uncut = rounds(maxc);
  double least = sweep(uncut, maxc) + uncut;
  for (int more : {0, 1, 2, 3, 5, 7, 11, 15}) {
    const long long r = uncut + more;
    int lo = 1, hi = maxc;  // the shortest segments with at most r rounds
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (rounds(mid) <= r) hi = mid; else lo = mid + 1;
    }
    const double cost = lo >= maxc ? least : 1.6 * sweep(r, lo) + r + 2.5;
    if (cost < least) {
      least = cost;
      best = lo;
    }
  }
  return best;
}

ScanPlan scan_plan(const gdn_scan_args& a, bool bwd, bool own_states) {
  ScanPlan p;
  long long total = 0;
  int maxc = 0;
  for (int n = 0; n < a.num_seqs; ++n) {
    const int nc = (seq_len(a, n) + gdn::CH - 1) / gdn::CH;
    total += nc;
    maxc = std::max(maxc, nc);
  }
  p.nchunk = (int)total;
  if (a.seg_mode == -1) {
    p.segc = std::max(1, maxc);
  } else if (a.seg_mode > 0) {
    p.segc = std::min(a.seg_mode, std::max(1, maxc));
  } else {
    p.segc = auto_segment(a, maxc, total);
  }
  long long nseg = 0;
  for (int n = 0; n < a.num_seqs; ++n) {
    const int nc = (seq_len(a, n) + gdn::CH - 1) / gdn::CH;
    nseg += nc == 0 ? 1 : (nc + p.segc - 1) / p.segc;
  }
  p.nseg = (int)nseg;
  p.multi = p.nseg > a.num_seqs;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes); return o; };
  p.o_chunk_first = take(sizeof(int) * (a.num_seqs + 1));
  p.o_seg_first = take(sizeof(int) * (a.num_seqs + 1));
  p.o_segs = take(sizeof(gdn::SegDesc) * p.nseg);
  p.o_chunk_tab = take(sizeof(int2) * std::max(1, p.nchunk));
  const size_t st = p.multi ? sizeof(float) * state_elems(a) * p.nseg : 0;
  if (own_states) p.o_state = take(st);
  p.o_dec = take(sizeof(float) * a.H * (size_t)p.nseg);
  if (bwd) {
    const size_t tokens = (size_t)a.B * a.T, vh = (size_t)a.H * (a.Dv / gdn::PS);
    p.o_grad = take(st);
    p.o_rt = take(sizeof(float) * vh * tokens);
    p.o_rt2 = take(sizeof(float) * vh * tokens);
    p.o_ct = take(sizeof(float) * vh * tokens);
    p.o_ct2 = take(sizeof(float) * vh * tokens);
    p.o_xd = take(sizeof(float) * vh * tokens);
    p.o_cb = take(sizeof(float) * a.G * tokens);
    const size_t chunks = (size_t)p.nchunk;
    p.o_anchor = take(sizeof(double) * vh * chunks);
    p.o_dump = take(sizeof(float) * state_elems(a) * chunks);
    p.o_sums = take(sizeof(double) * 3 * a.H * chunks);
    const int parts = gdn::sweep_parts_per_group(a.dtype, a.H, a.G, a.Dv);
    if (parts > 1) p.o_part = take(sizeof(float) * parts * (size_t)a.G * tokens * a.Dk);
  }
  p.total = off;
  return p;
}

gdn_status check_scan(const gdn_scan_args& a) {
  if (!known_dtype(a.dtype) || !known_dtype(a.dt_dtype))
    return fail(GDN_E_UNSUPPORTED, "unknown dtype %d / dt_dtype %d", a.dtype, a.dt_dtype);
  if (a.B < 1 || a.T < 0 || a.H < 1 || a.G < 1 || a.Dk < 1 || a.Dv < 1)
    return fail(GDN_E_INVALID, "bad sizes B=%d T=%d H=%d G=%d Dk=%d Dv=%d", a.B, a.T, a.H, a.G, a.Dk, a.Dv);
  if (a.H % a.G != 0) return fail(GDN_E_INVALID, "H = %d is not a multiple of G = %d", a.H, a.G);
  if (!((a.Dk == 64 || a.Dk == 128) && a.Dv % gdn::PS == 0 && a.Dv <= 256))
    return fail(GDN_E_UNSUPPORTED, "unsupported head sizes Dk=%d Dv=%d", a.Dk, a.Dv);
  if (a.dt_softplus != 0 && a.dt_softplus != 1) return fail(GDN_E_INVALID, "dt_softplus must be 0 or 1");
  if (a.round_once != 0 && a.round_once != 1) return fail(GDN_E_INVALID, "round_once must be 0 or 1");
  const long long tokens = (long long)a.B * a.T;
  if (tokens >= (1LL << 31) || tokens * a.H * std::max(a.Dk, a.Dv) >= (1LL << 40) || (long long)a.H * a.Dv / gdn::PS > 65535)
    return fail(GDN_E_INVALID, "problem too large");
  if (tokens > 0 && (!a.x || !a.dt || !a.b || !a.c)) return fail(GDN_E_INVALID, "null input pointer");
  if (!a.A) return fail(GDN_E_INVALID, "null A");
  const int64_t v = 16 / (int64_t)esize(a.dtype);
  if (!aligned(a.x, 16) || !aligned(a.b, 16) || !aligned(a.c, 16))
    return fail(GDN_E_INVALID, "x, b and c must be 16-byte aligned");
  if (a.x_stride < (int64_t)a.H * a.Dv || a.b_stride < (int64_t)a.G * a.Dk || a.c_stride < (int64_t)a.G * a.Dk ||
      a.dt_stride < a.H)
    return fail(GDN_E_INVALID, "a token stride is below its row's width");
  if (a.x_stride % v || a.b_stride % v || a.c_stride % v)
    return fail(GDN_E_INVALID, "the token strides of x, b and c must be whole 16 bytes");
  const int64_t most = std::max({a.x_stride, a.b_stride, a.c_stride, a.dt_stride, (int64_t)a.H * a.Dv});
  if (most >= (1 << 22)) return fail(GDN_E_INVALID, "a token's row of %lld elements is too wide", (long long)most);
  if (!aligned(a.dt, esize(a.dt_dtype)) || !aligned(a.A, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4) ||
      !aligned(a.h0, 4))
    return fail(GDN_E_INVALID, "dt, A, D, dt_bias or h0 misaligned");
  if (a.cu_seqlens) {
    if (a.B != 1) return fail(GDN_E_INVALID, "cu_seqlens requires B == 1 (got %d)", a.B);
    if (!a.cu_seqlens_host) return fail(GDN_E_INVALID, "cu_seqlens needs its host copy cu_seqlens_host");
    if (a.num_seqs < 1) return fail(GDN_E_INVALID, "num_seqs must be >= 1 with cu_seqlens");
    const int32_t* cu = a.cu_seqlens_host;
    if (cu[0] != 0) return fail(GDN_E_INVALID, "cu_seqlens[0] must be 0");
    for (int n = 0; n < a.num_seqs; ++n)
      if (cu[n + 1] < cu[n]) return fail(GDN_E_INVALID, "cu_seqlens must be non-decreasing (index %d)", n);
    if (cu[a.num_seqs] != a.T) return fail(GDN_E_INVALID, "cu_seqlens[N] = %d != T = %d", cu[a.num_seqs], a.T);
  } else if (a.cu_seqlens_host) {
    return fail(GDN_E_INVALID, "cu_seqlens_host given without cu_seqlens");
  } else if (a.num_seqs != a.B) {
    return fail(GDN_E_INVALID, "num_seqs (%d) must equal B (%d) without cu_seqlens", a.num_seqs, a.B);
  }
  if (a.num_seqs > 65535) return fail(GDN_E_INVALID, "more than 65535 sequences");
  if (a.seg_mode < -1) return fail(GDN_E_INVALID, "seg_mode must be -1, 0 or a positive chunk count");
  return GDN_OK;
}

gdn_status check_grid(const gdn_scan_args& a, const ScanPlan& pl) {
  if (!launchable(512. * pl.nseg * gdn::sweep_workgroups(a.dtype, a.H, a.G, a.Dv)))
    return fail(GDN_E_INVALID, "problem too large: %d segments", pl.nseg);
  return GDN_OK;
}

gdn_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need)
    return fail(GDN_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? have : (size_t)0);
  if (!aligned(ws, 16)) return fail(GDN_E_INVALID, "workspace must be 16-byte aligned");
  return GDN_OK;
}

// The sweep parameters that do not depend on the direction.
gdn::SweepParams sweep_base(const gdn_scan_args& a, const ScanPlan& pl) {
  void* ws = a.workspace;
  gdn::SweepParams p{};
  p.dt = a.dt; p.dt_stride = a.dt_stride; p.dt_f32 = a.dt_dtype == GDN_F32; p.softplus = a.dt_softplus;
  p.dt_bias = a.dt_bias; p.A = a.A; p.H = a.H; p.G = a.G; p.Dk = a.Dk; p.Dv = a.Dv;
  p.tokens = (int64_t)a.B * a.T;
  p.seq.cu = a.cu_seqlens; p.seq.T = a.T; p.seq.segc = pl.segc;
  p.segs = at<gdn::SegDesc>(ws, pl.o_segs);
  p.seg_first = at<int>(ws, pl.o_seg_first);
  p.chunk_first = at<int>(ws, pl.o_chunk_first);
  p.per_seg = pl.multi;
  p.round_once = a.round_once;
  p.s_dec = at<float>(ws, pl.o_dec);
  return p;
}
// Forwards in time: keys B, queries C, values x; backwards: keys C, queries B, values dy.
void sweep_dir(gdn::SweepParams& p, const gdn_scan_args& a, bool rev, const void* dy) {
  p.k = rev ? a.c : a.b; p.k_stride = rev ? a.c_stride : a.b_stride;
  p.q = rev ? a.b : a.c; p.q_stride = rev ? a.b_stride : a.c_stride;
  const int64_t ys = (int64_t)a.H * a.Dv;
  p.v = rev ? dy : a.x; p.v_stride = rev ? ys : a.x_stride;
  p.w = rev ? a.x : dy; p.w_stride = rev ? a.x_stride : ys;
}

gdn_status scan_tables(const gdn_scan_args& a, const ScanPlan& pl, hipStream_t s) {
  if (!a.cu_seqlens) return GDN_OK;
  gdn::SeqInfo sq;
  sq.cu = a.cu_seqlens; sq.T = a.T; sq.segc = pl.segc;
  void* ws = a.workspace;
  hipError_t e = timed("plan", s, [&] {
    return gdn::launch_plan(sq, a.num_seqs, pl.segc, a.T, pl.nchunk, pl.nseg, at<int>(ws, pl.o_chunk_first),
                            at<int>(ws, pl.o_seg_first), at<gdn::SegDesc>(ws, pl.o_segs), at<int2>(ws, pl.o_chunk_tab), s);
  });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "plan launch");
}

// States entering every segment (in sweep order), into `state`.
gdn_status scan_states(const gdn_scan_args& a, const ScanPlan& pl, bool rev, const void* dy, const float* s0,
                       float* state, hipStream_t s) {
  gdn::SweepParams p = sweep_base(a, pl);
  sweep_dir(p, a, rev, dy);
  p.s_loc = state;
  hipError_t e = timed(rev ? "scan_state_rev" : "scan_state", s, [&] {
    return gdn::launch_sweep(a.dtype, rev, gdn::SWEEP_STATE, p, pl.nseg, s);
  });
  if (e != hipSuccess) return hip_fail(e, "scan state sweep launch");
  gdn::ScanJoinParams j{};
  j.s_loc = state; j.s_dec = p.s_dec; j.s0 = s0; j.H = a.H; j.Dk = a.Dk; j.Dv = a.Dv; j.rev = rev;
  j.seq = p.seq; j.segs = p.segs; j.seg_first = p.seg_first; j.N = a.num_seqs;
  e = timed("scan_join", s, [&] { return gdn::launch_scan_join(j, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "scan join launch");
}

// ---------------------------------------------------------------- norm
gdn_status check_norm(const gdn_norm_args& a) {
  if (!known_dtype(a.dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", a.dtype);
  if (a.R < 0 || a.G < 1 || a.D < 1)
    return fail(GDN_E_INVALID, "bad sizes R=%lld G=%d D=%d", (long long)a.R, a.G, a.D);
  if (a.R >= (1LL << 40) / a.G / a.D || a.R * a.G >= (1LL << 31) || a.G > 65535 ||
      a.D >= INT_MAX - 1024)
    return fail(GDN_E_INVALID, "problem too large");
  if ((a.shared | a.center | a.gate_first) & ~1) return fail(GDN_E_INVALID, "shared, center and gate_first must be 0 or 1");
  if (!(a.eps > 0.f) || !std::isfinite(a.eps)) return fail(GDN_E_INVALID, "eps must be positive and finite");
  if (!a.w) return fail(GDN_E_INVALID, "null weight");
  if (a.R > 0 && !a.x) return fail(GDN_E_INVALID, "null input x");
  if (a.gate_first && !a.z) return fail(GDN_E_INVALID, "gate_first needs z");
  const int64_t width = (int64_t)a.G * a.D;
  if (a.x_stride < width || (a.z && a.z_stride < width)) return fail(GDN_E_INVALID, "a token stride is below G * D");
  const size_t es = esize(a.dtype);
  if (!aligned(a.x, es) || !aligned(a.z, es) || !aligned(a.w, es) || !aligned(a.bias, es))
    return fail(GDN_E_INVALID, "x, z, w or bias misaligned");
  return GDN_OK;
}
bool norm_vec(const gdn_norm_args& a) {
  return vec_row(a.x, a.D, a.dtype) && vec_row(a.x, a.x_stride, a.dtype) && vec_row(a.w, a.D, a.dtype) &&
         vec_row(a.bias, a.D, a.dtype) && (!a.z || (vec_row(a.z, a.z_stride, a.dtype)));
}
gdn::NormParams norm_params(const gdn_norm_args& a) {
  gdn::NormParams p{};
  p.x = a.x; p.x_stride = a.x_stride; p.z = a.z; p.z_stride = a.z_stride; p.w = a.w; p.bias = a.bias;
  p.R = a.R; p.G = a.G; p.D = a.D; p.shared = a.shared; p.center = a.center; p.gate_first = a.gate_first; p.eps = a.eps;
  return p;
}
// Workgroups of the gradient, per weight group: each walks many rows and writes
// one row of parts, so about as many as are resident at once (rows of up to 64
// vectors: four a compute unit; longer ones, with more registers: two), but no
// more than there are rows.
int norm_blocks(const gdn_norm_args& a) {
  const int64_t groups = a.shared ? 1 : a.G, rows = a.shared ? a.R * a.G : a.R;
  const int64_t per_cu = a.D * (int64_t)esize(a.dtype) <= 64 * 16 ? 4 : 2;
  return (int)std::max<int64_t>(1, std::min<int64_t>(rows, per_cu * cu_count() / groups));
}
// Parts for the most workgroups: those that take one row at a time (how many they
// take depends on the pointers' alignment).
size_t norm_part_bytes(const gdn_norm_args& a) {
  const int64_t rows = a.shared ? a.R * a.G : a.R;
  const int64_t blocks = std::max<int64_t>(norm_blocks(a), (rows + gdn::NORM_ROWS - 1) / gdn::NORM_ROWS);
  return sizeof(float) * (a.shared ? 1 : a.G) * (size_t)blocks * (a.bias ? 2 : 1) * a.D;
}

}  // namespace

extern "C" {

gdn_status gdn_conv_fwd(const gdn_conv_fwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_conv_args& a = args->a;
  if (gdn_status st = check_conv(a); st != GDN_OK) return st;
  if ((long long)a.B * a.T > 0 && !args->y) return fail(GDN_E_INVALID, "null output y");
  if (!aligned(args->y, esize(a.dtype)) || !aligned(args->final_state, esize(a.dtype)))
    return fail(GDN_E_INVALID, "y or final_state misaligned");
  gdn::ConvParams p = conv_params(a);
  p.y = args->y;
  p.fin = args->final_state;
  const bool vec = conv_vec(a) && aligned(p.y, 16) && aligned(p.fin, 16);
  p.run = conv_run(a, vec, 4, 32, 16);
  p.nruns = runs_of(a, p.run);
  if (!conv_launchable(a, p.run, vec ? 16 / (int)esize(a.dtype) : 1, p.fin)) return fail(GDN_E_INVALID, "problem too large");
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("conv_fwd", s, [&] { return gdn::launch_conv_fwd(a.dtype, a.W, vec, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "convolution launch");
}

size_t gdn_conv_bwd_workspace_size(const gdn_conv_bwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  const gdn_conv_args& a = args->a;
  if (check_conv(a) != GDN_OK) return 0;
  return std::max<size_t>(16, sizeof(float) * (size_t)runs_of(a, conv_bwd_run(a)) * (a.W + 1) * a.D);
}

gdn_status gdn_conv_bwd(const gdn_conv_bwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_conv_args& a = args->a;
  if (gdn_status st = check_conv(a); st != GDN_OK) return st;
  const size_t es = esize(a.dtype);
  if ((long long)a.B * a.T > 0 && (!args->dy || !args->dx)) return fail(GDN_E_INVALID, "null gradient pointer");
  if (!args->dw) return fail(GDN_E_INVALID, "null gradient pointer");
  if (!aligned(args->dy, es) || !aligned(args->dfinal, es) || !aligned(args->dx, es) || !aligned(args->dw, es) ||
      !aligned(args->dbias, es) || !aligned(args->dinit, es))
    return fail(GDN_E_INVALID, "a gradient pointer is misaligned");
  if (gdn_status st = check_ws(args->workspace, args->workspace_bytes, gdn_conv_bwd_workspace_size(args)); st != GDN_OK)
    return st;
  gdn::ConvParams p = conv_params(a);
  p.dy = args->dy; p.dfin = args->dfinal; p.dx = args->dx; p.dw = args->dw; p.dbias = args->dbias; p.dinit = args->dinit;
  p.part = static_cast<float*>(args->workspace);
  p.run = conv_bwd_run(a);
  p.nruns = runs_of(a, p.run);
  const bool vec = conv_vec(a) && aligned(p.dy, 16) && aligned(p.dx, 16) && aligned(p.dfin, 16) && aligned(p.dinit, 16);
  if (!conv_launchable(a, p.run, vec ? 4 : 1, p.dinit) || !launchable(16. * (a.W + 1) * a.D))
    return fail(GDN_E_INVALID, "problem too large");
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("conv_bwd", s, [&] { return gdn::launch_conv_bwd(a.dtype, a.W, vec, p, s); });
  if (e != hipSuccess) return hip_fail(e, "convolution gradient launch");
  e = timed("conv_dw", s, [&] { return gdn::launch_conv_dw(a.dtype, a.W, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "convolution weight gradient launch");
}

gdn_status gdn_conv_step(const gdn_conv_step_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_conv_step_args& a = *args;
  if (!known_dtype(a.dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", a.dtype);
  if (a.N < 0 || a.D < 1) return fail(GDN_E_INVALID, "bad sizes N=%d D=%d", a.N, a.D);
  if (a.W < 2 || a.W > 4) return fail(GDN_E_UNSUPPORTED, "unsupported convolution width %d (2 to 4)", a.W);
  if (a.silu != 0 && a.silu != 1) return fail(GDN_E_INVALID, "silu must be 0 or 1");
  if ((long long)a.N * a.D >= (1LL << 32) - 64) return fail(GDN_E_INVALID, "problem too large");
  if (a.N == 0) return GDN_OK;
  if (!a.x || !a.state || !a.w || !a.y) return fail(GDN_E_INVALID, "null pointer");
  if (a.x_stride < a.D) return fail(GDN_E_INVALID, "x_stride %lld below D = %d", (long long)a.x_stride, a.D);
  const size_t es = esize(a.dtype);
  if (!aligned(a.x, es) || !aligned(a.state, es) || !aligned(a.w, es) || !aligned(a.bias, es) || !aligned(a.y, es) ||
      !aligned(a.state_idx, 4))
    return fail(GDN_E_INVALID, "misaligned pointer");
  if (a.num_slots < (a.state_idx ? 0 : a.N))
    return fail(GDN_E_INVALID, "num_slots (%d) must be >= N (%d) without state_idx", a.num_slots, a.N);
  gdn::ConvStepParams p{};
  p.x = a.x; p.x_stride = a.x_stride; p.state = a.state; p.state_idx = a.state_idx; p.num_slots = a.num_slots;
  p.w = a.w; p.bias = a.bias; p.y = a.y; p.N = a.N; p.D = a.D; p.silu = a.silu;
  const bool vec = vec_row(a.x, a.D, a.dtype) && vec_row(a.x, a.x_stride, a.dtype) && aligned(a.state, 16) && aligned(a.y, 16) &&
                   aligned(a.w, 16) && aligned(a.bias, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("conv_step", s, [&] { return gdn::launch_conv_step(a.dtype, a.W, vec, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "convolution step launch");
}

size_t gdn_scan_fwd_workspace_size(const gdn_scan_fwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_scan(args->a) != GDN_OK) return 0;
  return scan_plan(args->a, false, args->h_save == nullptr).total;
}
size_t gdn_scan_bwd_workspace_size(const gdn_scan_bwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_scan(args->a) != GDN_OK) return 0;
  return scan_plan(args->a, true, args->h_saved == nullptr).total;
}
size_t gdn_scan_states_bytes(const gdn_scan_args* a) {
  if (!a) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_scan(*a) != GDN_OK) return 0;
  const ScanPlan pl = scan_plan(*a, false, false);
  return pl.multi ? sizeof(float) * (size_t)state_elems(*a) * pl.nseg : 0;
}

gdn_status gdn_scan_fwd(const gdn_scan_fwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_scan_args& a = args->a;
  if (gdn_status st = check_scan(a); st != GDN_OK) return st;
  if ((long long)a.B * a.T > 0 && !args->y) return fail(GDN_E_INVALID, "null output y");
  if (!aligned(args->y, 16)) return fail(GDN_E_INVALID, "y must be 16-byte aligned");
  if (!aligned(args->hT, 4) || !aligned(args->h_save, 4)) return fail(GDN_E_INVALID, "hT or h_save misaligned");
  const ScanPlan pl = scan_plan(a, false, args->h_save == nullptr);
  if (gdn_status st = check_grid(a, pl); st != GDN_OK) return st;
  if (gdn_status st = check_ws(a.workspace, a.workspace_bytes, pl.total); st != GDN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (gdn_status st = scan_tables(a, pl, s); st != GDN_OK) return st;
  gdn::SweepParams p = sweep_base(a, pl);
  sweep_dir(p, a, false, nullptr);
  p.s_in = a.h0;
  if (pl.multi) {
    float* state = args->h_save ? args->h_save : at<float>(a.workspace, pl.o_state);
    if (gdn_status st = scan_states(a, pl, false, nullptr, a.h0, state, s); st != GDN_OK) return st;
    p.s_in = state;
  }
  p.D = a.D;
  p.out1 = args->y;
  p.s_end = args->hT;
  hipError_t e = timed("scan_fwd", s, [&] { return gdn::launch_sweep(a.dtype, 0, gdn::SWEEP_VALUE, p, pl.nseg, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "scan launch");
}

gdn_status gdn_scan_bwd(const gdn_scan_bwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_scan_args& a = args->a;
  if (gdn_status st = check_scan(a); st != GDN_OK) return st;
  if ((long long)a.B * a.T > 0 && (!args->dy || !args->dx || !args->ddt || !args->db || !args->dc))
    return fail(GDN_E_INVALID, "null gradient pointer");
  if (!args->dA) return fail(GDN_E_INVALID, "null gradient pointer");
  if (!aligned(args->dy, 16) || !aligned(args->dx, 16) || !aligned(args->db, 16) || !aligned(args->dc, 16))
    return fail(GDN_E_INVALID, "dy, dx, db and dc must be 16-byte aligned");
  if (!aligned(args->ddt, esize(a.dt_dtype)) || !aligned(args->dA, 4) || !aligned(args->dD, 4) ||
      !aligned(args->ddt_bias, 4) || !aligned(args->dh0, 4) || !aligned(args->dhT, 4) || !aligned(args->h_saved, 4))
    return fail(GDN_E_INVALID, "a gradient pointer is misaligned");
  const ScanPlan pl = scan_plan(a, true, args->h_saved == nullptr);
  if (gdn_status st = check_grid(a, pl); st != GDN_OK) return st;
  if (gdn_status st = check_ws(a.workspace, a.workspace_bytes, pl.total); st != GDN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  void* ws = a.workspace;
  if (gdn_status st = scan_tables(a, pl, s); st != GDN_OK) return st;
  // states entering the segments, in both directions
  const float* hs = a.h0;
  const float* gs = args->dhT;
  if (pl.multi) {
    hs = args->h_saved;
    if (!hs) {
      float* own = at<float>(ws, pl.o_state);
      if (gdn_status st = scan_states(a, pl, false, nullptr, a.h0, own, s); st != GDN_OK) return st;
      hs = own;
    }
    float* grad = at<float>(ws, pl.o_grad);
    if (gdn_status st = scan_states(a, pl, true, args->dy, args->dhT, grad, s); st != GDN_OK) return st;
    gs = grad;
  }
  gdn::ScanReduceParams red{};
  red.part = at<float>(ws, pl.o_part);
  red.G = a.G; red.ppg = gdn::sweep_parts_per_group(a.dtype, a.H, a.G, a.Dv); red.Dk = a.Dk; red.tokens = (int64_t)a.B * a.T;
  // dC, the forward row terms, and the states at the anchors
  gdn::SweepParams p = sweep_base(a, pl);
  sweep_dir(p, a, false, args->dy);
  red.seq = p.seq; red.segs = p.segs;
  p.s_in = hs;
  p.out2 = at<float>(ws, pl.o_part);
  p.out2_whole = args->dc;
  p.rt = at<float>(ws, pl.o_rt);
  p.rt2 = at<float>(ws, pl.o_rt2);
  p.dump = at<float>(ws, pl.o_dump);
  hipError_t e = timed("scan_dc", s, [&] { return gdn::launch_sweep(a.dtype, 0, gdn::SWEEP_KEY, p, pl.nseg, s); });
  if (e != hipSuccess) return hip_fail(e, "scan dC launch");
  red.out = args->dc;
  if (red.ppg > 1) e = timed("scan_reduce", s, [&] { return gdn::launch_scan_reduce(a.dtype, red, s); });
  if (e != hipSuccess) return hip_fail(e, "scan reduce launch");
  // dB, and the backward row terms
  p = sweep_base(a, pl);
  sweep_dir(p, a, true, args->dy);
  p.s_in = gs;
  p.out2 = at<float>(ws, pl.o_part);
  p.out2_whole = args->db;
  p.rt = at<float>(ws, pl.o_ct);
  p.rt2 = at<float>(ws, pl.o_ct2);
  p.xd = at<float>(ws, pl.o_xd);
  p.cb = at<float>(ws, pl.o_cb);
  p.dump = at<float>(ws, pl.o_dump);
  p.anchor = at<double>(ws, pl.o_anchor);
  e = timed("scan_db", s, [&] { return gdn::launch_sweep(a.dtype, 1, gdn::SWEEP_KEY, p, pl.nseg, s); });
  if (e != hipSuccess) return hip_fail(e, "scan dB launch");
  red.out = args->db;
  if (red.ppg > 1) e = timed("scan_reduce", s, [&] { return gdn::launch_scan_reduce(a.dtype, red, s); });
  if (e != hipSuccess) return hip_fail(e, "scan reduce launch");
  // dx, dh0
  p.xd = nullptr; p.cb = nullptr;
  p.D = a.D;
  p.out1 = args->dx;
  p.s_end = args->dh0;
  e = timed("scan_dx", s, [&] { return gdn::launch_sweep(a.dtype, 1, gdn::SWEEP_VALUE, p, pl.nseg, s); });
  if (e != hipSuccess) return hip_fail(e, "scan dx launch");
  gdn::ScanGradParams g{};
  g.dt = a.dt; g.dt_stride = a.dt_stride; g.dt_f32 = a.dt_dtype == GDN_F32; g.softplus = a.dt_softplus;
  g.dt_bias = a.dt_bias; g.A = a.A; g.H = a.H; g.G = a.G; g.Dk = a.Dk; g.Dv = a.Dv; g.tokens = (int64_t)a.B * a.T;
  g.seq = p.seq; g.segs = p.segs; g.chunk_tab = at<int2>(ws, pl.o_chunk_tab);
  g.rt = at<float>(ws, pl.o_rt); g.rt2 = at<float>(ws, pl.o_rt2); g.ct = at<float>(ws, pl.o_ct); g.ct2 = at<float>(ws, pl.o_ct2); g.xd = at<float>(ws, pl.o_xd); g.cb = at<float>(ws, pl.o_cb);
  g.anchor = at<double>(ws, pl.o_anchor);
  g.has_h0 = a.h0 != nullptr;
  g.ddt = args->ddt; g.part = at<double>(ws, pl.o_sums); g.dA = args->dA; g.dD = args->dD; g.ddt_bias = args->ddt_bias;
  e = timed("scan_ddt", s, [&] { return gdn::launch_scan_grad(g, pl.nchunk, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "scan step gradient launch");
}

gdn_status gdn_scan_step(const gdn_scan_step_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_scan_step_args& a = *args;
  if (!known_dtype(a.dtype) || !known_dtype(a.dt_dtype))
    return fail(GDN_E_UNSUPPORTED, "unknown dtype %d / dt_dtype %d", a.dtype, a.dt_dtype);
  if (a.N < 0 || a.H < 1 || a.G < 1 || a.Dk < 1 || a.Dv < 1)
    return fail(GDN_E_INVALID, "bad sizes N=%d H=%d G=%d Dk=%d Dv=%d", a.N, a.H, a.G, a.Dk, a.Dv);
  if (a.H % a.G != 0) return fail(GDN_E_INVALID, "H = %d is not a multiple of G = %d", a.H, a.G);
  if (!((a.Dk == 64 || a.Dk == 128) && a.Dv % gdn::PS == 0 && a.Dv <= 256))
    return fail(GDN_E_UNSUPPORTED, "unsupported head sizes Dk=%d Dv=%d", a.Dk, a.Dv);
  if (a.dt_softplus != 0 && a.dt_softplus != 1) return fail(GDN_E_INVALID, "dt_softplus must be 0 or 1");
  if ((long long)a.N * a.H >= (1LL << 24)) return fail(GDN_E_INVALID, "problem too large");
  if (a.N == 0) return GDN_OK;
  if (!a.x || !a.dt || !a.b || !a.c || !a.A || !a.state || !a.y) return fail(GDN_E_INVALID, "null pointer");
  if (a.x_stride < (int64_t)a.H * a.Dv || a.b_stride < (int64_t)a.G * a.Dk || a.c_stride < (int64_t)a.G * a.Dk ||
      a.dt_stride < a.H)
    return fail(GDN_E_INVALID, "a token stride is below its row's width");
  const size_t es = esize(a.dtype);
  if (!aligned(a.x, 16) || a.x_stride % (16 / (int64_t)es) || !aligned(a.state, 16))
    return fail(GDN_E_INVALID, "x and state must be 16-byte aligned, x_stride whole 16 bytes");
  if (!aligned(a.b, es) || !aligned(a.c, es) || !aligned(a.y, es) || !aligned(a.dt, esize(a.dt_dtype)) ||
      !aligned(a.A, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4) || !aligned(a.state_idx, 4))
    return fail(GDN_E_INVALID, "misaligned pointer");
  if (a.num_slots < (a.state_idx ? 0 : a.N))
    return fail(GDN_E_INVALID, "num_slots (%d) must be >= N (%d) without state_idx", a.num_slots, a.N);
  gdn::ScanStepParams p{};
  p.x = a.x; p.dt = a.dt; p.b = a.b; p.c = a.c;
  p.x_stride = a.x_stride; p.dt_stride = a.dt_stride; p.b_stride = a.b_stride; p.c_stride = a.c_stride;
  p.A = a.A; p.D = a.D; p.dt_bias = a.dt_bias; p.dt_f32 = a.dt_dtype == GDN_F32; p.softplus = a.dt_softplus;
  p.state = a.state; p.state_idx = a.state_idx; p.num_slots = a.num_slots; p.y = a.y; p.N = a.N; p.H = a.H; p.G = a.G; p.Dv = a.Dv;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("scan_step", s, [&] { return gdn::launch_scan_step(a.dtype, a.Dk, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "scan step launch");
}

gdn_status gdn_norm_fwd(const gdn_norm_fwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_norm_args& a = args->a;
  if (gdn_status st = check_norm(a); st != GDN_OK) return st;
  if (a.R == 0) return GDN_OK;
  if (!args->y) return fail(GDN_E_INVALID, "null output y");
  if (!aligned(args->y, esize(a.dtype))) return fail(GDN_E_INVALID, "y misaligned");
  gdn::NormParams p = norm_params(a);
  p.y = args->y;
  const bool vec = norm_vec(a) && aligned(p.y, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("norm_fwd", s, [&] { return gdn::launch_norm_fwd(a.dtype, vec, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "norm launch");
}

size_t gdn_norm_bwd_workspace_size(const gdn_norm_bwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_norm(args->a) != GDN_OK) return 0;
  return std::max<size_t>(16, norm_part_bytes(args->a));
}

gdn_status gdn_norm_bwd(const gdn_norm_bwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_norm_args& a = args->a;
  if (gdn_status st = check_norm(a); st != GDN_OK) return st;
  if (a.R > 0 && (!args->dy || !args->dx || (a.z && !args->dz))) return fail(GDN_E_INVALID, "null gradient pointer");
  if (!args->dw || (a.bias && !args->dbias)) return fail(GDN_E_INVALID, "null gradient pointer");
  if (!launchable((a.bias ? 32. : 16.) * a.D)) return fail(GDN_E_INVALID, "problem too large");
  const size_t es = esize(a.dtype);
  if (!aligned(args->dy, es) || !aligned(args->dx, es) || !aligned(args->dz, es) || !aligned(args->dw, es) ||
      !aligned(args->dbias, es))
    return fail(GDN_E_INVALID, "a gradient pointer is misaligned");
  if (gdn_status st = check_ws(args->workspace, args->workspace_bytes, gdn_norm_bwd_workspace_size(args)); st != GDN_OK)
    return st;
  gdn::NormParams p = norm_params(a);
  p.dy = args->dy; p.dx = args->dx; p.dz = a.z ? args->dz : nullptr; p.dw = args->dw; p.dbias = a.bias ? args->dbias : nullptr;
  p.part = static_cast<float*>(args->workspace);
  p.blocks = norm_blocks(a);
  const bool vec = norm_vec(a) && aligned(p.dy, 16) && aligned(p.dx, 16) && aligned(p.dz, 16);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("norm_bwd", s, [&] { return gdn::launch_norm_bwd(a.dtype, vec, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "norm gradient launch");
}

}  // extern "C"
