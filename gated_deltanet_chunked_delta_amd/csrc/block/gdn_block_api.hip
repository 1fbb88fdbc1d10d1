// gdn_block_api.hip -- host side of a block's operators: argument checks, work
// division, workspaces and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "gdn_block.h"
#include "gdn_host.h"

namespace {

using namespace gdn_host;

bool known_dtype(int d) { return d == GDN_F32 || d == GDN_BF16; }
size_t esize(int d) { return d == GDN_BF16 ? 2 : 4; }

gdn_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need)
    return fail(GDN_E_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? have : (size_t)0);
  if (!aligned(ws, 16)) return fail(GDN_E_INVALID, "workspace must be 16-byte aligned");
  return GDN_OK;
}

// ---------------------------------------------------------------- residual norm
gdn_status check_rows(int64_t R, int32_t D) {
  if (R < 0 || D < 1) return fail(GDN_E_INVALID, "bad sizes R=%lld D=%d", (long long)R, D);
  if (R >= (1LL << 31) || R >= (1LL << 40) / D || D >= (1 << 24)) return fail(GDN_E_INVALID, "problem too large");
  return GDN_OK;
}
gdn_status check_addnorm(int dtype, int res_dtype, int64_t R, int32_t D, float eps, bool res) {
  if (!known_dtype(dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", dtype);
  if (res_dtype != dtype && (!res || res_dtype != GDN_F32))
    return fail(GDN_E_UNSUPPORTED, "res_dtype %d: the residual is in x's type or fp32", res_dtype);
  if (gdn_status st = check_rows(R, D); st != GDN_OK) return st;
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(GDN_E_INVALID, "eps must be positive and finite");
  return GDN_OK;
}
gdn_status check_addnorm_bwd(const gdn_addnorm_bwd_args& a) {
  return check_addnorm(a.dtype, a.res_dtype, a.R, a.D, a.eps, true);
}
int norm_blocks(const gdn_addnorm_bwd_args& a) { return gdn::addnorm_blocks(a.R, a.D, (int)esize(a.dtype), cu_count()); }

// ---------------------------------------------------------------- gated linear recurrence
bool launchable(double threads) { return threads < 4294967296. - 512.; }

gdn_status check_rec(const gdn_rec_args& a) {
  if (!known_dtype(a.dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", a.dtype);
  if (a.g_dtype != a.dtype && a.g_dtype != GDN_F32)
    return fail(GDN_E_UNSUPPORTED, "g_dtype %d: g is in x's type or fp32", a.g_dtype);
  if (a.B < 1 || a.T < 0 || a.D < 1) return fail(GDN_E_INVALID, "bad sizes B=%d T=%d D=%d", a.B, a.T, a.D);
  const long long tokens = (long long)a.B * a.T;
  if (tokens >= std::min((1LL << 40) / a.D, (1LL << 31) - 1024) || a.num_seqs >= (1LL << 37) / a.D || a.D >= (1 << 24))
    return fail(GDN_E_INVALID, "problem too large");
  if (a.cu_seqlens) {
    if (a.B != 1) return fail(GDN_E_INVALID, "cu_seqlens requires B == 1 (got %d)", a.B);
    if (a.num_seqs < 1) return fail(GDN_E_INVALID, "num_seqs must be >= 1 with cu_seqlens");
    if (!aligned(a.cu_seqlens, 4)) return fail(GDN_E_INVALID, "cu_seqlens misaligned");
  } else if (a.num_seqs != a.B) {
    return fail(GDN_E_INVALID, "num_seqs (%d) must equal B (%d) without cu_seqlens", a.num_seqs, a.B);
  }
  if (tokens > 0 && (!a.x || !a.g)) return fail(GDN_E_INVALID, "null input pointer");
  if (a.x_stride < a.D || a.g_stride < a.D || (a.i && a.i_stride < a.D))
    return fail(GDN_E_INVALID, "a token stride is below D = %d", a.D);
  const size_t es = esize(a.dtype);
  if (!aligned(a.x, es) || !aligned(a.i, es) || !aligned(a.g, esize(a.g_dtype)) || !aligned(a.scale, 4) || !aligned(a.h0, 4))
    return fail(GDN_E_INVALID, "a pointer is misaligned");
  return GDN_OK;
}
int64_t rec_chunks(const gdn_rec_args& a, int tokens) { return ((int64_t)a.B * a.T + tokens - 1) / tokens; }
struct RecPlan {
  int fwd, bwd;  // chunks
  size_t o_words = 0, o_enter = 0, o_part = 0, total = 0;
};
RecPlan rec_plan(const gdn_rec_args& a, bool bwd, bool own_states) {
  RecPlan p;
  p.fwd = (int)rec_chunks(a, gdn::REC_W * gdn::REC_FS);
  p.bwd = (int)rec_chunks(a, gdn::REC_W * gdn::REC_BS);
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes); return o; };
  p.o_words = take(8 * (size_t)gdn::rec_words(bwd ? p.bwd : p.fwd, a.D));
  if (bwd) {
    const size_t rows = 4 * (size_t)p.bwd * a.D;
    if (own_states) p.o_enter = take(rows);
    if (a.scale) p.o_part = take(rows);
  }
  p.total = off;
  return p;
}
gdn::RecParams rec_params(const gdn_rec_args& a, const RecPlan& pl, int nchunk) {
  gdn::RecParams p{};
  p.x = a.x; p.g = a.g; p.i = a.i; p.x_stride = a.x_stride; p.g_stride = a.g_stride; p.i_stride = a.i_stride;
  p.g_f32 = a.g_dtype == GDN_F32; p.scale = a.scale; p.h0 = a.h0; p.cu = a.cu_seqlens;
  p.T = a.T; p.D = a.D; p.N = a.num_seqs; p.tokens = a.B * a.T; p.nchunk = nchunk;
  p.words = nchunk > 1 ? at<uint64_t>(a.workspace, pl.o_words) : nullptr;
  return p;
}
gdn_status run_rec_fwd(const gdn_rec_args& a, const gdn::RecParams& p, hipStream_t s) {
  hipError_t e = timed("rec_fwd", s, [&] { return gdn::launch_rec_fwd(a.dtype, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "recurrence launch");
}

// ---------------------------------------------------------------- products
size_t bytes_of(int d) { return d == GDN_E4M3 ? 1 : esize(d); }
constexpr int64_t ROW_BYTES = 1 << 23;  // of an operand's row: 256 of them stay within a buffer's 2^31
int64_t row16(int64_t n, int dtype) { return (n * (int64_t)bytes_of(dtype) + 15) / 16 * 16; }

gdn_status check_linear(const gdn_linear_args& a, bool bwd) {
  const bool q = a.dtype == GDN_E4M3 && !bwd;
  if (!known_dtype(a.dtype) && !q) return fail(GDN_E_UNSUPPORTED, "unsupported dtype %d", a.dtype);
  if (!known_dtype(a.out_dtype) || (!q && a.out_dtype != a.dtype))
    return fail(GDN_E_UNSUPPORTED, "out_dtype %d does not go with dtype %d", a.out_dtype, a.dtype);
  if (a.M < 0 || a.N < 1 || a.K < 1) return fail(GDN_E_INVALID, "bad sizes M=%lld N=%d K=%d", (long long)a.M, a.N, a.K);
  if (a.act < GDN_ACT_NONE || a.act > GDN_ACT_GELU) return fail(GDN_E_UNSUPPORTED, "unknown activation %d", a.act);
  constexpr int64_t most = 1LL << 39;  // of a tensor's elements: more than the card's memory in any type
  if (a.M >= (1LL << 31) || a.N >= (1LL << 31) - 1024 || row16(a.K, a.dtype) >= ROW_BYTES || a.M * a.N >= most || a.M * a.K >= most || (int64_t)a.N * a.K >= most)
    return fail(GDN_E_INVALID, "problem too large");
  if (!a.w) return fail(GDN_E_INVALID, "null weight");
  if (a.M > 0 && !a.x) return fail(GDN_E_INVALID, "null input x");
  if (q && (!a.x_scale || !a.w_scale)) return fail(GDN_E_INVALID, "8-bit rows need x_scale and w_scale");
  if (!q && (a.x_scale || a.w_scale)) return fail(GDN_E_INVALID, "scales belong to 8-bit rows");
  if (a.x_stride < a.K || (a.r && a.r_stride < a.N)) return fail(GDN_E_INVALID, "a row stride is below its row's width");
  const size_t es = bytes_of(a.dtype), os = esize(a.out_dtype);
  if (!aligned(a.x, es) || !aligned(a.w, es) || !aligned(a.bias, os) || !aligned(a.r, os) || !aligned(a.x_scale, 4) ||
      !aligned(a.w_scale, 4))
    return fail(GDN_E_INVALID, "a pointer is misaligned");
  return GDN_OK;
}
// dx sums along N, dw along M: those are their operands' rows.
gdn_status check_linear_bwd(const gdn_linear_bwd_args& b) {
  if (gdn_status st = check_linear(b.a, true); st != GDN_OK) return st;
  if ((b.dx && row16(b.a.N, b.a.dtype) >= ROW_BYTES) || (b.dw && row16(b.a.M, b.a.dtype) >= ROW_BYTES))
    return fail(GDN_E_INVALID, "problem too large");
  return GDN_OK;
}
// Whether a product can read these rows as they lie.
bool rows_fit(const void* p, int64_t stride, int64_t n, int dtype) {
  const int64_t es = (int64_t)bytes_of(dtype);
  return aligned(p, 16) && stride * es % 16 == 0 && n * es % 16 == 0 && stride * es < ROW_BYTES;
}
struct LinearPlan {
  gdn::GemmPlan g;
  bool skinny = false;
  size_t o_x = 0, o_w = 0, o_part = 0, total = 0;
};
LinearPlan linear_plan(const gdn_linear_args& a) {
  LinearPlan p;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes); return o; };
  p.skinny = a.M <= gdn::SKINNY_M;
  if (!p.skinny) {
    const int64_t row = row16(a.K, a.dtype);
    if (!rows_fit(a.x, a.x_stride, a.K, a.dtype)) p.o_x = take((size_t)a.M * row);
    if (!rows_fit(a.w, a.K, a.K, a.dtype)) p.o_w = take((size_t)a.N * row);
    p.g = gdn::gemm_plan(a.M, a.N, row, (int)bytes_of(a.dtype), cu_count());
    p.o_part = take(gdn::gemm_part_bytes(p.g, a.M, a.N));
  }
  p.total = std::max<size_t>(off, 16);
  return p;
}
struct LinearBwdPlan {
  gdn::GemmPlan gx, gw;
  bool pre = false;  // dy act'(v), or dy re-laid, is written out
  size_t o_pre = 0, o_pre_t = 0, o_w_t = 0, o_x_t = 0, o_sums = 0, o_part = 0, total = 0;
};
LinearBwdPlan linear_bwd_plan(const gdn_linear_bwd_args& b) {
  const gdn_linear_args& a = b.a;
  LinearBwdPlan p;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes); return o; };
  const int64_t rn = row16(a.N, a.dtype), rm = row16(a.M, a.dtype);
  p.pre = b.dx && (a.act || !rows_fit(b.dy, a.N, a.N, a.dtype));
  if (p.pre) p.o_pre = take((size_t)a.M * rn);
  size_t part = 0;
  if (b.dx) {
    p.o_w_t = take((size_t)a.K * rn);
    p.gx = gdn::gemm_plan(a.M, a.K, rn, (int)bytes_of(a.dtype), cu_count());
    part = gdn::gemm_part_bytes(p.gx, a.M, a.K);
  }
  if (b.dw) {
    p.o_pre_t = take((size_t)a.N * rm);
    p.o_x_t = take((size_t)a.K * rm);
    p.gw = gdn::gemm_plan(a.N, a.K, rm, (int)bytes_of(a.dtype), cu_count());
    part = std::max(part, gdn::gemm_part_bytes(p.gw, a.N, a.K));
  }
  if (b.dbias) p.o_sums = take(4 * (size_t)((a.M + 63) / 64) * a.N);
  p.o_part = take(part);
  p.total = std::max<size_t>(off, 16);
  return p;
}
gdn::Epilogue epilogue(const gdn_linear_fwd_args& f) {
  const gdn_linear_args& a = f.a;
  gdn::Epilogue e{};
  e.x_scale = a.x_scale; e.w_scale = a.w_scale; e.bias = a.bias; e.r = a.r; e.r_stride = a.r_stride; e.act = a.act;
  e.out = f.y; e.v_save = f.v_save;
  return e;
}
gdn_status run_pack(int dtype, const gdn::PackJobs& jobs, hipStream_t s) {
  if (jobs.n == 0) return GDN_OK;
  hipError_t e = timed("linear_pack", s, [&] { return gdn::launch_pack(dtype, jobs, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "row copy launch");
}
// A product's names among the timed kernels, by its tiles.
struct GemmName { const char *large, *small; };
gdn_status run_gemm(GemmName name, int dtype, int out_dtype, gdn::GemmParams p, const gdn::GemmPlan& g, hipStream_t s) {
  p.splits = g.splits;
  p.steps = g.steps;
  hipError_t e = timed(g.tile == 256 ? name.large : name.small, s, [&] { return gdn::launch_gemm(dtype, out_dtype, p, g, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "product launch");
}

}  // namespace

extern "C" {

gdn_status gdn_addnorm_fwd(const gdn_addnorm_fwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_addnorm_fwd_args& a = *args;
  if (gdn_status st = check_addnorm(a.dtype, a.res_dtype, a.R, a.D, a.eps, a.r != nullptr); st != GDN_OK) return st;
  if (a.y && a.q) return fail(GDN_E_INVALID, "y and q are two forms of one output: give one of them");
  if (!a.w) return fail(GDN_E_INVALID, "null weight");
  if (a.R == 0) return GDN_OK;
  if (!a.x) return fail(GDN_E_INVALID, "null input x");
  if (!a.y && !a.q) return fail(GDN_E_INVALID, "null output");
  if (a.q && !a.q_scale) return fail(GDN_E_INVALID, "q needs q_scale");
  if (a.r && !a.s) return fail(GDN_E_INVALID, "r needs the sum s");
  if (a.x_stride < a.D || (a.r && a.r_stride < a.D)) return fail(GDN_E_INVALID, "a row stride is below D = %d", a.D);
  const size_t es = esize(a.dtype), rs = esize(a.res_dtype);
  if (!aligned(a.x, es) || !aligned(a.r, rs) || !aligned(a.w, es) || !aligned(a.s, rs) || !aligned(a.y, es) || !aligned(a.q_scale, 4))
    return fail(GDN_E_INVALID, "a pointer is misaligned");
  gdn::AddNormParams p{};
  p.x = a.x; p.x_stride = a.x_stride; p.r = a.r; p.r_stride = a.r_stride; p.w = a.w; p.s = a.s; p.y = a.y;
  p.q = static_cast<uint8_t*>(a.q); p.q_scale = a.q_scale; p.R = a.R; p.D = a.D; p.eps = a.eps;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("addnorm_fwd", s, [&] { return gdn::launch_addnorm_fwd(a.dtype, a.res_dtype, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "residual norm launch");
}

size_t gdn_addnorm_bwd_workspace_size(const gdn_addnorm_bwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_addnorm_bwd(*args) != GDN_OK) return 0;
  return std::max<size_t>(16, sizeof(float) * (size_t)norm_blocks(*args) * args->D);
}

gdn_status gdn_addnorm_bwd(const gdn_addnorm_bwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_addnorm_bwd_args& a = *args;
  if (gdn_status st = check_addnorm_bwd(a); st != GDN_OK) return st;
  if (!a.w) return fail(GDN_E_INVALID, "null weight");
  if (a.R > 0 && (!a.s || !a.dy)) return fail(GDN_E_INVALID, "null input pointer");
  if (!a.dx && !a.dr && !a.dw) return fail(GDN_E_INVALID, "no gradient asked for");
  if (a.s_stride < a.D) return fail(GDN_E_INVALID, "s_stride %lld below D = %d", (long long)a.s_stride, a.D);
  const size_t es = esize(a.dtype), rs = esize(a.res_dtype);
  if (!aligned(a.s, rs) || !aligned(a.w, es) || !aligned(a.dy, es) || !aligned(a.ds, rs) || !aligned(a.dx, es) ||
      !aligned(a.dr, rs) || !aligned(a.dw, es))
    return fail(GDN_E_INVALID, "a pointer is misaligned");
  if (gdn_status st = check_ws(a.workspace, a.workspace_bytes, gdn_addnorm_bwd_workspace_size(args)); st != GDN_OK) return st;
  gdn::AddNormParams p{};
  p.s = const_cast<void*>(a.s); p.x_stride = a.s_stride; p.w = a.w; p.dy = a.dy; p.ds = a.ds; p.dx = a.dx; p.dr = a.dr; p.dw = a.dw;
  p.R = a.R; p.D = a.D; p.eps = a.eps; p.part = static_cast<float*>(a.workspace); p.blocks = norm_blocks(a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("addnorm_bwd", s, [&] { return gdn::launch_addnorm_bwd(a.dtype, a.res_dtype, p, s); });
  if (e != hipSuccess) return hip_fail(e, "residual norm gradient launch");
  if (!a.dw) return GDN_OK;
  e = timed("addnorm_dw", s, [&] { return gdn::launch_join_parts(a.dtype, p.part, p.blocks, a.D, a.dw, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "weight gradient launch");
}

gdn_status gdn_quant_rows(const gdn_quant_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_quant_args& a = *args;
  if (!known_dtype(a.dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", a.dtype);
  if (gdn_status st = check_rows(a.R, a.D); st != GDN_OK) return st;
  if (a.R == 0) return GDN_OK;
  if (!a.x || !a.q || !a.q_scale) return fail(GDN_E_INVALID, "null pointer");
  if (a.x_stride < a.D) return fail(GDN_E_INVALID, "x_stride %lld below D = %d", (long long)a.x_stride, a.D);
  if (!aligned(a.x, esize(a.dtype)) || !aligned(a.q_scale, 4)) return fail(GDN_E_INVALID, "a pointer is misaligned");
  gdn::AddNormParams p{};
  p.x = a.x; p.x_stride = a.x_stride; p.q = static_cast<uint8_t*>(a.q); p.q_scale = a.q_scale; p.R = a.R; p.D = a.D;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("quant_rows", s, [&] { return gdn::launch_quant_rows(a.dtype, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "row quantisation launch");
}

size_t gdn_rec_fwd_workspace_size(const gdn_rec_fwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_rec(args->a) != GDN_OK) return 0;
  return rec_plan(args->a, false, !args->h_save).total;
}
size_t gdn_rec_bwd_workspace_size(const gdn_rec_bwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_rec(args->a) != GDN_OK) return 0;
  return rec_plan(args->a, true, !args->h_saved).total;
}
size_t gdn_rec_states_bytes(const gdn_rec_args* a) {
  if (!a) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_rec(*a) != GDN_OK) return 0;
  return std::max<size_t>(16, 4 * (size_t)rec_plan(*a, false, false).bwd * a->D);
}

gdn_status gdn_rec_fwd(const gdn_rec_fwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_rec_args& a = args->a;
  if (gdn_status st = check_rec(a); st != GDN_OK) return st;
  if ((long long)a.B * a.T > 0 && !args->y) return fail(GDN_E_INVALID, "null output y");
  if (!aligned(args->y, esize(a.dtype)) || !aligned(args->hT, 4) || !aligned(args->h_save, 4))
    return fail(GDN_E_INVALID, "a pointer is misaligned");
  const RecPlan pl = rec_plan(a, false, !args->h_save);
  if (gdn_status st = check_ws(a.workspace, a.workspace_bytes, pl.total); st != GDN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  gdn::RecParams p = rec_params(a, pl, pl.fwd);
  p.enter = args->h_save;
  p.y = args->y;
  p.hT = args->hT;
  return run_rec_fwd(a, p, s);
}

gdn_status gdn_rec_bwd(const gdn_rec_bwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_rec_args& a = args->a;
  if (gdn_status st = check_rec(a); st != GDN_OK) return st;
  if ((long long)a.B * a.T > 0 && (!args->dy || !args->dx || !args->dg || (a.i && !args->di)))
    return fail(GDN_E_INVALID, "null gradient pointer");
  if (a.scale && !args->dscale) return fail(GDN_E_INVALID, "null gradient pointer");
  const size_t es = esize(a.dtype);
  if (!aligned(args->dy, es) || !aligned(args->dx, es) || !aligned(args->di, es) || !aligned(args->dg, esize(a.g_dtype)) ||
      !aligned(args->dscale, 4) || !aligned(args->dh0, 4) || !aligned(args->dhT, 4) || !aligned(args->h_saved, 4))
    return fail(GDN_E_INVALID, "a gradient pointer is misaligned");
  const RecPlan pl = rec_plan(a, true, !args->h_saved);
  if (gdn_status st = check_ws(a.workspace, a.workspace_bytes, pl.total); st != GDN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  gdn::RecParams p = rec_params(a, pl, pl.bwd);
  p.enter = const_cast<float*>(args->h_saved);
  if (!args->h_saved) {  // the forward pass's states alone; its words lie where the gradient's will
    p.enter = at<float>(a.workspace, pl.o_enter);
    gdn::RecParams f = rec_params(a, pl, pl.fwd);
    f.enter = p.enter;
    if (gdn_status st = run_rec_fwd(a, f, s); st != GDN_OK) return st;
  }
  p.dy = args->dy; p.dhT = args->dhT; p.dx = args->dx; p.dg = args->dg; p.di = args->di; p.dh0 = args->dh0;
  p.part = a.scale ? at<float>(a.workspace, pl.o_part) : nullptr;
  hipError_t e = timed("rec_bwd", s, [&] { return gdn::launch_rec_bwd(a.dtype, p, s); });
  if (e != hipSuccess) return hip_fail(e, "recurrence gradient launch");
  if (!a.scale) return GDN_OK;
  e = timed("rec_dscale", s, [&] { return gdn::launch_join_parts(GDN_F32, p.part, pl.bwd, a.D, args->dscale, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "scale gradient launch");
}

gdn_status gdn_rec_step(const gdn_rec_step_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_rec_step_args& a = *args;
  if (!known_dtype(a.dtype)) return fail(GDN_E_UNSUPPORTED, "unknown dtype %d", a.dtype);
  if (a.g_dtype != a.dtype && a.g_dtype != GDN_F32)
    return fail(GDN_E_UNSUPPORTED, "g_dtype %d: g is in x's type or fp32", a.g_dtype);
  if (a.N < 0 || a.D < 1) return fail(GDN_E_INVALID, "bad sizes N=%d D=%d", a.N, a.D);
  if (a.D >= (1 << 24) || !launchable((a.D + 128.) * a.N)) return fail(GDN_E_INVALID, "problem too large");
  if (a.N == 0) return GDN_OK;
  if (!a.x || !a.g || !a.state || !a.y) return fail(GDN_E_INVALID, "null pointer");
  if (a.x_stride < a.D || a.g_stride < a.D || (a.i && a.i_stride < a.D))
    return fail(GDN_E_INVALID, "a token stride is below D = %d", a.D);
  const size_t es = esize(a.dtype);
  if (!aligned(a.x, es) || !aligned(a.i, es) || !aligned(a.y, es) || !aligned(a.g, esize(a.g_dtype)) || !aligned(a.scale, 4) ||
      !aligned(a.state, 4) || !aligned(a.state_idx, 4))
    return fail(GDN_E_INVALID, "misaligned pointer");
  if (a.num_slots < (a.state_idx ? 0 : a.N))
    return fail(GDN_E_INVALID, "num_slots (%d) must be >= N (%d) without state_idx", a.num_slots, a.N);
  gdn::RecStepParams p{};
  p.x = a.x; p.g = a.g; p.i = a.i; p.x_stride = a.x_stride; p.g_stride = a.g_stride; p.i_stride = a.i_stride;
  p.g_f32 = a.g_dtype == GDN_F32; p.scale = a.scale; p.state = a.state; p.state_idx = a.state_idx; p.num_slots = a.num_slots;
  p.N = a.N; p.D = a.D; p.y = a.y;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = timed("rec_step", s, [&] { return gdn::launch_rec_step(a.dtype, p, s); });
  return e == hipSuccess ? GDN_OK : hip_fail(e, "recurrence step launch");
}

size_t gdn_linear_fwd_workspace_size(const gdn_linear_fwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_linear(args->a, false) != GDN_OK) return 0;
  return linear_plan(args->a).total;
}
size_t gdn_linear_bwd_workspace_size(const gdn_linear_bwd_args* args) {
  if (!args) { fail(GDN_E_INVALID, "null args"); return 0; }
  if (check_linear_bwd(*args) != GDN_OK) return 0;
  return linear_bwd_plan(*args).total;
}

gdn_status gdn_linear_fwd(const gdn_linear_fwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_linear_args& a = args->a;
  if (gdn_status st = check_linear(a, false); st != GDN_OK) return st;
  if (a.M == 0) return GDN_OK;
  if (!args->y) return fail(GDN_E_INVALID, "null output y");
  if (!aligned(args->y, esize(a.out_dtype)) || !aligned(args->v_save, 4)) return fail(GDN_E_INVALID, "a pointer is misaligned");
  const LinearPlan pl = linear_plan(a);
  if (gdn_status st = pl.skinny ? GDN_OK : check_ws(a.workspace, a.workspace_bytes, pl.total); st != GDN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t es = (int64_t)bytes_of(a.dtype), row = row16(a.K, a.dtype);
  if (pl.skinny) {
    gdn::SkinnyParams p{};
    p.x = a.x; p.w = a.w; p.x_stride = a.x_stride * es; p.w_stride = a.K * es; p.M = (int)a.M; p.N = a.N;
    p.kbytes = (int)(a.K * es);
    p.e = epilogue(*args);
    hipError_t e = timed("linear_few", s, [&] { return gdn::launch_skinny(a.dtype, a.out_dtype, p, s); });
    return e == hipSuccess ? GDN_OK : hip_fail(e, "product launch");
  }
  gdn::GemmParams p{};
  p.a = a.x; p.lda = a.x_stride * es; p.b = a.w; p.ldb = a.K * es; p.M = a.M; p.N = a.N; p.kbytes = (int)row;
  p.part = at<float>(a.workspace, pl.o_part);
  p.e = epilogue(*args);
  auto relay = [&](const void* in, int64_t stride, int64_t R, size_t off) {
    gdn::PackJobs jobs{};
    gdn::PackParams& k = jobs.job[jobs.n++];
    k.in = in; k.ld = stride; k.R = R; k.C = a.K; k.rows = at<char>(a.workspace, off); k.ldo = row / es;
    return run_pack(a.dtype, jobs, s);
  };
  if (!rows_fit(a.x, a.x_stride, a.K, a.dtype)) {
    if (gdn_status st = relay(a.x, a.x_stride, a.M, pl.o_x); st != GDN_OK) return st;
    p.a = at<char>(a.workspace, pl.o_x);
    p.lda = row;
  }
  if (!rows_fit(a.w, a.K, a.K, a.dtype)) {
    if (gdn_status st = relay(a.w, a.K, a.N, pl.o_w); st != GDN_OK) return st;
    p.b = at<char>(a.workspace, pl.o_w);
    p.ldb = row;
  }
  return run_gemm({"linear_fwd_256", "linear_fwd_128"}, a.dtype, a.out_dtype, p, pl.g, s);
}

gdn_status gdn_linear_bwd(const gdn_linear_bwd_args* args, void* stream) {
  if (!args) return fail(GDN_E_INVALID, "null args");
  const gdn_linear_args& a = args->a;
  if (gdn_status st = check_linear_bwd(*args); st != GDN_OK) return st;
  if (a.M > 0 && !args->dy) return fail(GDN_E_INVALID, "null gradient pointer");
  if (!args->dx && !args->dw && !args->dbias) return fail(GDN_E_INVALID, "no gradient asked for");
  if (a.act && a.M > 0 && !args->v_saved) return fail(GDN_E_INVALID, "an activation's gradient needs v_saved");
  const size_t es = esize(a.dtype);
  if (!aligned(args->dy, es) || !aligned(args->dx, es) || !aligned(args->dw, es) || !aligned(args->dbias, es) ||
      !aligned(args->v_saved, 4))
    return fail(GDN_E_INVALID, "a pointer is misaligned");
  const LinearBwdPlan pl = linear_bwd_plan(*args);
  if (gdn_status st = check_ws(a.workspace, a.workspace_bytes, pl.total); st != GDN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  void* ws = a.workspace;
  const int64_t rn = row16(a.N, a.dtype), rm = row16(a.M, a.dtype);
  // dy act'(v): as it lies, turned, and its column sums; w and x turned
  gdn::PackParams k{}, wt{}, xt{};
  k.in = args->dy; k.ld = a.N; k.R = a.M; k.C = a.N;
  k.v = a.act ? args->v_saved : nullptr; k.act = a.act;
  if (pl.pre) { k.rows = at<char>(ws, pl.o_pre); k.ldo = rn / es; }
  if (args->dw) { k.cols = at<char>(ws, pl.o_pre_t); k.ldt = rm / es; }
  if (args->dbias) k.sums = at<float>(ws, pl.o_sums);
  // One launch for all copies, or x's own right before dw's product, its reader: made earlier it
  // leaves the 256 MB cache in front of the memory, as the sizes where this turns suggest, once the
  // turned copies of x and dy with dx's product between them fill enough of it.  Late against
  // early (us, bf16): copies of 67 + 67 MB 317, 310 (16,384 x 2,048 -> 2,048) and 228, 218 (32,768 x
  // 1,024 -> 1,024); 34 + 101 MB 418, 416; 101 + 50 MB 703, 731 (6,144 x 8,192 -> 4,096); 50 + 134 MB
  // 513, 510; 67 + 201 MB 832, 855 (16,384 x 2,048 -> 6,144); 134 + 134 MB 944, 983 (16,384 x 4,096
  // -> 4,096) and 418, 414 (65,536 x 1,024 -> 1,024).
  const bool x_late = args->dx && ((double)a.K + a.N) * rm > 144e6;
  gdn::PackJobs jobs{};
  if (a.M > 0) {
    if (k.rows || k.cols || k.sums) jobs.job[jobs.n++] = k;
    if (args->dx) {
      wt.in = a.w; wt.ld = a.K; wt.R = a.N; wt.C = a.K; wt.cols = at<char>(ws, pl.o_w_t); wt.ldt = rn / es;
      jobs.job[jobs.n++] = wt;
    }
    if (args->dw) {
      xt.in = a.x; xt.ld = a.x_stride; xt.R = a.M; xt.C = a.K; xt.cols = at<char>(ws, pl.o_x_t); xt.ldt = rm / es;
      if (!x_late) jobs.job[jobs.n++] = xt;
    }
  }
  if (gdn_status st = run_pack(a.dtype, jobs, s); st != GDN_OK) return st;
  if (args->dbias) {
    hipError_t e = timed("linear_dbias", s, [&] { return gdn::launch_join_parts(a.dtype, k.sums, (a.M + 63) / 64, a.N, args->dbias, s); });
    if (e != hipSuccess) return hip_fail(e, "bias gradient launch");
  }
  gdn::GemmParams p{};
  p.part = at<float>(ws, pl.o_part);
  if (args->dx && a.M > 0) {
    p.a = pl.pre ? k.rows : args->dy; p.lda = rn; p.b = wt.cols; p.ldb = rn;
    p.M = a.M; p.N = a.K; p.kbytes = (int)rn;
    p.e = gdn::Epilogue{};
    p.e.out = args->dx;
    if (gdn_status st = run_gemm({"linear_dx_256", "linear_dx_128"}, a.dtype, a.dtype, p, pl.gx, s); st != GDN_OK) return st;
  }
  if (args->dw) {
    if (x_late && a.M > 0) {
      gdn::PackJobs late{};
      late.job[late.n++] = xt;
      if (gdn_status st = run_pack(a.dtype, late, s); st != GDN_OK) return st;
    }
    p.a = k.cols; p.lda = rm; p.b = at<char>(ws, pl.o_x_t); p.ldb = rm;
    p.M = a.N; p.N = a.K; p.kbytes = (int)rm;
    p.e = gdn::Epilogue{};
    p.e.out = args->dw;
    if (gdn_status st = run_gemm({"linear_dw_256", "linear_dw_128"}, a.dtype, a.dtype, p, pl.gw, s); st != GDN_OK) return st;
  }
  return GDN_OK;
}

}  // extern "C"
