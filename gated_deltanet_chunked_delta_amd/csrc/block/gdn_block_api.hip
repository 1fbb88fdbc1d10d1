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

}  // extern "C"
