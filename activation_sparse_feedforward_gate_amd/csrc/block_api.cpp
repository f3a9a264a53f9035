// C-ABI entry points of the operators around the layer (residual sum, norm and
// dropout) and of those on 4-bit weights: argument checks on the host, then
// kernel launches on the caller's stream.  No allocation, no synchronisation.
#include <math.h>

#include "../../include/twell.h"
#include "internal.hpp"

using namespace twell;

namespace {

#define FAIL(st, ...) ((twell_status)set_error((st), __VA_ARGS__))

twell_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return TWELL_OK;
  return FAIL(TWELL_EHIP, "%s: %s", what, hipGetErrorString(e));
}

bool float_dt(int dt) { return dt == TWELL_F32 || dt == TWELL_BF16; }
int dt_size(int dt) { return dt == TWELL_F32 ? 4 : dt == TWELL_BF16 ? 2 : 1; }

twell_status check_norm_shape(const twell_norm_shape* sh, bool mx_y) {
  if (!sh) return FAIL(TWELL_EINVAL, "shape is NULL");
  if (sh->T < 0 || sh->d <= 0) return FAIL(TWELL_EINVAL, "bad shape T=%d d=%d", sh->T, sh->d);
  if (!float_dt(sh->x_dt) || !float_dt(sh->res_dt) || !float_dt(sh->w_dt) ||
      !(float_dt(sh->y_dt) || (mx_y && sh->y_dt == TWELL_MXFP8)))
    return FAIL(TWELL_EINVAL, "bad dtype");
  if (!(sh->p >= 0.f && sh->p <= 1.f)) return FAIL(TWELL_EINVAL, "dropout probability outside 0..1");
  if (!(sh->eps >= 0.f) || isinf(sh->eps)) return FAIL(TWELL_EINVAL, "eps must be finite and >= 0");
  if (sh->d > 65536) return FAIL(TWELL_EUNSUPPORTED, "d=%d too large (max 65536)", sh->d);
  return TWELL_OK;
}

// One matrix argument: its pointer's alignment and its row stride.
twell_status mat(RowMat* m, const twell_norm_shape* sh, const void* p, int64_t ld, int dt, const char* name) {
  m->p = const_cast<void*>(p);
  m->ld = sh->T <= 1 ? sh->d : ld;
  m->dt = dt;
  if (!p) return TWELL_OK;
  if ((uintptr_t)p % dt_size(dt)) return FAIL(TWELL_EINVAL, "%s is not aligned to its elements", name);
  if (m->ld < sh->d) return FAIL(TWELL_EINVAL, "row stride %lld of %s < d=%d", (long long)ld, name, sh->d);
  return TWELL_OK;
}

// Whether a (written) and b share memory.  Exact for one pitch (columns of one wider
// buffer share none); with two, any common range of addresses counts.
bool overlap(const RowMat& a, const RowMat& b, int T, int d) {
  typedef __int128 wide;
  if (!a.p || !b.p || T <= 0) return false;
  const wide la = (wide)d * dt_size(a.dt), lb = (wide)d * dt_size(b.dt);           // bytes of a row
  const wide pa = (wide)a.ld * dt_size(a.dt), pb = (wide)b.ld * dt_size(b.dt);     // and of a row's stride
  const wide by = (wide)(uintptr_t)b.p - (wide)(uintptr_t)a.p;
  if (by >= (T - 1) * pa + la || -by >= (T - 1) * pb + lb) return false;
  if (pa != pb) return true;
  // row i of a and row j of b share memory where -lb < by + (j - i) pa < la: the least
  // such j - i, of -T + 1 .. T - 1
  const wide n = -lb - by, down = n >= 0 ? n / pa : -((-n + pa - 1) / pa);
  const wide k = down + 1 > 1 - T ? down + 1 : 1 - T;
  return k < T && by + k * pa < la;
}
bool in_place(const RowMat& a, const RowMat& b) { return a.p == b.p && a.ld == b.ld && a.dt == b.dt; }

// The norm's weights; row: a row of type row_dt that stands in where there are none.
twell_status weights(NormArgs* a, const twell_norm_shape* sh, const void* w, const void* row, int row_dt) {
  a->w = w ? w : row;
  a->w_dt = w ? (int)sh->w_dt : row_dt;
  a->w_given = w != nullptr;
  if ((uintptr_t)w % dt_size(sh->w_dt)) return FAIL(TWELL_EINVAL, "w is not aligned to its elements");
  return TWELL_OK;
}

twell_status dropout(NormArgs* a, const twell_norm_shape* sh, const uint64_t* rng) {
  a->drop = (uint32_t)lrintf(sh->p * 65536.f);
  a->keep_scale = a->drop >= 65536u ? 0.f : 65536.f / (float)(65536u - a->drop);
  a->rng = rng;
  if (a->drop && sh->T > 0 && !rng) return FAIL(TWELL_EINVAL, "dropout needs rng");
  if ((uintptr_t)rng % 8) return FAIL(TWELL_EINVAL, "rng is not aligned to its elements");
  return TWELL_OK;
}

NormArgs args_of(const twell_norm_shape* sh) {
  NormArgs a{};
  a.T = sh->T;
  a.d = sh->d;
  a.eps = sh->eps;
  return a;
}

// One 4-bit weight matrix.
twell_status w4(W4View* v, const twell_w4* W, const char* name) {
  if (!W) return FAIL(TWELL_EINVAL, "%s is NULL", name);
  if (W->N <= 0 || W->K <= 0) return FAIL(TWELL_EINVAL, "bad %s: N=%d K=%d", name, W->N, W->K);
  if (W->K % 32) return FAIL(TWELL_EUNSUPPORTED, "%s: K=%d is not a multiple of 32", name, W->K);
  if (W->K >= 1 << 30) return FAIL(TWELL_EUNSUPPORTED, "%s: K=%d is not below 2^30", name, W->K);
  if (!W->codes || !W->scales) return FAIL(TWELL_EINVAL, "%s: NULL array", name);
  if ((uintptr_t)W->codes % 16) return FAIL(TWELL_EINVAL, "%s: codes are not 16-byte aligned", name);
  v->code = W->codes;
  v->scale = W->scales;
  return TWELL_OK;
}

bool token_dt(int dt) { return dt == TWELL_BF16 || dt == TWELL_MXFP8; }

// Activations of a product with 4-bit weights, of a type that token_dt takes.
twell_status tokens(W4Args* a, const void* x, int x_dt, const uint8_t* x_scale) {
  if ((x_dt == TWELL_MXFP8) != (x_scale != nullptr))
    return FAIL(TWELL_EINVAL, "x_scale goes with an MXFP8 x and with no other");
  if ((uintptr_t)x % dt_size(x_dt)) return FAIL(TWELL_EINVAL, "x is not aligned to its elements");
  a->x = x;
  a->x_scale = x_scale;
  return TWELL_OK;
}

#define CHECK(call) \
  if (twell_status st_ = (call)) return st_

}  // namespace

extern "C" {

twell_status twell_add_rmsnorm_fwd(const twell_norm_shape* sh, const void* x, int64_t ldx, const void* residual,
                                   int64_t ldres, const void* w, const uint64_t* rng, void* sum, int64_t ldsum,
                                   void* y, int64_t ldy, uint8_t* y_scale, float* rstd, hipStream_t stream) {
  CHECK(check_norm_shape(sh, true));
  if (sh->T == 0) return TWELL_OK;
  NormArgs a = args_of(sh);
  CHECK(mat(&a.x, sh, x, ldx, sh->x_dt, "x"));
  CHECK(mat(&a.res, sh, residual, ldres, sh->res_dt, "residual"));
  CHECK(mat(&a.sum, sh, sum, ldsum, sh->res_dt, "sum"));
  CHECK(mat(&a.y, sh, y, ldy, sh->y_dt, "y"));
  CHECK(weights(&a, sh, w, x, sh->x_dt));
  CHECK(dropout(&a, sh, rng));
  if (!x || !y) return FAIL(TWELL_EINVAL, "NULL tensor argument");
  if (!sum && (residual || a.drop)) return FAIL(TWELL_EINVAL, "sum is required with a residual or dropout");
  if ((sh->y_dt == TWELL_MXFP8) != (y_scale != nullptr))
    return FAIL(TWELL_EINVAL, "y_scale goes with an MXFP8 y and with no other");
  if ((uintptr_t)rstd % 4) return FAIL(TWELL_EINVAL, "rstd is not aligned to its elements");
  a.y_scale = y_scale;
  a.rstd = rstd;
  return hip_status(launch_norm_fwd(a, stream), "residual sum and norm");
}

size_t twell_add_rmsnorm_bwd_workspace(const twell_norm_shape* sh) {
  if (check_norm_shape(sh, false) != TWELL_OK) return 0;
  return (size_t)norm_bwd_parts(sh->T, sh->d) * sh->d * 4;
}

twell_status twell_add_rmsnorm_bwd(const twell_norm_shape* sh, const void* dy, int64_t lddy, const void* dsum,
                                   int64_t lddsum, const void* sum, int64_t ldsum, const void* w, const float* rstd,
                                   const uint64_t* rng, void* dres, int64_t lddres, void* dx, int64_t lddx,
                                   float* dw, void* ws, size_t ws_bytes, hipStream_t stream) {
  CHECK(check_norm_shape(sh, false));
  NormArgs a = args_of(sh);
  CHECK(mat(&a.y, sh, dy, lddy, sh->y_dt, "dy"));
  CHECK(mat(&a.res, sh, dsum, lddsum, sh->res_dt, "dsum"));
  CHECK(mat(&a.sum, sh, sum, ldsum, sh->res_dt, "sum"));
  CHECK(mat(&a.dres, sh, dres, lddres, sh->res_dt, "dres"));
  CHECK(mat(&a.x, sh, dx, lddx, sh->x_dt, "dx"));
  CHECK(weights(&a, sh, w, sum, sh->res_dt));
  CHECK(dropout(&a, sh, rng));
  if (sh->T > 0 && (!dy || !sum || !rstd || (!dres && !dx))) return FAIL(TWELL_EINVAL, "NULL tensor argument");
  if ((uintptr_t)rstd % 4 || (uintptr_t)dw % 4) return FAIL(TWELL_EINVAL, "rstd or dw is not aligned to its elements");
  if (dw && sh->T > 0) {
    const size_t need = twell_add_rmsnorm_bwd_workspace(sh);
    if (!ws || ws_bytes < need) return FAIL(TWELL_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    if ((uintptr_t)ws % 16) return FAIL(TWELL_EINVAL, "the workspace must be 16-byte aligned");
  }
  if (sh->T == 0 && !dw) return TWELL_OK;
  const RowMat in[] = {a.y, a.res, a.sum};
  for (const RowMat& o : {a.dres, a.x})
    for (const RowMat& i : in)
      if (overlap(o, i, sh->T, sh->d) && !in_place(o, i))
        return FAIL(TWELL_EINVAL, "dres or dx overlaps dy, dsum or sum and is not written in place");
  if (overlap(a.dres, a.x, sh->T, sh->d)) return FAIL(TWELL_EINVAL, "dres and dx overlap");
  a.dw_may_reread = true;
  for (const RowMat& o : {a.dres, a.x})
    for (const RowMat& i : {a.y, a.sum})
      if (o.p && o.p == i.p) a.dw_may_reread = false;
  a.rstd_in = rstd;
  a.dw = dw;
  a.part = (float*)ws;
  return hip_status(launch_norm_bwd(a, stream), "residual sum and norm backward");
}

twell_status twell_dropout_add(const twell_norm_shape* sh, const void* x, int64_t ldx, const void* residual,
                               int64_t ldres, const uint64_t* rng, void* y, int64_t ldy, hipStream_t stream) {
  CHECK(check_norm_shape(sh, false));
  if (sh->T == 0) return TWELL_OK;
  NormArgs a = args_of(sh);
  CHECK(mat(&a.x, sh, x, ldx, sh->x_dt, "x"));
  CHECK(mat(&a.res, sh, residual, ldres, sh->res_dt, "residual"));
  CHECK(mat(&a.y, sh, y, ldy, sh->y_dt, "y"));
  CHECK(dropout(&a, sh, rng));
  if (!x || !y) return FAIL(TWELL_EINVAL, "NULL tensor argument");
  return hip_status(launch_dropout_add(a, stream), "dropout");
}

twell_status twell_w4_matvec(int32_t T, const void* x, twell_dtype x_dt, int64_t ldx, const uint8_t* x_scale,
                             const twell_w4* W, const void* bias, void* y, twell_dtype y_dt, int64_t ldy,
                             hipStream_t stream) {
  W4Args a{};
  if (T < 0) return FAIL(TWELL_EINVAL, "bad T=%d", T);
  CHECK(w4(&a.W, W, "W"));
  if (!token_dt(x_dt)) return FAIL(TWELL_EINVAL, "x must be BF16 or MXFP8");
  if (!float_dt(y_dt)) return FAIL(TWELL_EINVAL, "y must be F32 or BF16");
  if (T == 0) return TWELL_OK;
  CHECK(tokens(&a, x, x_dt, x_scale));
  if ((uintptr_t)y % dt_size(y_dt) || (uintptr_t)bias % 2)
    return FAIL(TWELL_EINVAL, "y or bias is not aligned to its elements");
  if (!x || !y) return FAIL(TWELL_EINVAL, "NULL tensor argument");
  if (T > 1 && (ldx < W->K || ldy < W->N))
    return FAIL(TWELL_EINVAL, "row stride of x (%lld) or y (%lld) below K=%d or N=%d", (long long)ldx, (long long)ldy,
                W->K, W->N);
  a.T = T;
  a.N = W->N;
  a.K = W->K;
  a.ldx = T > 1 ? ldx : W->K;
  a.ldy = T > 1 ? ldy : W->N;
  a.bias = (const uint16_t*)bias;
  a.y = y;
  a.y_bf16 = y_dt == TWELL_BF16;
  return hip_status(launch_w4_matvec(a, stream), "4-bit product");
}

static twell_status check_ffn_w4_shape(const twell_ffn_shape* sh) {
  if (!sh) return FAIL(TWELL_EINVAL, "shape is NULL");
  if (sh->T < 0 || sh->d <= 0 || sh->F <= 0) return FAIL(TWELL_EINVAL, "bad shape T=%d d=%d F=%d", sh->T, sh->d, sh->F);
  if (!token_dt(sh->in_dt) || !float_dt(sh->out_dt))
    return FAIL(TWELL_EINVAL, "bad dtype (x BF16 or MXFP8, y F32 or BF16)");
  if (sh->d % 64 || sh->F % 64) return FAIL(TWELL_EUNSUPPORTED, "d=%d and F=%d must be multiples of 64", sh->d, sh->F);
  const int64_t lim = (int64_t)1 << 31;
  if ((int64_t)sh->T * sh->d >= lim || (int64_t)sh->T * sh->F >= lim || (int64_t)sh->F * sh->d >= lim)
    return FAIL(TWELL_EUNSUPPORTED, "T*d, T*F and F*d must be below 2^31");
  return TWELL_OK;
}

size_t twell_ffn_fwd_w4_workspace(const twell_ffn_shape* sh) {
  return check_ffn_w4_shape(sh) == TWELL_OK ? ffn_w4_ws_bytes(sh->T, sh->d, sh->F) : 0;
}

twell_status twell_ffn_fwd_w4(const twell_ffn_shape* sh, const void* x, const uint8_t* x_scale, const twell_w4* Wg,
                              const void* bg, const twell_w4* Wu, const twell_w4* Wd, void* y, void* ws,
                              size_t ws_bytes, hipStream_t stream) {
  CHECK(check_ffn_w4_shape(sh));
  if (sh->T == 0) return TWELL_OK;
  W4Args a{};
  CHECK(w4(&a.W, Wg, "Wg"));
  CHECK(w4(&a.Wu, Wu, "Wu"));
  CHECK(w4(&a.Wd, Wd, "Wd"));
  for (const twell_w4* W : {Wg, Wu, Wd})
    if (W->N != sh->F || W->K != sh->d)
      return FAIL(TWELL_EINVAL, "a weight matrix is [%d][%d], not [F=%d][d=%d]", W->N, W->K, sh->F, sh->d);
  CHECK(tokens(&a, x, sh->in_dt, x_scale));
  if (!x || !y) return FAIL(TWELL_EINVAL, "NULL tensor argument");
  if ((uintptr_t)y % dt_size(sh->out_dt) || (uintptr_t)bg % 2)
    return FAIL(TWELL_EINVAL, "y or bg is not aligned to its elements");
  const size_t need = ffn_w4_ws_bytes(sh->T, sh->d, sh->F);
  if (!ws || ws_bytes < need) return FAIL(TWELL_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
  if ((uintptr_t)ws % 16) return FAIL(TWELL_EINVAL, "the workspace must be 16-byte aligned");
  a.T = sh->T;
  a.N = sh->F;
  a.K = sh->d;
  a.ldx = a.ldy = sh->d;
  a.bias = (const uint16_t*)bg;
  a.y = y;
  a.y_bf16 = sh->out_dt == TWELL_BF16;
  return hip_status(launch_ffn_w4(a, ws, stream), "layer on 4-bit weights");
}

}  // extern "C"
