// C-ABI entry points of the operators around the layer (residual sum, norm and
// dropout): argument checks on the host, then kernel launches on the caller's
// stream.  No allocation, no synchronisation.
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

twell_status weights(NormArgs* a, const twell_norm_shape* sh, const void* w) {
  a->w = w;
  a->w_dt = sh->w_dt;
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
  CHECK(weights(&a, sh, w));
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
  CHECK(weights(&a, sh, w));
  CHECK(dropout(&a, sh, rng));
  if (sh->T > 0 && (!dy || !sum || !rstd || (!dres && !dx))) return FAIL(TWELL_EINVAL, "NULL tensor argument");
  if ((uintptr_t)rstd % 4 || (uintptr_t)dw % 4) return FAIL(TWELL_EINVAL, "rstd or dw is not aligned to its elements");
  if (dw && sh->T > 0) {
    const size_t need = twell_add_rmsnorm_bwd_workspace(sh);
    if (!ws || ws_bytes < need) return FAIL(TWELL_EWORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes, need);
    if ((uintptr_t)ws % 16) return FAIL(TWELL_EINVAL, "the workspace must be 16-byte aligned");
  }
  if (sh->T == 0 && !dw) return TWELL_OK;
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

}  // extern "C"
