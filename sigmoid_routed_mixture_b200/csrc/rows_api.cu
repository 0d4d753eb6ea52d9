// rows_api.cu -- host side of the C ABI declared in include/srm_rows.h:
// validation and the launches of the row kernels (rows.cu), asynchronous on
// the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/srm_rows.h"
#include "host_util.h"
#include "kernels.h"

namespace {

using namespace srm::host;

moe_status_t check(const moe_rows_cfg_t *c, bool int8_rows, bool slots) {
  if (!c) return MOE_ERR_ARG;
  const bool one_group = c->E == 0 && c->K == 0 && c->has_shared == 1;
  if (c->T < 0 || c->H < 1 || (!one_group && (c->E < 1 || c->K < 1 || c->K > c->E))) return MOE_ERR_ARG;
  if (c->has_shared != 0 && c->has_shared != 1) return MOE_ERR_ARG;
  if (!float_dtype(c->dtype) && !(int8_rows && c->dtype == MOE_DTYPE_INT8)) return MOE_ERR_ARG;
  if (slots && !float_dtype(c->slot_dtype)) return MOE_ERR_ARG;
  if (c->E > 256 || c->K > 16 || c->H > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (c->T >= (int64_t(1) << 31) || c->T * (c->K + 1) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// strides x rows stay far inside 64 bits
bool good_ld(const moe_rows_cfg_t *c, int64_t ld) { return ld >= c->H && ld <= (int64_t(1) << 31); }

srm::RowsArgs args(const moe_rows_cfg_t &c, void *ws) {
  srm::RowsArgs a;
  a.T = static_cast<int>(c.T);
  a.H = c.H;
  a.E = c.E;
  a.K = c.K;
  a.has_shared = c.has_shared;
  a.P = static_cast<int>(c.T * c.K + c.T * c.has_shared);
  a.ld_token = c.ld_token;
  a.ld_slot = c.ld_slot;
  a.ld_residual = c.ld_residual;
  a.ld_dys = c.ld_dys;
  a.err = static_cast<int *>(ws);
  return a;
}

}  // namespace

extern "C" {

moe_status_t moe_rows_sort(const moe_rows_cfg_t *cfg, const void *x, const float *x_scale,
                           const int32_t *offsets, const int32_t *sorted, int32_t *pos, void *xs,
                           float *xs_scale, void *ws, void *stream) {
  moe_status_t st = check(cfg, true, false);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!x || !offsets || !sorted || !pos || !xs || !ws) return MOE_ERR_ARG;
  if ((x_scale == nullptr) != (xs_scale == nullptr)) return MOE_ERR_ARG;
  if (!good_ld(cfg, cfg->ld_token) || !good_ld(cfg, cfg->ld_slot)) return MOE_ERR_ARG;
  const size_t e = dtype_size(cfg->dtype);
  if (!aligned(x, e) || !aligned(xs, e) || !aligned(offsets, 4) || !aligned(sorted, 4) || !aligned(pos, 4) ||
      (x_scale && (!aligned(x_scale, 4) || !aligned(xs_scale, 4))) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  return cuda_status(srm::launch_rows_sort(args(*cfg, ws), static_cast<int>(e), x, x_scale, offsets, sorted,
                                           pos, xs, xs_scale, num_sms(), static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rows_unsort(const moe_rows_cfg_t *cfg, const void *ys, const float *gate,
                             const int32_t *pos, const void *residual, void *y, void *ws, void *stream) {
  moe_status_t st = check(cfg, false, true);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ys || !pos || !y || !ws) return MOE_ERR_ARG;
  if (!good_ld(cfg, cfg->ld_token) || !good_ld(cfg, cfg->ld_slot) ||
      (residual && !good_ld(cfg, cfg->ld_residual)) ||
      (residual == y && cfg->T > 1 && cfg->ld_residual != cfg->ld_token))
    return MOE_ERR_ARG;
  const size_t e = dtype_size(cfg->dtype);
  if (!aligned(ys, dtype_size(cfg->slot_dtype)) || (gate && !aligned(gate, 4)) || !aligned(pos, 4) ||
      (residual && !aligned(residual, e)) || !aligned(y, e) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  return cuda_status(srm::launch_rows_unsort(args(*cfg, ws), cfg->dtype, cfg->slot_dtype, ys, gate, pos,
                                             residual, y, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_rows_sort_grad(const moe_rows_cfg_t *cfg, const void *dxs, const int32_t *pos, void *dx,
                                void *ws, void *stream) {
  // the sorted rows' gradients summed with weights 1: unsort's sum, rows of dtype
  if (!cfg) return MOE_ERR_ARG;
  moe_rows_cfg_t c = *cfg;
  c.slot_dtype = c.dtype;
  return moe_rows_unsort(&c, dxs, nullptr, pos, nullptr, dx, ws, stream);
}

moe_status_t moe_rows_unsort_grad(const moe_rows_cfg_t *cfg, const void *dy, const void *ys,
                                  const float *gate, const int32_t *pos, void *dys, float *dgate, void *ws,
                                  void *stream) {
  moe_status_t st = check(cfg, false, true);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!dy || !pos || !ws || (!dys && !dgate) || (dgate && !ys)) return MOE_ERR_ARG;
  if (!good_ld(cfg, cfg->ld_token) || (dgate && !good_ld(cfg, cfg->ld_slot)) ||
      (dys && !good_ld(cfg, cfg->ld_dys)) || (dys && dgate && dys == ys && cfg->ld_dys != cfg->ld_slot))
    return MOE_ERR_ARG;
  const size_t es = dtype_size(cfg->slot_dtype);
  if (!aligned(dy, dtype_size(cfg->dtype)) || (ys && !aligned(ys, es)) || (gate && !aligned(gate, 4)) ||
      !aligned(pos, 4) || (dys && !aligned(dys, es)) || (dgate && !aligned(dgate, 4)) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  return cuda_status(srm::launch_rows_unsort_grad(args(*cfg, ws), cfg->dtype, cfg->slot_dtype, dy, ys, gate,
                                                  pos, dys, dgate, num_sms(),
                                                  static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
