// q8_api.cu -- host side of the C ABI declared in include/srm_q8.h:
// validation and the launches of the 8-bit row and product kernels
// (q8_norm.cu, q8_gemm.cu), asynchronous on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/srm_q8.h"
#include "host_util.h"
#include "kernels.h"

namespace {

using namespace srm::host;

constexpr int64_t kMaxLd = int64_t(1) << 40;  // strides x rows stay far inside 64 bits

size_t dtype_size(int32_t d) {
  return d == MOE_DTYPE_FP32 ? 4 : d == MOE_DTYPE_INT8 ? 1 : 2;
}

bool float_dtype(int32_t d) {
  return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_FP16 || d == MOE_DTYPE_FP32;
}

bool good_ld(int64_t ld, int64_t h) { return ld >= h && ld <= kMaxLd; }

moe_status_t check_rows(const moe_q8_rows_t *c) {
  if (!c) return MOE_ERR_ARG;
  if (c->T < 0 || c->H < 1 || !float_dtype(c->dtype)) return MOE_ERR_ARG;
  if (c->H > (1 << 20) || c->T >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t run_rows(const moe_q8_rows_t *cfg, const void *x, const void *delta, const void *gamma,
                      float eps, void *x_sum, void *y, int8_t *q, float *scale, cudaStream_t s) {
  if (!x || !q || !scale) return MOE_ERR_ARG;
  if (!good_ld(cfg->ld_x, cfg->H) || !good_ld(cfg->ld_q, cfg->H) ||
      (delta && !good_ld(cfg->ld_delta, cfg->H)) || (x_sum && !good_ld(cfg->ld_sum, cfg->H)) ||
      (y && !good_ld(cfg->ld_y, cfg->H)))
    return MOE_ERR_ARG;
  if (y && y == x_sum) return MOE_ERR_ARG;  // two results in one place
  const size_t e = dtype_size(cfg->dtype);
  const void *ptrs[] = {x, delta, gamma, x_sum, y};
  for (const void *p : ptrs)
    if (p && !aligned(p, e)) return MOE_ERR_ALIGN;
  if (!aligned(scale, 4)) return MOE_ERR_ALIGN;
  srm::Q8RowArgs a = {};
  a.x = x;
  a.delta = delta;
  a.gamma = gamma;
  a.x_sum = x_sum;
  a.y = y;
  a.q = q;
  a.scale = scale;
  a.T = cfg->T;
  a.H = cfg->H;
  a.ld_x = cfg->ld_x;
  a.ld_delta = cfg->ld_delta;
  a.ld_sum = cfg->ld_sum;
  a.ld_y = cfg->ld_y;
  a.ld_q = cfg->ld_q;
  a.eps = eps;
  a.unit_offset = -1;
  return cuda_status(srm::launch_q8_rows(cfg->dtype, a, num_sms(), s));
}

}  // namespace

extern "C" {

moe_status_t moe_q8_add_rmsnorm(const moe_q8_rows_t *cfg, const void *x, const void *delta,
                                const void *gamma, float eps, void *x_sum, void *y, int8_t *q,
                                float *scale, void *stream) {
  moe_status_t st = check_rows(cfg);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f) || !isfinite(eps)) return MOE_ERR_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!gamma) return MOE_ERR_ARG;
  return run_rows(cfg, x, delta, gamma, eps, x_sum, y, q, scale, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_q8_quantize(const moe_q8_rows_t *cfg, const void *x, int8_t *q, float *scale,
                             void *stream) {
  moe_status_t st = check_rows(cfg);
  if (st != MOE_OK || cfg->T == 0) return st;
  return run_rows(cfg, x, nullptr, nullptr, 0.f, nullptr, nullptr, q, scale,
                  static_cast<cudaStream_t>(stream));
}

moe_status_t moe_q8_dequantize(const moe_q8_rows_t *cfg, const int8_t *q, const float *scale, void *y,
                               void *stream) {
  moe_status_t st = check_rows(cfg);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!q || !scale || !y) return MOE_ERR_ARG;
  if (!good_ld(cfg->ld_q, cfg->H) || !good_ld(cfg->ld_y, cfg->H)) return MOE_ERR_ARG;
  if (!aligned(y, dtype_size(cfg->dtype)) || !aligned(scale, 4)) return MOE_ERR_ALIGN;
  return cuda_status(srm::launch_q8_dequantize(cfg->dtype, q, scale, y, cfg->T, cfg->H, cfg->ld_q, cfg->ld_y,
                                               num_sms(), static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_q8_pack_weights(const moe_cfg_t *cfg, const void *w1, const void *w3, const void *w2,
                                 const void *ws1, const void *ws3, const void *ws2, int8_t *w13_q,
                                 float *w13_scale, int8_t *w2_q, float *w2_scale, void *stream) {
  moe_status_t st = srm::check_block_cfg(cfg);
  if (st != MOE_OK) return st;
  if (!w13_q || !w13_scale || !w2_q || !w2_scale || (cfg->E > 0 && (!w1 || !w3 || !w2)) ||
      (cfg->has_shared && (!ws1 || !ws3 || !ws2)))
    return MOE_ERR_ARG;
  const void *ptrs[] = {w1, w3, w2, ws1, ws3, ws2, w13_q, w2_q};
  for (const void *p : ptrs)
    if (p && !aligned(p, 16)) return MOE_ERR_ALIGN;
  if (!aligned(w13_scale, 4) || !aligned(w2_scale, 4)) return MOE_ERR_ALIGN;
  const int64_t E = cfg->E, H = cfg->H, I = cfg->I;
  auto pack = [&](const void *w, int64_t rows, int64_t cols, int8_t *q, float *scale, int unit_offset) {
    if (rows == 0) return cudaSuccess;
    srm::Q8RowArgs a = {};
    a.x = w;
    a.q = q;
    a.scale = scale;
    a.T = rows;
    a.H = static_cast<int>(cols);
    a.ld_x = a.ld_q = cols;
    a.unit_offset = unit_offset;
    return srm::launch_q8_rows(MOE_DTYPE_BF16, a, num_sms(), static_cast<cudaStream_t>(stream));
  };
  struct {
    const void *w1, *w3, *w2;
    int64_t first, n;
  } parts[] = {{w1, w3, w2, 0, E}, {ws1, ws3, ws2, E, cfg->has_shared ? 1 : 0}};
  for (const auto &p : parts) {
    int8_t *up = w13_q + p.first * 2 * I * H;
    float *up_scale = w13_scale + p.first * 2 * I;
    if (pack(p.w1, p.n * I, H, up, up_scale, 0) != cudaSuccess ||
        pack(p.w3, p.n * I, H, up, up_scale, 16) != cudaSuccess ||
        pack(p.w2, p.n * H, I, w2_q + p.first * H * I, w2_scale + p.first * H, -1) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
