// q8_api.cu -- host side of the C ABI declared in include/srm_q8.h:
// validation and the launches of the 8-bit row and product kernels
// (q8_norm.cu, q8_gemm.cu), asynchronous on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include "../../include/srm_q8.h"
#include "host_util.h"
#include "kernels.h"

namespace {

using namespace srm::host;

constexpr int64_t kMaxLd = int64_t(1) << 40;  // strides x rows stay far inside 64 bits

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
  // a result in an input's place has its rows where the input has them
  auto same_rows = [&](const void *out, int64_t ld_out) {
    return !out || cfg->T < 2 || ((out != x || ld_out == cfg->ld_x) && (out != delta || ld_out == cfg->ld_delta));
  };
  if (!same_rows(x_sum, cfg->ld_sum) || !same_rows(y, cfg->ld_y)) return MOE_ERR_ARG;
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

moe_status_t check_matmul(const moe_q8_matmul_t *c) {
  if (!c) return MOE_ERR_ARG;
  if (c->R < 0 || c->N < 1 || c->K < 1 || c->groups < 1 || !float_dtype(c->dtype)) return MOE_ERR_ARG;
  if (c->swiglu != 0 && c->swiglu != 1) return MOE_ERR_ARG;
  if (c->K % 16 != 0 || c->K > 65536 || (c->swiglu && c->N % 32 != 0)) return MOE_ERR_UNSUPPORTED;
  // rows and channels are 32-bit numbers, up to a tile's end
  if (c->groups > srm::kQ8MaxGroups || c->R >= (int64_t(1) << 31) - 1024 ||
      static_cast<int64_t>(c->groups) * c->N > (int64_t(1) << 31) - 256)
    return MOE_ERR_UNSUPPORTED;
  // tile numbers are 32-bit
  const srm::Q8Plan p = srm::q8_plan(c->R, c->N, c->K, c->groups, num_sms());
  if (p.max_mtiles * ((c->N + 127) / 128) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Workspace: control words (the device error word at 0, the tile counter at
// 64, the ready word at 128, from 256 on the part counters), then the partial
// sums.  The control words have the same place in every workspace, so that one
// serves products of several shapes in turn.
constexpr size_t kReadyOffset = 128, kPartCounters = 256;
size_t control_bytes() {
  // cut tiles are no more than the units (a CTA, or two), with a counter for
  // each epilogue warp of each CTA of a tile
  return kPartCounters + sizeof(unsigned) * srm::kQ8EpiWarps * static_cast<size_t>((num_sms() + 31) / 32 * 32);
}
size_t matmul_ws_bytes(int64_t R) {
  return control_bytes() + sizeof(int32_t) * static_cast<size_t>(srm::q8_partials(R, num_sms()));
}

}  // namespace

extern "C" {

size_t moe_q8_matmul_workspace_size(const moe_q8_matmul_t *cfg) {
  if (check_matmul(cfg) != MOE_OK) return 0;
  return matmul_ws_bytes(cfg->R);
}

moe_status_t moe_q8_workspace_init(void *ws, size_t ws_bytes, void *stream) {
  if (!ws) return MOE_ERR_ARG;
  if (!aligned(ws, 256)) return MOE_ERR_ALIGN;
  if (ws_bytes < control_bytes()) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int byte = srm::kQ8Ready & 0xff;  // kQ8Ready is four times the same byte
  if (cudaMemsetAsync(ws, 0, control_bytes(), s) != cudaSuccess ||
      cudaMemsetAsync(static_cast<uint8_t *>(ws) + kReadyOffset, byte, sizeof(int), s) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status_t moe_q8_matmul(const moe_q8_matmul_t *cfg, const int8_t *x, const float *x_scale,
                           const int8_t *w, const float *w_scale, const int32_t *offsets,
                           const void *residual, void *y, void *ws, size_t ws_bytes, void *stream) {
  moe_status_t st = check_matmul(cfg);
  if (st != MOE_OK || cfg->R == 0) return st;
  if (!x || !x_scale || !w || !w_scale || !y || !ws || (cfg->groups > 1 && !offsets)) return MOE_ERR_ARG;
  if (residual && cfg->swiglu) return MOE_ERR_ARG;
  const int64_t cols = cfg->swiglu ? cfg->N / 2 : cfg->N;
  if (!good_ld(cfg->ld_x, cfg->K) || !good_ld(cfg->ld_y, cols) ||
      (residual && !good_ld(cfg->ld_residual, cols)) ||
      (residual == y && cfg->R > 1 && cfg->ld_residual != cfg->ld_y))
    return MOE_ERR_ARG;
  const size_t e = dtype_size(cfg->dtype);
  if (!aligned(x, 16) || cfg->ld_x % 16 != 0 || !aligned(w, 16) || !aligned(x_scale, 4) ||
      !aligned(w_scale, 4) || (offsets && !aligned(offsets, 4)) || (residual && !aligned(residual, e)) ||
      !aligned(y, e) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  const srm::Q8Plan plan = srm::q8_plan(cfg->R, cfg->N, cfg->K, cfg->groups, num_sms());
  if (ws_bytes < matmul_ws_bytes(cfg->R)) return MOE_ERR_WORKSPACE;
  uint8_t *wsb = static_cast<uint8_t *>(ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  srm::Q8Maps maps;
  const uint64_t K = cfg->K, R = cfg->R, pitch = cfg->ld_x;
  bool ok = make_tmap_8bit(&maps.w, w, K, static_cast<uint64_t>(cfg->groups) * cfg->N, K, 128);
  for (int i = 0; i < 3; ++i) ok = ok && make_tmap_8bit(&maps.tok[i], x, K, R, pitch, 32u << i);
  if (!ok) return MOE_ERR_CUDA;
  srm::Q8GemmArgs p = {};
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.offsets = offsets;
  p.residual = residual;
  p.y = y;
  p.ld_residual = cfg->ld_residual;
  p.ld_y = cfg->ld_y;
  p.err = reinterpret_cast<int *>(wsb);
  p.ready = reinterpret_cast<int *>(wsb + kReadyOffset);
  p.tile_counter = reinterpret_cast<unsigned *>(wsb + 64);
  p.part_counter = reinterpret_cast<unsigned *>(wsb + kPartCounters);
  p.partial = reinterpret_cast<int32_t *>(wsb + control_bytes());
  p.R = static_cast<int>(cfg->R);
  p.N = cfg->N;
  p.K = cfg->K;
  p.groups = cfg->groups;
  p.units = plan.units;
  p.max_parts = plan.max_parts;
  p.max_mtiles = static_cast<int>(plan.max_mtiles);
  const char *inject = getenv("SRM_MOE_INJECT_STALL");
  p.stall = (inject && inject[0] == '1') ? 1 : 0;
  return cuda_status(srm::launch_q8_gemm(cfg->swiglu != 0, cfg->dtype, plan.pair, maps, p, num_sms(), s));
}

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
                                               static_cast<cudaStream_t>(stream)));
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
