// rows.cu -- token rows to the experts' order and back with the routing
// weights applied, and the gradients of both (formulas: include/srm_rows.h).
//
// All of it is bound by memory: each token row is read once and each sorted
// row written once, or the reverse; the gradient of the way back reads dy once
// for all of a token's slots.  No atomics: every output element is the work of
// one thread, and a sum over slots or over a row runs in a fixed order.
#include "kernels.h"
#include "rowio.cuh"

namespace srm {

namespace {

// Eight elements of a row as fp32 values (16-byte loads), or one element for
// rows that are not 16-byte aligned.
template <typename T, int E>
struct Unit;
template <typename T>
struct Unit<T, 8> {  // 16-bit types
  uint4 r;
  __device__ __forceinline__ void load(const T *p) { r = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const { RowIo<T, 8>::unpack(r, f); }
  static __device__ __forceinline__ void store(T *p, const float (&f)[8]) { RowIo<T, 8>::store(p, f); }
};
template <>
struct Unit<float, 8> {
  uint4 r, r2;
  __device__ __forceinline__ void load(const float *p) {
    r = reinterpret_cast<const uint4 *>(p)[0];
    r2 = reinterpret_cast<const uint4 *>(p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
    f[4] = __uint_as_float(r2.x);
    f[5] = __uint_as_float(r2.y);
    f[6] = __uint_as_float(r2.z);
    f[7] = __uint_as_float(r2.w);
  }
  static __device__ __forceinline__ void store(float *p, const float (&f)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <typename T>
struct Unit<T, 1> {
  T r;
  __device__ __forceinline__ void load(const T *p) { r = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_float(r); }
  static __device__ __forceinline__ void store(T *p, const float (&f)[1]) { *p = from_float<T>(f[0]); }
};

// The number of positions that hold a row: offsets[E + 1], or 0 (flagged) when
// it is no count of rows.
__device__ __forceinline__ int row_total(const int32_t *offsets, int groups_end, int P, int *err) {
  const int n = offsets[groups_end];
  if (n >= 0 && n <= P) return n;
  record_error(err, MOE_ERR_BAD_INDEX);
  return 0;
}

// pos[a] as a position in [0, P), or -1.
__device__ __forceinline__ int row_pos(const int32_t *pos, int a, int P, int *err) {
  const int p = pos[a];
  if (p >= -1 && p < P) return p;
  record_error(err, MOE_ERR_BAD_INDEX);
  return -1;
}

constexpr int kBatch = 8;  // vectors a lane has in flight

}  // namespace

// pos[sorted[p]] = p over the positions that hold a row (pos is -1 before).
__global__ void __launch_bounds__(256)
    rows_invert_kernel(const RowsArgs p, const int32_t *__restrict__ offsets,
                       const int32_t *__restrict__ sorted, int32_t *__restrict__ pos) {
  const int n = row_total(offsets, p.E + 1, p.P, p.err);
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    const int a = sorted[i];
    if (a < 0 || a >= p.P)
      record_error(p.err, MOE_ERR_BAD_INDEX);
    else
      pos[a] = i;
  }
}

// The rows by token: each token row is read once and written to its positions.
// W: the widest vector all rows are aligned to; a warp moves a part of a row.
template <typename W>
__global__ void __launch_bounds__(256)
    rows_scatter_kernel(const RowsArgs p, const int32_t *__restrict__ pos, const uint8_t *__restrict__ x,
                        uint8_t *__restrict__ xs, const float *__restrict__ x_scale,
                        float *__restrict__ xs_scale, int64_t row_bytes, int64_t x_pitch, int64_t xs_pitch,
                        int wpt) {
  const int lane = threadIdx.x & 31;
  const int vecs = static_cast<int>(row_bytes / sizeof(W));
  const int part = (vecs + wpt - 1) / wpt;
  const int64_t jobs = static_cast<int64_t>(p.T) * wpt;
  for (int64_t job = blockIdx.x * 8ll + (threadIdx.x >> 5); job < jobs; job += gridDim.x * 8ll) {
    const int t = static_cast<int>(job / wpt);
    const int begin = static_cast<int>(job - static_cast<int64_t>(t) * wpt) * part;
    const int end = min(vecs, begin + part);
    // lane k holds the token's k-th position, the shared row's behind the slots
    int mine = -1;
    if (lane < p.K)
      mine = row_pos(pos, t * p.K + lane, p.P, p.err);
    else if (lane == p.K && p.has_shared)
      mine = row_pos(pos, p.T * p.K + t, p.P, p.err);
    if (xs_scale && begin == 0 && mine >= 0) xs_scale[mine] = x_scale[t];
    const int n_dst = p.K + p.has_shared;
    const W *src = reinterpret_cast<const W *>(x + t * x_pitch);
    for (int v0 = begin; v0 < end; v0 += 32 * kBatch) {
      W buf[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (v0 + j * 32 + lane < end) buf[j] = src[v0 + j * 32 + lane];
      for (int k = 0; k < n_dst; ++k) {
        const int d = __shfl_sync(0xffffffffu, mine, k);
        if (d < 0) continue;
        W *out = reinterpret_cast<W *>(xs + d * xs_pitch);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (v0 + j * 32 + lane < end) out[v0 + j * 32 + lane] = buf[j];
      }
    }
  }
}

// The way back: y[t] = (residual[t] +) the weighted sum of the token's rows.
// NB: slots and the shared row at most, all loads issued before the sums.
template <typename Tt, typename Ts, int E, int NB>
__global__ void __launch_bounds__(256)
    rows_unsort_kernel(const RowsArgs p, const Ts *__restrict__ ys, const float *__restrict__ gate,
                       const int32_t *__restrict__ pos, const Tt *residual, Tt *y) {
  const int units = (p.H + E - 1) / E;
  const int64_t total = static_cast<int64_t>(p.T) * units;
  const int n = p.K + p.has_shared;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int t = static_cast<int>(i / units);
    const int c = static_cast<int>(i - static_cast<int64_t>(t) * units) * E;
    Unit<Ts, E> v[NB];
    int at[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      at[k] = -1;
      if (k < n) at[k] = row_pos(pos, k < p.K ? t * p.K + k : p.T * p.K + t, p.P, p.err);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k)
      if (at[k] >= 0) v[k].load(ys + at[k] * p.ld_slot + c);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (at[k] < 0) continue;
      const float g = gate && k < p.K ? gate[static_cast<int64_t>(t) * p.K + k] : 1.f;
      float f[E];
      v[k].get(f);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(g, f[e], acc[e]);
    }
    if (residual) {
      Unit<Tt, E> r;
      float f[E];
      r.load(residual + t * p.ld_residual + c);
      r.get(f);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = f[e] + acc[e];
    }
    Unit<Tt, E>::store(y + t * p.ld_token + c, acc);
  }
}

// The gradient of the way back.  WPT warps share a token's row; dy's part
// stays in registers while the token's slots pass.
template <typename Tt, typename Ts, int E, int KM>
__global__ void __launch_bounds__(256)
    rows_unsort_grad_kernel(const RowsArgs p, const Tt *__restrict__ dy, const Ts *ys,
                            const float *__restrict__ gate, const int32_t *__restrict__ pos, Ts *dys,
                            float *dgate, int wpt) {
  constexpr int B = E == 8 && sizeof(Tt) == 4 ? kBatch / 2 : kBatch;
  __shared__ float part[8][KM];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (8 / wpt) + warp / wpt;
  const int w = warp % wpt;
  const int units = (p.H + E - 1) / E;
  const int share = (units + wpt - 1) / wpt;
  const int begin = min(units, w * share), end = min(units, begin + share);
  float dot[KM];
#pragma unroll
  for (int k = 0; k < KM; ++k) dot[k] = 0.f;
  if (t < p.T) {
    int mine = -1;  // lane k: the token's k-th position (k <= 16)
    float my_gate = 1.f;
    if (lane < p.K) {
      mine = row_pos(pos, t * p.K + lane, p.P, p.err);
      if (gate) my_gate = gate[static_cast<int64_t>(t) * p.K + lane];
    } else if (lane == p.K && p.has_shared) {
      mine = row_pos(pos, p.T * p.K + t, p.P, p.err);
    }
    for (int u0 = begin; u0 < end; u0 += 32 * B) {
      Unit<Tt, E> d[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (u0 + j * 32 + lane < end) d[j].load(dy + t * p.ld_token + (u0 + j * 32 + lane) * E);
#pragma unroll
      for (int k = 0; k <= KM; ++k) {
        if (k >= p.K + p.has_shared) break;
        const int at = __shfl_sync(0xffffffffu, mine, k);
        const float g = __shfl_sync(0xffffffffu, my_gate, k);
        if (at < 0) continue;
        if (dgate && k < p.K) {
          Unit<Ts, E> v[B];
#pragma unroll
          for (int j = 0; j < B; ++j)
            if (u0 + j * 32 + lane < end) v[j].load(ys + at * p.ld_slot + (u0 + j * 32 + lane) * E);
          float s = 0.f;
#pragma unroll
          for (int j = 0; j < B; ++j)
            if (u0 + j * 32 + lane < end) {
              float a[E], b[E];
              d[j].get(a);
              v[j].get(b);
#pragma unroll
              for (int e = 0; e < E; ++e) s = fmaf(a[e], b[e], s);
            }
          if (k < KM) dot[k < KM ? k : 0] += s;
        }
        if (dys) {
#pragma unroll
          for (int j = 0; j < B; ++j)
            if (u0 + j * 32 + lane < end) {
              float a[E];
              d[j].get(a);
#pragma unroll
              for (int e = 0; e < E; ++e) a[e] *= g;
              Unit<Ts, E>::store(dys + at * p.ld_dys + (u0 + j * 32 + lane) * E, a);
            }
        }
      }
    }
  }
  if (!dgate) return;
#pragma unroll
  for (int k = 0; k < KM; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
    if (lane == 0) part[warp][k] = dot[k];
  }
  __syncthreads();
  if (t < p.T && w == 0 && lane < p.K) {
    float s = 0.f;
    for (int j = 0; j < wpt; ++j) s += part[warp + j][lane];
    dgate[static_cast<int64_t>(t) * p.K + lane] = s;
  }
}

namespace {

bool is_aligned(const void *p, int64_t pitch_bytes, int a) {
  return !p || (reinterpret_cast<uintptr_t>(p) % a == 0 && pitch_bytes % a == 0);
}

template <typename W>
cudaError_t launch_scatter(const RowsArgs &p, const int32_t *pos, const void *x, void *xs,
                           const float *x_scale, float *xs_scale, int elem, int num_sms,
                           cudaStream_t stream) {
  int wpt = 1;  // warps per token: at least ~32 warps per SM in flight
  while (wpt < 8 && static_cast<int64_t>(p.T) * wpt < num_sms * 32) wpt *= 2;
  const int64_t blocks = (static_cast<int64_t>(p.T) * wpt + 7) / 8, cap = num_sms * 16ll;
  rows_scatter_kernel<W><<<static_cast<unsigned>(blocks < cap ? blocks : cap), 256, 0, stream>>>(
      p, pos, static_cast<const uint8_t *>(x), static_cast<uint8_t *>(xs), x_scale, xs_scale,
      static_cast<int64_t>(p.H) * elem, p.ld_token * elem, p.ld_slot * elem, wpt);
  return cudaGetLastError();
}

template <typename Tt, typename Ts, int E>
cudaError_t launch_unsort_e(const RowsArgs &p, const void *ys, const float *gate, const int32_t *pos,
                            const void *residual, void *y, int num_sms, cudaStream_t stream) {
  const int64_t total = static_cast<int64_t>(p.T) * ((p.H + E - 1) / E);
  const int64_t blocks = (total + 255) / 256, cap = num_sms * 32ll;
  const unsigned grid = static_cast<unsigned>(blocks < cap ? blocks : cap);
  auto go = [&](auto kern) {
    kern<<<grid, 256, 0, stream>>>(p, static_cast<const Ts *>(ys), gate, pos,
                                   static_cast<const Tt *>(residual), static_cast<Tt *>(y));
  };
  const int n = p.K + p.has_shared;
  if (n <= 5)
    go(rows_unsort_kernel<Tt, Ts, E, 5>);
  else if (n <= 9)
    go(rows_unsort_kernel<Tt, Ts, E, 9>);
  else
    go(rows_unsort_kernel<Tt, Ts, E, 17>);
  return cudaGetLastError();
}

template <typename Tt, typename Ts, int E>
cudaError_t launch_grad_e(const RowsArgs &p, const void *dy, const void *ys, const float *gate,
                          const int32_t *pos, void *dys, float *dgate, int num_sms, cudaStream_t stream) {
  int wpt = 1;
  while (wpt < 8 && static_cast<int64_t>(p.T) * wpt < num_sms * 32) wpt *= 2;
  const unsigned grid = static_cast<unsigned>((p.T + 8 / wpt - 1) / (8 / wpt));
  auto go = [&](auto kern) {
    kern<<<grid, 256, 0, stream>>>(p, static_cast<const Tt *>(dy), static_cast<const Ts *>(ys), gate, pos,
                                   static_cast<Ts *>(dys), dgate, wpt);
  };
  if (p.K <= 4)
    go(rows_unsort_grad_kernel<Tt, Ts, E, 4>);
  else if (p.K <= 8)
    go(rows_unsort_grad_kernel<Tt, Ts, E, 8>);
  else
    go(rows_unsort_grad_kernel<Tt, Ts, E, 16>);
  return cudaGetLastError();
}

// f(Tt{}, Ts{}) for the two element types
template <typename F>
cudaError_t by_types(int tok, int slot, F f) {
  auto inner = [&](auto tt) {
    if (slot == MOE_DTYPE_BF16) return f(tt, Bf16{});
    if (slot == MOE_DTYPE_FP16) return f(tt, Fp16{});
    return f(tt, float{});
  };
  if (tok == MOE_DTYPE_BF16) return inner(Bf16{});
  if (tok == MOE_DTYPE_FP16) return inner(Fp16{});
  return inner(float{});
}

}  // namespace

cudaError_t launch_rows_sort(const RowsArgs &p, int elem, const void *x, const float *x_scale,
                             const int32_t *offsets, const int32_t *sorted, int32_t *pos, void *xs,
                             float *xs_scale, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(pos, 0xff, sizeof(int32_t) * static_cast<size_t>(p.P), stream);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (p.P + 255ll) / 256, cap = num_sms * 8ll;
  rows_invert_kernel<<<static_cast<unsigned>(blocks < cap ? blocks : cap), 256, 0, stream>>>(p, offsets,
                                                                                            sorted, pos);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t row = static_cast<int64_t>(p.H) * elem;
  auto fits = [&](int a) {
    return row % a == 0 && is_aligned(x, p.ld_token * elem, a) && is_aligned(xs, p.ld_slot * elem, a);
  };
  if (fits(16)) return launch_scatter<uint4>(p, pos, x, xs, x_scale, xs_scale, elem, num_sms, stream);
  if (fits(8)) return launch_scatter<uint2>(p, pos, x, xs, x_scale, xs_scale, elem, num_sms, stream);
  if (fits(4)) return launch_scatter<uint32_t>(p, pos, x, xs, x_scale, xs_scale, elem, num_sms, stream);
  if (fits(2)) return launch_scatter<uint16_t>(p, pos, x, xs, x_scale, xs_scale, elem, num_sms, stream);
  return launch_scatter<uint8_t>(p, pos, x, xs, x_scale, xs_scale, elem, num_sms, stream);
}

cudaError_t launch_rows_unsort(const RowsArgs &p, int dtype, int slot_dtype, const void *ys,
                               const float *gate, const int32_t *pos, const void *residual, void *y,
                               int num_sms, cudaStream_t stream) {
  return by_types(dtype, slot_dtype, [&](auto tt, auto ts) {
    using Tt = decltype(tt);
    using Ts = decltype(ts);
    const int64_t a = sizeof(Tt), b = sizeof(Ts);
    if (p.H % 8 == 0 && is_aligned(ys, p.ld_slot * b, 16) && is_aligned(residual, p.ld_residual * a, 16) &&
        is_aligned(y, p.ld_token * a, 16))
      return launch_unsort_e<Tt, Ts, 8>(p, ys, gate, pos, residual, y, num_sms, stream);
    return launch_unsort_e<Tt, Ts, 1>(p, ys, gate, pos, residual, y, num_sms, stream);
  });
}

cudaError_t launch_rows_unsort_grad(const RowsArgs &p, int dtype, int slot_dtype, const void *dy,
                                    const void *ys, const float *gate, const int32_t *pos, void *dys,
                                    float *dgate, int num_sms, cudaStream_t stream) {
  return by_types(dtype, slot_dtype, [&](auto tt, auto ts) {
    using Tt = decltype(tt);
    using Ts = decltype(ts);
    const int64_t a = sizeof(Tt), b = sizeof(Ts);
    if (p.H % 8 == 0 && is_aligned(dy, p.ld_token * a, 16) && is_aligned(ys, p.ld_slot * b, 16) &&
        is_aligned(dys, p.ld_dys * b, 16))
      return launch_grad_e<Tt, Ts, 8>(p, dy, ys, gate, pos, dys, dgate, num_sms, stream);
    return launch_grad_e<Tt, Ts, 1>(p, dy, ys, gate, pos, dys, dgate, num_sms, stream);
  });
}

}  // namespace srm
