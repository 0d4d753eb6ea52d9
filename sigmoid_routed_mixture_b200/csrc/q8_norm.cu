// q8_norm.cu -- rows to 8 bits with one scale per row, optionally after the
// residual's addition and the RMSNorm in the same pass:
//     x' = round(x + delta),  n = x' * gamma / sqrt(mean(x'^2) + eps),
//     scale = max |n| / 127,  q = rne(n / scale).
// Sums and statistics are fp32; x' is rounded to the stream's type because
// that is the value the stream stores, and the norm reads the stored value.
//
// One read of the row: a group of TPR threads holds a whole row in registers
// (U loads of E elements a thread) through its two reductions, the sum of
// squares and the maximum, so the bytes are the floor's.  Rows that do not fit
// (more than 1024 threads x U x E elements) are read three times.
#include "kernels.h"
#include "rowio.cuh"

namespace srm {

namespace {

// |v|'s bits: as an integer maximum they order like |v| and carry infinities
// and NaN (any pattern >= 0x7f800000) past every finite value.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Sum / maximum over a row's threads, the same value in each of them.  Fixed
// order: lanes by a shuffle tree, warps in turn.
template <int kWarps>
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (kWarps == 1) return v;
  const int n = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < n ? buf[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int kWarps>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *buf) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (kWarps == 1) return v;
  const int n = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < n ? buf[threadIdx.x & 31] : 0u);
}

// scale and the factor that takes n to q: q = rne((n * up) * r).  `up` keeps
// 127 / max finite for rows below 2^-100.  r = 0 for a zero row; a row with an
// infinity or NaN gets scale NaN and is written as zeros.
struct QScale {
  float scale, up, r;
  bool finite;
};
__device__ __forceinline__ QScale q_scale(uint32_t max_bits) {
  QScale s;
  s.finite = max_bits < 0x7f800000u;
  const float m = __uint_as_float(max_bits);
  s.scale = s.finite ? m / 127.f : __uint_as_float(0x7fc00000u);
  s.up = m < 0x1p-100f ? 0x1p100f : 1.f;
  s.r = m > 0.f ? 127.f / (m * s.up) : 0.f;
  return s;
}
__device__ __forceinline__ int q_of(float n, const QScale &s) {
  return s.finite ? max(-127, min(127, __float2int_rn((n * s.up) * s.r))) : 0;
}

template <int E>
__device__ __forceinline__ void store_q(int8_t *p, const float (&n)[E], const QScale &s) {
  if (E == 1) {
    *p = static_cast<int8_t>(q_of(n[0], s));
  } else {
    uint32_t w[(E + 3) / 4];
#pragma unroll
    for (int k = 0; k < E / 4; ++k)
      w[k] = (q_of(n[4 * k], s) & 0xff) | (q_of(n[4 * k + 1], s) & 0xff) << 8 |
             (q_of(n[4 * k + 2], s) & 0xff) << 16 | q_of(n[4 * k + 3], s) << 24;
    if (E == 8)
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[E / 4 - 1]);
    else
      *reinterpret_cast<uint32_t *>(p) = w[0];
  }
}

// Where a row goes: itself, or (packing the gate and up weights) row f of W1 /
// W3 to row (f / 16) * 32 + f % 16 (+ 16 for W3) of the interleaved matrix.
__device__ __forceinline__ int64_t dst_row(int64_t t, int unit_offset) {
  return unit_offset < 0 ? t : (t >> 4) * 32 + (t & 15) + unit_offset;
}

}  // namespace

// kWarps == 1: a warp per row (several rows a CTA); otherwise a CTA per row.
template <typename T, int E, int U, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 1024)
    q8_rows_kernel(const Q8RowArgs p) {
  __shared__ float sum_buf[2][32];
  __shared__ uint32_t max_buf[32];
  const int tid = kWarps == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int tpr = kWarps == 1 ? 32 : blockDim.x;
  const int64_t t = kWarps == 1 ? blockIdx.x * 4ll + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.T) return;  // whole warps (or CTAs) only
  const T *x = static_cast<const T *>(p.x) + t * p.ld_x;
  const T *delta = p.delta ? static_cast<const T *>(p.delta) + t * p.ld_delta : nullptr;
  const T *gamma = static_cast<const T *>(p.gamma);
  float v[U][E];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int i = (j * tpr + tid) * E;
#pragma unroll
    for (int k = 0; k < E; ++k) v[j][k] = 0.f;
    if (i < p.H) RowIo<T, E>::load(x + i, v[j]);
  }
  if (delta) {
    T *x_sum = p.x_sum ? static_cast<T *>(p.x_sum) + t * p.ld_sum : nullptr;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = (j * tpr + tid) * E;
      if (i < p.H) {
        float d[E];
        RowIo<T, E>::load(delta + i, d);
#pragma unroll
        for (int k = 0; k < E; ++k) v[j][k] = to_float(from_float<T>(v[j][k] + d[k]));
        if (x_sum) RowIo<T, E>::store(x_sum + i, v[j]);
      }
    }
  } else if (p.x_sum) {
    T *x_sum = static_cast<T *>(p.x_sum) + t * p.ld_sum;
#pragma unroll
    for (int j = 0; j < U; ++j)
      if ((j * tpr + tid) * E < p.H) RowIo<T, E>::store(x_sum + (j * tpr + tid) * E, v[j]);
  }
  if (gamma) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < E; ++k) ss = fmaf(v[j][k], v[j][k], ss);
    float ms = row_sum<kWarps>(ss, sum_buf[0]) / static_cast<float>(p.H) + p.eps;
    if (!(ms >= 0x1p-100f && ms <= 0x1p120f)) {
      // the squares left fp32's range (the same decision in the whole row):
      // once more with the row under a power of two
      const float f = ms < 0x1p-100f ? 0x1p96f : 0x1p-96f;
      ss = 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          v[j][k] *= f;
          ss = fmaf(v[j][k], v[j][k], ss);
        }
      ms = row_sum<kWarps>(ss, sum_buf[1]) / static_cast<float>(p.H) + (p.eps * f) * f;
    }
    const float inv = 1.0f / sqrtf(ms);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = (j * tpr + tid) * E;
      if (i < p.H) {
        float g[E];
        RowIo<T, E>::load(gamma + i, g);
#pragma unroll
        for (int k = 0; k < E; ++k) v[j][k] = v[j][k] * inv * g[k];
      }
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int k = 0; k < E; ++k)
      if ((j * tpr + tid) * E < p.H) m = max(m, abs_bits(v[j][k]));
  const QScale s = q_scale(row_max<kWarps>(m, max_buf));
  const int64_t to = dst_row(t, p.unit_offset);
  if (tid == 0) p.scale[to] = s.scale;
  int8_t *q = p.q + to * p.ld_q;
  T *y = p.y ? static_cast<T *>(p.y) + t * p.ld_y : nullptr;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int i = (j * tpr + tid) * E;
    if (i < p.H) {
      store_q<E>(q + i, v[j], s);
      if (y) RowIo<T, E>::store(y + i, v[j]);
    }
  }
}

// Rows too long for one CTA's registers: element loads, three passes over the
// row.  x_sum and y are written in the last pass only, each element by the
// thread that has just read it, so that they may be x or delta themselves.
template <typename T>
__global__ void __launch_bounds__(1024) q8_long_rows_kernel(const Q8RowArgs p) {
  __shared__ float sum_buf[2][32];
  __shared__ uint32_t max_buf[32];
  const int64_t t = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + t * p.ld_x;
  const T *delta = p.delta ? static_cast<const T *>(p.delta) + t * p.ld_delta : nullptr;
  const T *gamma = static_cast<const T *>(p.gamma);
  auto at = [&](int i) {
    const float v = to_float(x[i]);
    return delta ? to_float(from_float<T>(v + to_float(delta[i]))) : v;
  };
  float f = 1.f, inv = 1.f;
  if (gamma) {
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.H; i += blockDim.x) ss = fmaf(at(i), at(i), ss);
    float ms = row_sum<32>(ss, sum_buf[0]) / static_cast<float>(p.H) + p.eps;
    if (!(ms >= 0x1p-100f && ms <= 0x1p120f)) {
      f = ms < 0x1p-100f ? 0x1p96f : 0x1p-96f;
      ss = 0.f;
      for (int i = threadIdx.x; i < p.H; i += blockDim.x) ss = fmaf(at(i) * f, at(i) * f, ss);
      ms = row_sum<32>(ss, sum_buf[1]) / static_cast<float>(p.H) + (p.eps * f) * f;
    }
    inv = 1.0f / sqrtf(ms);
  }
  auto normed = [&](int i, float v) { return gamma ? v * f * inv * to_float(gamma[i]) : v; };
  uint32_t m = 0;
  for (int i = threadIdx.x; i < p.H; i += blockDim.x) m = max(m, abs_bits(normed(i, at(i))));
  const QScale s = q_scale(row_max<32>(m, max_buf));
  const int64_t to = dst_row(t, p.unit_offset);
  if (threadIdx.x == 0) p.scale[to] = s.scale;
  for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
    const float v = at(i), n = normed(i, v);
    if (p.x_sum) static_cast<T *>(p.x_sum)[t * p.ld_sum + i] = from_float<T>(v);
    if (p.y) static_cast<T *>(p.y)[t * p.ld_y + i] = from_float<T>(n);
    p.q[to * p.ld_q + i] = static_cast<int8_t>(q_of(n, s));
  }
}

// y = q * scale: E elements a thread, rows of ceil(H / E) threads.
template <typename T, int E>
__global__ void __launch_bounds__(256)
    q8_dequantize_kernel(const int8_t *q, const float *scale, T *y, int64_t T_, int H, int64_t ld_q,
                         int64_t ld_y) {
  const int per_row = (H + E - 1) / E;
  const int64_t total = T_ * per_row;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t t = i / per_row;
    const int c = static_cast<int>(i - t * per_row) * E;
    const float s = scale[t];
    float f[E];
    if (E == 1) {
      f[0] = q[t * ld_q + c] * s;
    } else {
      uint32_t w[(E + 3) / 4];
      if (E == 8) {
        const uint2 r = *reinterpret_cast<const uint2 *>(q + t * ld_q + c);
        w[0] = r.x;
        w[E / 4 - 1] = r.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t *>(q + t * ld_q + c);
      }
#pragma unroll
      for (int k = 0; k < E; ++k)
        f[k] = static_cast<float>(static_cast<int8_t>(w[k / 4] >> (8 * (k % 4)))) * s;
    }
    RowIo<T, E>::store(y + t * ld_y + c, f);
  }
}

namespace {

template <typename T, int E, int U>
cudaError_t launch_rows_u(const Q8RowArgs &p, cudaStream_t stream) {
  const int loads = (p.H + E - 1) / E;
  if (loads <= 32 * U) {
    q8_rows_kernel<T, E, U, 1><<<static_cast<unsigned>((p.T + 3) / 4), 128, 0, stream>>>(p);
  } else {
    const int threads = ((loads + U - 1) / U + 31) & ~31;
    q8_rows_kernel<T, E, U, 32><<<static_cast<unsigned>(p.T), threads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T, int E>
cudaError_t launch_rows_e(const Q8RowArgs &p, int num_sms, cudaStream_t stream) {
  const int loads = (p.H + E - 1) / E;
  if (loads <= 1024 && p.T <= 2 * num_sms) return launch_rows_u<T, E, 1>(p, stream);
  if (loads <= 4 * 1024) return launch_rows_u<T, E, 4>(p, stream);
  q8_long_rows_kernel<T><<<static_cast<unsigned>(p.T), 1024, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows_t(const Q8RowArgs &p, int num_sms, cudaStream_t stream) {
  constexpr int E = kVec<T>;
  auto vec = [&](const void *ptr, int64_t ld, int64_t size, int64_t bytes) {
    return !ptr || (reinterpret_cast<uintptr_t>(ptr) % bytes == 0 && (ld * size) % bytes == 0);
  };
  constexpr int64_t S = sizeof(T);
  if (p.H % E == 0 && vec(p.x, p.ld_x, S, 16) && vec(p.delta, p.ld_delta, S, 16) &&
      vec(p.gamma, 0, S, 16) && vec(p.x_sum, p.ld_sum, S, 16) && vec(p.y, p.ld_y, S, 16) &&
      vec(p.q, p.ld_q, 1, E))
    return launch_rows_e<T, E>(p, num_sms, stream);
  return launch_rows_e<T, 1>(p, num_sms, stream);
}

template <typename T>
cudaError_t launch_dequant_t(const int8_t *q, const float *scale, void *y, int64_t T_, int H,
                             int64_t ld_q, int64_t ld_y, int num_sms, cudaStream_t stream) {
  constexpr int E = kVec<T>;
  const bool vec = H % E == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0 && ld_y % E == 0 &&
                   reinterpret_cast<uintptr_t>(q) % E == 0 && ld_q % E == 0;
  const int64_t total = T_ * ((H + (vec ? E : 1) - 1) / (vec ? E : 1));
  const int64_t cap = num_sms * 16ll;
  const unsigned blocks = static_cast<unsigned>((total + 255) / 256 < cap ? (total + 255) / 256 : cap);
  if (vec)
    q8_dequantize_kernel<T, E><<<blocks, 256, 0, stream>>>(q, scale, static_cast<T *>(y), T_, H, ld_q, ld_y);
  else
    q8_dequantize_kernel<T, 1><<<blocks, 256, 0, stream>>>(q, scale, static_cast<T *>(y), T_, H, ld_q, ld_y);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q8_rows(int dtype, const Q8RowArgs &p, int num_sms, cudaStream_t stream) {
  if (dtype == MOE_DTYPE_BF16) return launch_rows_t<Bf16>(p, num_sms, stream);
  if (dtype == MOE_DTYPE_FP16) return launch_rows_t<Fp16>(p, num_sms, stream);
  return launch_rows_t<float>(p, num_sms, stream);
}

cudaError_t launch_q8_dequantize(int dtype, const int8_t *q, const float *scale, void *y, int64_t T, int H,
                                 int64_t ld_q, int64_t ld_y, int num_sms, cudaStream_t stream) {
  if (dtype == MOE_DTYPE_BF16)
    return launch_dequant_t<Bf16>(q, scale, y, T, H, ld_q, ld_y, num_sms, stream);
  if (dtype == MOE_DTYPE_FP16)
    return launch_dequant_t<Fp16>(q, scale, y, T, H, ld_q, ld_y, num_sms, stream);
  return launch_dequant_t<float>(q, scale, y, T, H, ld_q, ld_y, num_sms, stream);
}

}  // namespace srm
