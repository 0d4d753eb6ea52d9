// q8_norm.cu -- rows to 8 bits with one scale per row, optionally after the
// residual's addition and the RMSNorm in the same pass:
//     x' = round(x + delta),  n = x' * gamma / sqrt(mean(x'^2) + eps),
//     scale = max |n| / 127,  q = rne(n / scale).
// Sums and statistics are fp32; x' is rounded to the stream's type because
// that is the value the stream stores, and the norm reads the stored value.
//
// The root cancels in n / scale.  It is split into a power of two p and a
// factor r, 1 <= r < 2; u = x' p gamma is exact in fp32 for 16-bit types (8 + 8
// and 11 + 11 bits), n = u r, and q = rne(127 u / max |u|) is the definition's
// integer, ties included.  (From n rounded to fp32, one q in 10^5 went to the
// neighbour.)
//
// One read of the row: a group of TPR threads holds a whole row in registers
// (U loads of E elements a thread) through its two reductions, the sum of
// squares and the maximum, so the bytes are the floor's.  Rows that do not fit
// (more than 1024 threads x U x E elements) are read three times.
#include <type_traits>

#include "kernels.h"
#include "launch.cuh"
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

// 1 / sqrt(mean square + eps) of a row as p * r, p a power of two, 1 <= r < 2.
// sum(f): this thread's part of the sum of squares of the row times f.  `up`: 1,
// or the power of two that the row has to be multiplied by first (exactly: only
// rows below 2^-40 have one).
struct Root {
  float p, r, up;
};
template <int kWarps, typename Sum>
__device__ __forceinline__ Root inv_root(Sum sum, float H, float eps, float (*buf)[32]) {
  float f = 1.f;
  float ms = row_sum<kWarps>(sum(1.f), buf[0]) / H + eps;
  if (!(ms >= 0x1p-100f && ms <= 0x1p120f)) {
    // the squares left fp32's range (the same decision in the whole row): once
    // more with the row under a power of two
    f = ms < 0x1p-100f ? 0x1p96f : 0x1p-96f;
    ms = row_sum<kWarps>(sum(f), buf[1]) / H + (eps * f) * f;
  }
  const float inv = 1.0f / sqrtf(ms);
  Root o;
  // (0 gives p = 0, r = 1; an infinity or NaN keeps itself as p)
  o.p = inv <= 0x1p126f ? __uint_as_float(__float_as_uint(inv) & 0x7f800000u) : inv;
  o.r = __uint_as_float((__float_as_uint(inv) & 0x007fffffu) | 0x3f800000u);
  o.up = f > 1.f ? f : 1.f;
  if (f < 1.f) o.p *= f;
  return o;
}

// scale and the factor 127 / max that takes u to q, as the sum of two fp32
// numbers, for rows multiplied by `up`: 1, or the power of two that brings rows
// below 2^-100 or above 2^100 away from the ends of fp32's range.  max_bits: max
// |u|, n = u * r.  Both are 0 for a zero row; a row whose n holds an infinity or
// NaN gets scale NaN and zeros.
struct QFactor {
  float hi, lo, max;
};
struct QScale {
  float scale, up;
  QFactor r;
  bool finite;
};
__device__ __forceinline__ QScale q_scale(uint32_t max_bits, float r = 1.f) {
  QScale s;
  const float m = __uint_as_float(max_bits), n = m * r;
  s.finite = abs_bits(n) < 0x7f800000u;
  s.scale = s.finite ? n / 127.f : __uint_as_float(0x7fc00000u);
  s.up = m < 0x1p-100f ? 0x1p100f : m > 0x1p100f ? 0x1p-100f : 1.f;
  s.r = {0.f, 0.f, 0.f};
  if (s.finite && m > 0.f) {
    const float mu = m * s.up;
    s.r.max = mu;
    s.r.hi = 127.f / mu;
    s.r.lo = fmaf(-s.r.hi, mu, 127.f) * (s.r.hi * (1.f / 127.f));  // a few bits of it count
  }
  return s;
}

// q = rne(n * 127 / max) in the low byte: n * hi + (n * lo) is the quotient
// rounded once to fp32 (what is lost before is 2^-46 of it), and adding
// 1.5 * 2^23 rounds that to the nearest integer, ties to even, in two's
// complement; the quotient is at most 127, so nothing has to be clamped.  A
// quotient of exactly k + 1/2 comes out as that, and one that is not is at least
// 1 / (254 m) of itself away from it, where n is m < 2^a units of its last bit:
// for a <= 16 (bf16 products) more than half a unit of fp32's last place, so it
// does not.  (By hi alone one element in 70000 of fp16 rows went astray.)
__device__ __forceinline__ float quotient(float n, QFactor r) { return fmaf(n, r.hi, n * r.lo); }
__device__ __forceinline__ uint32_t q_bits(float n, QFactor r) {
  return __float_as_uint(quotient(n, r) + 12582912.f);
}
__device__ __forceinline__ void q_bits2(float n0, float n1, QFactor r, uint32_t &q0, uint32_t &q1) {
  asm("{\n\t.reg .b64 n, h, l, c;\n\t"
      "mov.b64 n, {%2, %3};\n\t"
      "mov.b64 h, {%4, %4};\n\t"
      "mov.b64 l, {%5, %5};\n\t"
      "mov.b64 c, {%6, %6};\n\t"
      "mul.rn.f32x2 l, n, l;\n\t"
      "fma.rn.f32x2 h, n, h, l;\n\t"
      "add.rn.f32x2 h, h, c;\n\t"
      "mov.b64 {%0, %1}, h;\n\t}"
      : "=r"(q0), "=r"(q1)
      : "f"(n0), "f"(n1), "f"(r.hi), "f"(r.lo), "f"(12582912.f));
}

__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// fp16 products have 22 bits: a quotient beside k + 1/2 may come out as k + 1/2,
// though never on its other side.  `most` collects the distance of the quotients
// from their integers, and if one is 1/2 the thread goes through its elements
// once more with settle() (one element in 400,000, ties included).
__device__ __forceinline__ void q_near2(float n0, float n1, QFactor r, uint32_t &q0, uint32_t &q1, float &most) {
  float d0, d1;
  asm("{\n\t.reg .b64 n, h, l, c, s;\n\t"
      "mov.b64 n, {%4, %5};\n\t"
      "mov.b64 h, {%6, %6};\n\t"
      "mov.b64 l, {%7, %7};\n\t"
      "mov.b64 c, {%8, %8};\n\t"
      "mul.rn.f32x2 l, n, l;\n\t"
      "fma.rn.f32x2 h, n, h, l;\n\t"
      "add.rn.f32x2 s, h, c;\n\t"
      "mov.b64 {%0, %1}, s;\n\t"
      "sub.rn.f32x2 s, s, c;\n\t"
      "sub.rn.f32x2 h, h, s;\n\t"
      "mov.b64 {%2, %3}, h;\n\t}"
      : "=r"(q0), "=r"(q1), "=f"(d0), "=f"(d1)
      : "f"(n0), "f"(n1), "f"(r.hi), "f"(r.lo), "f"(12582912.f));
  most = fmaxf(most, fmaxf(fabsf(d0), fabsf(d1)));
}
__device__ __forceinline__ uint32_t q_near(float n, QFactor r, float &d) {
  const float x = quotient(n, r), s = x + 12582912.f;
  d = x - (s - 12582912.f);
  return __float_as_uint(s);
}
// q of a quotient near c = k + 1/2: whether 254 |n| is more than, equal to (to
// even) or less than 2 c max.  Both products are exact as two fp32 numbers, and
// so is their difference, the leading parts being within a factor of two.
__device__ __forceinline__ uint32_t settle(float n, QFactor r, uint32_t q, float d) {
  const float c2 = fabsf(2.f * (__uint_as_float(q) - 12582912.f) + copysignf(1.f, d));
  const float a = __fmul_rn(254.f, fabsf(n)), b = __fmul_rn(c2, r.max);
  const float more = __fsub_rn(a, b) + (fmaf(254.f, fabsf(n), -a) - fmaf(c2, r.max, -b));
  int k = static_cast<int>(c2) >> 1;
  if (more > 0.f || (more == 0.f && (k & 1))) ++k;
  return static_cast<uint32_t>(n < 0.f ? -k : k);
}
// An element's q again, where it may have gone to the wrong side.
__device__ __forceinline__ void settle_q(int8_t *p, float n, QFactor r) {
  float d;
  const uint32_t q = q_near(n, r, d);
  if (fabsf(d) == 0.5f) *p = static_cast<int8_t>(settle(n, r, q, d));
}

// E consecutive q of a row that is finite (n multiplied by up).  kNear: with `most`.
template <int E, bool kNear>
__device__ __forceinline__ void store_q(int8_t *p, const float (&n)[E], QFactor r, float &most) {
  if constexpr (E == 1) {
    float d = 0.f;
    *p = static_cast<int8_t>(kNear ? q_near(n[0], r, d) : q_bits(n[0], r));
    most = fmaxf(most, fabsf(d));
  } else {
    uint32_t q[E], w[E / 4];
#pragma unroll
    for (int k = 0; k < E; k += 2) {
      if constexpr (kNear)
        q_near2(n[k], n[k + 1], r, q[k], q[k + 1], most);
      else
        q_bits2(n[k], n[k + 1], r, q[k], q[k + 1]);
    }
#pragma unroll
    for (int k = 0; k < E / 4; ++k) w[k] = low_bytes(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
    if constexpr (E == 8)
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t *>(p) = w[0];
  }
}

// E products, two in one operation
template <int E>
__device__ __forceinline__ void mul_by(float (&v)[E], float f) {
  if constexpr (E == 1) {
    v[0] *= f;
  } else {
#pragma unroll
    for (int k = 0; k < E; k += 2) mul2(v[k], v[k + 1], f, f);
  }
}
template <int E>
__device__ __forceinline__ void mul_by(float (&v)[E], const float (&f)[E]) {
  if constexpr (E == 1) {
    v[0] *= f[0];
  } else {
#pragma unroll
    for (int k = 0; k < E; k += 2) mul2(v[k], v[k + 1], f[k], f[k + 1]);
  }
}

// Elements [from, to) of the E at p: as one vector where that is all of them
// and p is aligned, else one by one (zeros for the others).
template <typename R, int E, typename S>
__device__ __forceinline__ R load_part(const S *p, int from, int to) {
  static_assert(sizeof(R) == E * sizeof(S), "a unit of E elements");
  R r;
  if (from <= 0 && to >= E && reinterpret_cast<uintptr_t>(p) % sizeof(R) == 0) {
    r = *reinterpret_cast<const R *>(p);
  } else {
    S e[E];
#pragma unroll
    for (int k = 0; k < E; ++k) e[k] = k >= from && k < to ? p[k] : S{};
    memcpy(&r, e, sizeof(R));
  }
  return r;
}
template <typename T, int E>
__device__ __forceinline__ void store_part(T *p, const float (&f)[E], int from, int to) {
  if (from <= 0 && to >= E) {
    RowIo<T, E>::store(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k >= from && k < to) p[k] = from_float<T>(f[k]);
  }
}

// Where a row goes: itself, or (packing the gate and up weights) row f of W1 /
// W3 to row (f / 16) * 32 + f % 16 (+ 16 for W3) of the interleaved matrix.
__device__ __forceinline__ int64_t dst_row(int64_t t, int unit_offset) {
  return unit_offset < 0 ? t : (t >> 4) * 32 + (t & 15) + unit_offset;
}

}  // namespace

// kWarps == 1: a warp per row (several rows a CTA); otherwise a CTA per row.
// All of a row's loads (x, delta, gamma) are in flight before the first use.
// Rows whose elements are moved singly (E = 1) take code without a test around
// every element: threads past the row's end take its last element once more,
// which only the sum of squares has to leave out; a barrier keeps them from
// reading it after its owner has stored over it (4096 x 1541 bf16, all elements
// singly: 40 us with the tests, 25 without when this was taken, 29 now).
template <typename T, int E, int U, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps)
    q8_rows_kernel(const Q8RowArgs p) {
  using Io = RowIo<T, E>;
  constexpr bool kNear = std::is_same<T, Fp16>::value;
  __shared__ float sum_buf[2][32];
  __shared__ uint32_t max_buf[32];
  const int tid = kWarps == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int tpr = kWarps == 1 ? 32 : blockDim.x;
  const int64_t t = kWarps == 1 ? blockIdx.x * 4ll + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.T) return;  // whole warps (or CTAs) only
  previous_done();
  const T *x = static_cast<const T *>(p.x) + t * p.ld_x;
  const T *delta = p.delta ? static_cast<const T *>(p.delta) + t * p.ld_delta : nullptr;
  const T *gamma = static_cast<const T *>(p.gamma);
  constexpr bool kAgain = E == 1;
  // element j of this thread, and whether it is its own
  auto at = [&](int j) {
    const int i = (j * tpr + tid) * E;
    return kAgain ? min(i, p.H - 1) : i;
  };
  auto own = [&](int j) { return (j * tpr + tid) * E < p.H; };
  auto there = [&](int j) { return kAgain || own(j); };
  typename Io::Raw rx[U], rd[U], rg[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (there(j)) rx[j] = *reinterpret_cast<const typename Io::Raw *>(x + at(j));
  }
  if (delta) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (there(j)) rd[j] = *reinterpret_cast<const typename Io::Raw *>(delta + at(j));
    }
  }
  if (gamma) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (there(j)) rg[j] = *reinterpret_cast<const typename Io::Raw *>(gamma + at(j));
    }
  }
  if (kAgain) {
    if (kWarps == 1)
      __syncwarp();
    else
      __syncthreads();
  }
  float v[U][E];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (there(j)) {
      Io::unpack(rx[j], v[j]);
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) v[j][k] = 0.f;
    }
  }
  if (delta) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (there(j)) {
        float d[E];
        Io::unpack(rd[j], d);
#pragma unroll
        for (int k = 0; k < E; ++k) v[j][k] = to_float(from_float<T>(v[j][k] + d[k]));
      }
    }
  }
  if (p.x_sum) {
    T *x_sum = static_cast<T *>(p.x_sum) + t * p.ld_sum;
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (there(j)) Io::store(x_sum + at(j), v[j]);
  }
  float r = 1.f;  // n = v * r
  if (gamma) {
    auto sum = [&](float f) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < E; ++k) ss = fmaf(v[j][k] * f, kAgain && !own(j) ? 0.f : v[j][k] * f, ss);
      return ss;
    };
    const Root root = inv_root<kWarps>(sum, static_cast<float>(p.H), p.eps, sum_buf);
    r = root.r;
    if (root.up != 1.f) {
#pragma unroll
      for (int j = 0; j < U; ++j) mul_by(v[j], root.up);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (there(j)) {
        float g[E];
        Io::unpack(rg[j], g);
        mul_by(v[j], root.p);
        mul_by(v[j], g);
      }
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (there(j)) m = max(m, abs_bits(v[j][k]));
  if (p.y) {
    T *y = static_cast<T *>(p.y) + t * p.ld_y;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (there(j)) {
        float n[E];
#pragma unroll
        for (int k = 0; k < E; ++k) n[k] = v[j][k];
        mul_by(n, r);
        Io::store(y + at(j), n);
      }
    }
  }
  const QScale s = q_scale(row_max<kWarps>(m, max_buf), r);
  const int64_t to = dst_row(t, p.unit_offset);
  if (tid == 0) p.scale[to] = s.scale;
  int8_t *q = p.q + to * p.ld_q;
  if (!s.finite || s.up != 1.f) {  // rare, and the same in the whole row
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < E; ++k) v[j][k] = s.finite ? v[j][k] * s.up : 0.f;
  }
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (there(j)) store_q<E, kNear>(q + at(j), v[j], s.r, most);
  if (kNear && most == 0.5f) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < E; ++k)
        if (there(j)) settle_q(q + at(j) + k, v[j][k], s.r);
  }
}

// Quantisation alone.  Threads past the row's end take its last E elements once
// more (the same maximum, the same bytes stored), which spares a test around
// every step: 5003 x 1541 fp16, singly, 16 us with the tests (36 instructions an
// element), 10 without (1 of them the exact ties).
template <typename T, int E, int U, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps)
    q8_quantize_kernel(const Q8RowArgs p) {
  using Io = RowIo<T, E>;
  __shared__ uint32_t max_buf[32];
  const int tid = kWarps == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int tpr = kWarps == 1 ? 32 : blockDim.x;
  const int64_t t = kWarps == 1 ? blockIdx.x * 4ll + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.T) return;  // whole warps (or CTAs) only
  previous_done();
  const T *x = static_cast<const T *>(p.x) + t * p.ld_x;
  typename Io::Raw rx[U];
  const int last = p.H - E;
#pragma unroll
  for (int j = 0; j < U; ++j) rx[j] = *reinterpret_cast<const typename Io::Raw *>(x + min((j * tpr + tid) * E, last));
  float v[U][E];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    Io::unpack(rx[j], v[j]);
#pragma unroll
    for (int k = 0; k < E; ++k) m = max(m, abs_bits(v[j][k]));
  }
  const QScale s = q_scale(row_max<kWarps>(m, max_buf));
  const int64_t to = dst_row(t, p.unit_offset);
  if (tid == 0) p.scale[to] = s.scale;
  if (!s.finite || s.up != 1.f) {  // rare, and the same in the whole row
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < E; ++k) v[j][k] = s.finite ? v[j][k] * s.up : 0.f;
  }
  int8_t *q = p.q + to * p.ld_q;
  float most = 0.f;  // (not used)
  if constexpr (E == 1 && U % 2 == 0) {  // single elements: two of the row's at once
#pragma unroll
    for (int j = 0; j < U; j += 2) {
      uint32_t q0, q1;
      q_bits2(v[j][0], v[j + 1][0], s.r, q0, q1);
      q[min(j * tpr + tid, last)] = static_cast<int8_t>(q0);
      q[min((j + 1) * tpr + tid, last)] = static_cast<int8_t>(q1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) store_q<E, false>(q + min((j * tpr + tid) * E, last), v[j], s.r, most);
  }
}

// Rows that start at any element, in matrices that are aligned as a whole and
// whose row strides leave the same remainder of E: the units are those of the
// matrices, so a row's first and last one may be shared with its neighbours
// (each row's thread moves its own elements of them singly) and all others are
// whole vectors.  gamma, which starts anew in each row, is read singly except
// where it happens to be aligned.  (4096 x 1541 bf16 with sum, norm and 8 bits:
// 18.6 us, all elements singly 29; quantised alone 5003 x 1541 fp16 7.3 against
// 9.5.)
template <typename T, int U, int kWarps, bool kPlain>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps)
    q8_offset_rows_kernel(const Q8RowArgs p) {
  constexpr int E = kVec<T>;
  constexpr bool kNear = !kPlain && std::is_same<T, Fp16>::value;
  using Io = RowIo<T, E>;
  using Raw = typename Io::Raw;
  __shared__ float sum_buf[2][32];
  __shared__ uint32_t max_buf[32];
  const int tid = kWarps == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int tpr = kWarps == 1 ? 32 : blockDim.x;
  const int64_t t = kWarps == 1 ? blockIdx.x * 4ll + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= p.T) return;  // whole warps (or CTAs) only
  previous_done();
  // the row is elements lo .. hi - 1 from the unit that holds its first one
  const int lo = static_cast<int>(t * p.ld_x % E), hi = lo + p.H;
  auto at = [&](int j) { return (j * tpr + tid) * E; };
  const T *x = static_cast<const T *>(p.x) + (t * p.ld_x - lo);
  Raw rx[U], rd[kPlain ? 1 : U], rg[kPlain ? 1 : U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    rx[j] = Raw{};
    if (at(j) < hi) rx[j] = load_part<Raw, E>(x + at(j), lo - at(j), hi - at(j));
  }
  if (!kPlain && p.delta) {
    const T *delta = static_cast<const T *>(p.delta) + (t * p.ld_delta - lo);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      rd[kPlain ? 0 : j] = Raw{};
      if (at(j) < hi) rd[kPlain ? 0 : j] = load_part<Raw, E>(delta + at(j), lo - at(j), hi - at(j));
    }
  }
  if (!kPlain && p.gamma) {
    const T *gamma = static_cast<const T *>(p.gamma) - lo;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      rg[kPlain ? 0 : j] = Raw{};
      if (at(j) < hi) rg[kPlain ? 0 : j] = load_part<Raw, E>(gamma + at(j), lo - at(j), hi - at(j));
    }
  }
  float v[U][E];
#pragma unroll
  for (int j = 0; j < U; ++j) Io::unpack(rx[j], v[j]);
  if (!kPlain && p.delta) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float d[E];
      Io::unpack(rd[kPlain ? 0 : j], d);
#pragma unroll
      for (int k = 0; k < E; ++k) v[j][k] = to_float(from_float<T>(v[j][k] + d[k]));
    }
  }
  if (!kPlain && p.x_sum) {
    T *x_sum = static_cast<T *>(p.x_sum) + (t * p.ld_sum - lo);
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (at(j) < hi) store_part<T, E>(x_sum + at(j), v[j], lo - at(j), hi - at(j));
  }
  float r = 1.f;  // n = v * r
  if (!kPlain && p.gamma) {
    auto sum = [&](float f) {
      float ss = 0.f;  // the elements outside the row are zeros
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < E; ++k) ss = fmaf(v[j][k] * f, v[j][k] * f, ss);
      return ss;
    };
    const Root root = inv_root<kWarps>(sum, static_cast<float>(p.H), p.eps, sum_buf);
    r = root.r;
    if (root.up != 1.f) {
#pragma unroll
      for (int j = 0; j < U; ++j) mul_by(v[j], root.up);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float g[E];
      Io::unpack(rg[kPlain ? 0 : j], g);
      mul_by(v[j], root.p);
      mul_by(v[j], g);
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int k = 0; k < E; ++k) m = max(m, abs_bits(v[j][k]));
  if (!kPlain && p.y) {
    T *y = static_cast<T *>(p.y) + (t * p.ld_y - lo);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (at(j) < hi) {
        float n[E];
#pragma unroll
        for (int k = 0; k < E; ++k) n[k] = v[j][k];
        mul_by(n, r);
        store_part<T, E>(y + at(j), n, lo - at(j), hi - at(j));
      }
    }
  }
  const QScale s = q_scale(row_max<kWarps>(m, max_buf), r);
  if (tid == 0) p.scale[t] = s.scale;
  if (!s.finite || s.up != 1.f) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < E; ++k) v[j][k] = s.finite ? v[j][k] * s.up : 0.f;
  }
  int8_t *q = p.q + (t * p.ld_q - lo);
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int from = lo - at(j), to = hi - at(j);
    if (from <= 0 && to >= E) {
      store_q<E, kNear>(q + at(j), v[j], s.r, most);
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k)
        if (k >= from && k < to) store_q<1, kNear>(q + at(j) + k, {v[j][k]}, s.r, most);
    }
  }
  if (kNear && most == 0.5f) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int k = 0; k < E; ++k)
        if (k >= lo - at(j) && k < hi - at(j)) settle_q(q + at(j) + k, v[j][k], s.r);
  }
}

// Rows too long for one CTA's registers: element loads, three passes over the
// row.  x_sum and y are written in the last pass only, each element by the
// thread that has just read it, so that they may be x or delta themselves.
template <typename T>
__global__ void __launch_bounds__(1024) q8_long_rows_kernel(const Q8RowArgs p) {
  constexpr bool kNear = std::is_same<T, Fp16>::value;
  __shared__ float sum_buf[2][32];
  __shared__ uint32_t max_buf[32];
  previous_done();
  const int64_t t = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + t * p.ld_x;
  const T *delta = p.delta ? static_cast<const T *>(p.delta) + t * p.ld_delta : nullptr;
  const T *gamma = static_cast<const T *>(p.gamma);
  auto at = [&](int i) {
    const float v = to_float(x[i]);
    return delta ? to_float(from_float<T>(v + to_float(delta[i]))) : v;
  };
  Root root = {1.f, 1.f, 1.f};
  if (gamma) {
    auto sum = [&](float f) {
      float ss = 0.f;
      for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
        const float v = at(i) * f;
        ss = fmaf(v, v, ss);
      }
      return ss;
    };
    root = inv_root<32>(sum, static_cast<float>(p.H), p.eps, sum_buf);
  }
  auto before_r = [&](int i, float v) { return gamma ? v * root.up * root.p * to_float(gamma[i]) : v; };  // u = n / r
  uint32_t m = 0;
  for (int i = threadIdx.x; i < p.H; i += blockDim.x) m = max(m, abs_bits(before_r(i, at(i))));
  const QScale s = q_scale(row_max<32>(m, max_buf), root.r);
  const int64_t to = dst_row(t, p.unit_offset);
  if (threadIdx.x == 0) p.scale[to] = s.scale;
  for (int i = threadIdx.x; i < p.H; i += blockDim.x) {
    const float v = at(i), u = before_r(i, v);
    if (p.x_sum) static_cast<T *>(p.x_sum)[t * p.ld_sum + i] = from_float<T>(v);
    if (p.y) static_cast<T *>(p.y)[t * p.ld_y + i] = from_float<T>(u * root.r);
    const float n[1] = {s.finite ? u * s.up : 0.f};
    float most = 0.f;
    int8_t *q = p.q + to * p.ld_q + i;
    store_q<1, kNear>(q, n, s.r, most);
    if (kNear && most == 0.5f) settle_q(q, n[0], s.r);
  }
}

// y = q * scale.  tpr threads (a power of two) share a row, each with kBatch
// loads of E elements in flight; 256 / tpr rows a CTA.  kOffset: rows that
// start at any element, as in q8_offset_rows_kernel (5003 x 1541 to fp16: 4.8 us,
// all elements singly 8.5).
template <typename T, int E, bool kOffset>
__global__ void __launch_bounds__(256)
    q8_dequantize_kernel(const int8_t *q, const float *scale, T *y, int64_t T_, int H, int64_t ld_q,
                         int64_t ld_y, int tpr_log2) {
  constexpr int kBatch = 4;
  using Word = typename std::conditional<E == 8, uint2, typename std::conditional<E == 4, uint32_t, int8_t>::type>::type;
  const int tpr = 1 << tpr_log2;
  const int tid = threadIdx.x & (tpr - 1);
  const int64_t t = (static_cast<int64_t>(blockIdx.x) << (8 - tpr_log2)) + (threadIdx.x >> tpr_log2);
  if (t >= T_) return;
  previous_done();
  const int lo = kOffset ? static_cast<int>(t * ld_q % E) : 0;
  const int hi = kOffset ? lo + H : H;
  const int8_t *src = q + t * ld_q - lo;
  T *dst = y + t * ld_y - lo;
  const float s = scale[t];
  for (int i0 = tid * E; i0 < hi; i0 += kBatch * tpr * E) {
    Word w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if constexpr (kOffset) {
        const int c = i0 + j * tpr * E;
        if (c < hi) w[j] = load_part<Word, E>(src + c, lo - c, hi - c);
      } else {
        if (i0 + j * tpr * E < H) w[j] = *reinterpret_cast<const Word *>(src + i0 + j * tpr * E);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + j * tpr * E >= hi) break;
      float f[E];
      if constexpr (E == 1) {
        f[0] = w[j] * s;
      } else {
        uint32_t u[E / 4];
        if constexpr (E == 8) {
          u[0] = w[j].x;
          u[1] = w[j].y;
        } else {
          u[0] = w[j];
        }
#pragma unroll
        for (int k = 0; k < E; ++k)
          f[k] = static_cast<float>(static_cast<int8_t>(u[k / 4] >> (8 * (k % 4)))) * s;
      }
      if constexpr (kOffset) {
        const int c = i0 + j * tpr * E;
        store_part<T, E>(dst + c, f, lo - c, hi - c);
      } else {
        RowIo<T, E>::store(dst + i0 + j * tpr * E, f);
      }
    }
  }
}

namespace {

bool is_plain(const Q8RowArgs &p) { return !p.delta && !p.gamma && !p.x_sum && !p.y; }

// the fewer threads, the more registers each may have
template <typename T, int E, int U>
cudaError_t launch_rows_u(const Q8RowArgs &p, cudaStream_t stream) {
  const int loads = (p.H + E - 1) / E;
  const int threads = ((loads + U - 1) / U + 31) & ~31;
  const unsigned rows = static_cast<unsigned>(p.T);
  const bool plain = is_plain(p);
  auto go = [&](auto full, auto quantize) {
    auto kern = plain ? quantize : full;
    return threads <= 32 ? launch_overlapped(kern, (rows + 3) / 4, 128, 0, stream, p)
                         : launch_overlapped(kern, rows, threads, 0, stream, p);
  };
  if (threads <= 32) return go(q8_rows_kernel<T, E, U, 1>, q8_quantize_kernel<T, E, U, 1>);
  if (threads <= 256) return go(q8_rows_kernel<T, E, U, 8>, q8_quantize_kernel<T, E, U, 8>);
  if (threads <= 512) return go(q8_rows_kernel<T, E, U, 16>, q8_quantize_kernel<T, E, U, 16>);
  // (launch_rows_e gives the norm of single elements no more than 512 threads of U)
  return go(q8_rows_kernel<T, E, E == 1 ? 1 : U, 32>, q8_quantize_kernel<T, E, U, 32>);
}

template <typename T, int E>
cudaError_t launch_rows_e(const Q8RowArgs &p, int num_sms, cudaStream_t stream) {
  constexpr int U = E == 1 ? 16 : 4;  // loads a thread: 16 elements at least
  const int loads = (p.H + E - 1) / E;
  if (loads <= 1024 && p.T <= 2 * num_sms) return launch_rows_u<T, E, 1>(p, stream);
  // (with 1024 threads of 16 single elements the norm keeps much of its row in
  // local memory: 4096 x 9311 bf16 255 us against 222 in three passes.  With 1024
  // threads of 4 vectors it keeps 32 to 40 bytes a thread there, in fp32 8, and
  // 1024 x 24576 bf16 takes 52 us, where three passes over 20001 take 114.)
  if (loads <= U * (E == 1 && !is_plain(p) ? 512 : 1024)) return launch_rows_u<T, E, U>(p, stream);
  return launch_overlapped(q8_long_rows_kernel<T>, static_cast<unsigned>(p.T), 1024, 0, stream, p);
}

// (512 threads at most, 16384 elements of 16 bits or 8192 of 32; longer rows are
// moved singly.  1024 threads of 4 units would keep up to 100 bytes a thread in
// local memory and still be faster: 1024 x 20001 bf16 51 us against 114, 1024 x
// 9311 fp32 33 against 60.)
template <typename T, int U>
cudaError_t launch_rows_offset(const Q8RowArgs &p, int units, cudaStream_t stream) {
  const int threads = ((units + U - 1) / U + 31) & ~31;
  const unsigned rows = static_cast<unsigned>(p.T);
  const bool plain = is_plain(p);
  auto go = [&](auto full, auto quantize) {
    auto kern = plain ? quantize : full;
    return threads <= 32 ? launch_overlapped(kern, (rows + 3) / 4, 128, 0, stream, p)
                         : launch_overlapped(kern, rows, threads, 0, stream, p);
  };
  if (threads <= 32) return go(q8_offset_rows_kernel<T, U, 1, false>, q8_offset_rows_kernel<T, U, 1, true>);
  if (threads <= 256) return go(q8_offset_rows_kernel<T, U, 8, false>, q8_offset_rows_kernel<T, U, 8, true>);
  return go(q8_offset_rows_kernel<T, U, 16, false>, q8_offset_rows_kernel<T, U, 16, true>);
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
  auto whole = [&](const void *ptr, int64_t ld, int64_t bytes) {
    return !ptr || (reinterpret_cast<uintptr_t>(ptr) % bytes == 0 && (p.T == 1 || ld % E == p.ld_x % E));
  };
  // Short rows, and middling ones that are few, are faster singly: their first
  // and last units take two steps.  One rule for all types and both forms, us by
  // units / singly (bf16, fp16, fp32):
  //   norm      16384 x 385    26.3 / 24.7   30.5 / 23.8   19.3 / 23.8
  //             16384 x 513    27.9 / 52.1   31.9 / 48.5   29.7 / 44.2
  //             1024 x 1001    5.0 / 4.4     5.9 / 4.6     4.0 / 4.1
  //             1024 x 1281    5.3 / 6.6     5.4 / 6.4     4.6 / 5.7
  //   quantise  16384 x 385    11.0 / 7.7    10.6 / 7.5    6.4 / 7.6
  //             16384 x 513    10.4 / 15.0   9.9 / 14.6    12.0 / 15.4
  //             1024 x 1001    2.3 / 2.1     2.3 / 2.1     2.1 / 2.2
  //             16384 x 2047   30.5 / 30.5   30.9 / 31.6   30.4 / 35.9
  // (fp32 rows would gain from 385 on, 4096 x 9311 bf16 gains most: 90 / 220.)
  const bool gains = p.H > 1024 || (p.H > 512 && p.T > 8 * num_sms);
  const int units = (p.H + 2 * (E - 1)) / E;  // at most, wherever a row starts
  if (gains && p.unit_offset < 0 && whole(p.x, p.ld_x, 16) && whole(p.delta, p.ld_delta, 16) && whole(p.x_sum, p.ld_sum, 16) &&
      whole(p.y, p.ld_y, 16) && whole(p.q, p.ld_q, E)) {
    if (units <= 512 && p.T <= 2 * num_sms) return launch_rows_offset<T, 1>(p, units, stream);
    if (units <= 512 * 4) return launch_rows_offset<T, 4>(p, units, stream);
  }
  return launch_rows_e<T, 1>(p, num_sms, stream);
}

template <typename T>
cudaError_t launch_dequant_t(const int8_t *q, const float *scale, void *y, int64_t T_, int H,
                             int64_t ld_q, int64_t ld_y, cudaStream_t stream) {
  constexpr int E = kVec<T>;
  const bool whole = reinterpret_cast<uintptr_t>(y) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % E == 0;
  const bool vec = whole && H % E == 0 && ld_y % E == 0 && ld_q % E == 0;
  // (as for the rows to 8 bits, us by units / singly, bf16 and fp32: 1024 x 1001
  // 2.2 / 1.9 and 1.95 / 1.74, 1024 x 1281 2.0 / 2.5 and 2.1 / 2.3, 16384 x 129 3.4 /
  // 4.4 and 3.3 / 4.2, 1 x 6145 1.7 / 2.8 and 2.1 / 2.8)
  const bool gains = H > 2048 || T_ * H > 5 << 18;
  const bool offset = gains && whole && !vec && (T_ == 1 || ld_y % E == ld_q % E);
  const int loads = vec ? H / E : offset ? (H + 2 * (E - 1)) / E : H;
  int log2 = 0;  // threads per row: four loads each
  while (log2 < 8 && (4 << log2) < loads) ++log2;
  const unsigned blocks = static_cast<unsigned>((T_ + (256 >> log2) - 1) >> (8 - log2));
  auto kern = vec      ? q8_dequantize_kernel<T, E, false>
              : offset ? q8_dequantize_kernel<T, E, true>
                       : q8_dequantize_kernel<T, 1, false>;
  return launch_overlapped(kern, blocks, 256, 0, stream, q, scale, static_cast<T *>(y), T_, H, ld_q, ld_y, log2);
}

}  // namespace

cudaError_t launch_q8_rows(int dtype, const Q8RowArgs &p, int num_sms, cudaStream_t stream) {
  if (dtype == MOE_DTYPE_BF16) return launch_rows_t<Bf16>(p, num_sms, stream);
  if (dtype == MOE_DTYPE_FP16) return launch_rows_t<Fp16>(p, num_sms, stream);
  return launch_rows_t<float>(p, num_sms, stream);
}

cudaError_t launch_q8_dequantize(int dtype, const int8_t *q, const float *scale, void *y, int64_t T, int H,
                                 int64_t ld_q, int64_t ld_y, cudaStream_t stream) {
  if (dtype == MOE_DTYPE_BF16)
    return launch_dequant_t<Bf16>(q, scale, y, T, H, ld_q, ld_y, stream);
  if (dtype == MOE_DTYPE_FP16)
    return launch_dequant_t<Fp16>(q, scale, y, T, H, ld_q, ld_y, stream);
  return launch_dequant_t<float>(q, scale, y, T, H, ld_q, ld_y, stream);
}

}  // namespace srm
