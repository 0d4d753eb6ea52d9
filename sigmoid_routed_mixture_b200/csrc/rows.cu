// rows.cu -- token rows to the experts' order and back with the routing
// weights applied, and the gradients of both (formulas: include/srm_rows.h).
//
// All of it is bound by memory: each token row is read once and each sorted
// row written once, or the reverse; the gradient of the way back reads dy once
// for all of a token's slots.  No atomics on values: every output element is
// the work of one thread, and a sum over slots or over a row runs in a fixed
// order.  (The inverse is a maximum of positions, whose order does not matter.)
#include <type_traits>

#include "grid_walk.h"
#include "kernels.h"
#include "launch.cuh"
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

// p as a position in [0, P), or -1.
__device__ __forceinline__ int row_pos(int p, int P, int *err) {
  if (p >= -1 && p < P) return p;
  record_error(err, MOE_ERR_BAD_INDEX);
  return -1;
}

// pos[a] = p for the row id a that position p holds.  An id in two positions
// (of a list that is no permutation) goes to the later one, whatever the order
// of the threads, and is flagged.
__device__ __forceinline__ void invert(int32_t *pos, int a, int p, int P, int *err) {
  if (a < 0 || a >= P || atomicMax(&pos[a], p) >= 0) record_error(err, MOE_ERR_BAD_INDEX);
}

constexpr int kBatch = 8;              // vectors a lane has in flight
constexpr int kSmallPositions = 4096;  // the inverse in every CTA's shared memory: 16 KB

}  // namespace

// pos[sorted[p]] = p over the positions that hold a row (pos is -1 before).
__global__ void __launch_bounds__(256)
    rows_invert_kernel(const RowsArgs p, const int32_t *offsets,
                       const int32_t *sorted, int32_t *pos) {
  previous_done();
  const int n = row_total(offsets, p.E + 1, p.P, p.err);
  grid_walk(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, n, [&](int i) { invert(pos, sorted[i], i, p.P, p.err); });
}

// The rows by token: each token row is read once and written to its positions
// (pos: global or shared memory).  W: the widest vector all rows are aligned
// to; a warp moves a part of a row.
template <typename W>
__device__ __forceinline__ void scatter_tokens(const RowsArgs &p, const int32_t *pos, const uint8_t *x,
                                               uint8_t *xs, const float *x_scale, float *xs_scale,
                                               int64_t row_bytes, int64_t x_pitch, int64_t xs_pitch, int wpt) {
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
      mine = row_pos(pos[t * p.K + lane], p.P, p.err);
    else if (lane == p.K && p.has_shared)
      mine = row_pos(pos[p.T * p.K + t], p.P, p.err);
    if (xs_scale && begin == 0 && mine >= 0) xs_scale[mine] = x_scale[t];
    const int n_dst = p.K + p.has_shared;
    const W *src = reinterpret_cast<const W *>(x + t * x_pitch);
    for (int v0 = begin; v0 < end; v0 += 32 * kBatch) {
      const int at = v0 + lane;
      const bool full = v0 + 32 * kBatch <= end;  // no tests inside
      W buf[kBatch];
      if (full) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) buf[j] = src[at + j * 32];
      } else {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (at + j * 32 < end) buf[j] = src[at + j * 32];
      }
      for (int k = 0; k < n_dst; ++k) {
        const int d = __shfl_sync(0xffffffffu, mine, k);
        if (d < 0) continue;
        W *out = reinterpret_cast<W *>(xs + d * xs_pitch) + at;
        if (full) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) out[j * 32] = buf[j];
        } else {
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (at + j * 32 < end) out[j * 32] = buf[j];
        }
      }
    }
  }
}

template <typename W>
__global__ void __launch_bounds__(256)
    rows_scatter_kernel(const RowsArgs p, const int32_t *pos, const uint8_t *x,
                        uint8_t *xs, const float *x_scale,
                        float *xs_scale, int64_t row_bytes, int64_t x_pitch, int64_t xs_pitch,
                        int wpt) {
  previous_done();
  scatter_tokens<W>(p, pos, x, xs, x_scale, xs_scale, row_bytes, x_pitch, xs_pitch, wpt);
}

// The same in one launch for few positions: every CTA builds the whole inverse
// in its shared memory, CTA 0 writes it out, and each CTA moves its tokens.
// (64 tokens x 9 rows of 12 KB: 8.4 us as clear, invert and scatter.)
template <typename W>
__global__ void __launch_bounds__(256)
    rows_sort_small_kernel(const RowsArgs p, const int32_t *offsets,
                           const int32_t *sorted, int32_t *pos,
                           const uint8_t *x, uint8_t *xs,
                           const float *x_scale, float *xs_scale, int64_t row_bytes,
                           int64_t x_pitch, int64_t xs_pitch, int wpt) {
  __shared__ int32_t inverse[kSmallPositions];
  for (int i = threadIdx.x; i < p.P; i += 256) inverse[i] = -1;
  __syncthreads();
  previous_done();
  const int n = row_total(offsets, p.E + 1, p.P, p.err);
  // four ids on their way at a time (64 tokens x 9 rows of 12 KB, 400 of 4 KB: 4.0
  // and 6.6 us, with one 4.5 and 8.1, with eight 4.1 and 6.3)
  for (int i = threadIdx.x; i < n; i += 1024) {
    int a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + 256 * j < n) a[j] = sorted[i + 256 * j];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + 256 * j < n) invert(inverse, a[j], i + 256 * j, p.P, p.err);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.P; i += 256) pos[i] = inverse[i];
  scatter_tokens<W>(p, inverse, x, xs, x_scale, xs_scale, row_bytes, x_pitch, xs_pitch, wpt);
}

// The way back: y[t] = (residual[t] +) the weighted sum of the token's rows.
// 2^tpr_log2 threads share a token's row (256 >> tpr_log2 tokens a CTA); a
// thread issues the loads of all of the token's rows before the sums.  NB:
// slots and the shared row, at most or (kExact) exactly.  With kExact a token
// that has all its rows takes straight-line code.
template <typename Tt, typename Ts, int E, int NB, bool kExact>
__global__ void __launch_bounds__(256)
    rows_unsort_kernel(const RowsArgs p, const Ts *ys, const float *gate,
                       const int32_t *pos, const Tt *residual, Tt *y, int tpr_log2) {
  const int tpr = 1 << tpr_log2;
  const int64_t t64 = (static_cast<int64_t>(blockIdx.x) << (8 - tpr_log2)) + (threadIdx.x >> tpr_log2);
  if (t64 >= p.T) return;
  previous_done();
  const int t = static_cast<int>(t64);
  const int n = kExact ? NB : p.K + p.has_shared;
  // all on their way before the first check
  int at[NB];
  float g[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    at[k] = -1;
    g[k] = 1.f;
    if (k < n) {
      at[k] = pos[k < p.K ? t * p.K + k : p.T * p.K + t];
      if (gate && k < p.K) g[k] = gate[static_cast<int64_t>(t) * p.K + k];
    }
  }
  bool all = true;
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    if (k < n) {
      at[k] = row_pos(at[k], p.P, p.err);
      all = all && at[k] >= 0;
    }
  }
  for (int c = (threadIdx.x & (tpr - 1)) * E; c < p.H; c += tpr * E) {
    Unit<Ts, E> v[NB];
    Unit<Tt, E> r;
    if (residual) r.load(residual + t * p.ld_residual + c);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (kExact && all) {
#pragma unroll
      for (int k = 0; k < NB; ++k) v[k].load(ys + at[k] * p.ld_slot + c);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        float f[E];
        v[k].get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(g[k], f[e], acc[e]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (at[k] >= 0) v[k].load(ys + at[k] * p.ld_slot + c);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (at[k] < 0) continue;
        float f[E];
        v[k].get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(g[k], f[e], acc[e]);
      }
    }
    if (residual) {
      float f[E];
      r.get(f);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = f[e] + acc[e];
    }
    Unit<Tt, E>::store(y + t * p.ld_token + c, acc);
  }
}

// The gradient of the way back.  wpt warps share a token's row; a chunk of dy
// (B units a lane) stays in registers while the token's slots pass, the next
// slot's row already on its way.
template <typename Tt, typename Ts, int E>
__global__ void __launch_bounds__(256)
    rows_unsort_grad_kernel(const RowsArgs p, const Tt *dy, const Ts *ys,
                            const float *gate, const int32_t *pos, Ts *dys,
                            float *dgate, int wpt) {
  constexpr int B = E == 1 ? 16 : 4;
  __shared__ float partial[8][16];
  previous_done();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t64 = static_cast<int64_t>(blockIdx.x) * (8 / wpt) + warp / wpt;
  const int t = static_cast<int>(t64);
  const int w = warp % wpt;
  const int units = (p.H + E - 1) / E;
  // whole chunks to each warp, the row's ragged end to the last
  const int share = ((units + wpt - 1) / wpt + 32 * B - 1) / (32 * B) * (32 * B);
  const int begin = min(units, w * share), end = min(units, begin + share);
  float dot = 0.f;  // lane k: the k-th slot's
  if (t64 < p.T) {
    int mine = -1;  // lane k: the token's k-th position (k <= 16)
    float my_gate = 1.f;
    if (lane < p.K) {
      mine = row_pos(pos[t * p.K + lane], p.P, p.err);
      if (gate) my_gate = gate[static_cast<int64_t>(t) * p.K + lane];
    } else if (lane == p.K && p.has_shared) {
      mine = row_pos(pos[p.T * p.K + t], p.P, p.err);
    }
    auto chunk = [&](int u0, auto full) {
      constexpr bool kFull = decltype(full)::value;
      const Tt *dy_at = dy + t * p.ld_token + (u0 + lane) * E;
      auto inside = [&](int j) { return kFull || u0 + j * 32 + lane < end; };
      Unit<Tt, E> d[B];
#pragma unroll
      for (int j = 0; j < B; ++j)
        if (inside(j)) d[j].load(dy_at + j * 32 * E);
      Unit<Ts, E> v[B];
      auto fetch = [&](int k) {
        const int at = k < p.K ? __shfl_sync(0xffffffffu, mine, k) : -1;
        if (!dgate || at < 0) return;
        const Ts *src = ys + at * p.ld_slot + (u0 + lane) * E;
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (inside(j)) v[j].load(src + j * 32 * E);
      };
      fetch(0);
      for (int k = 0; k < p.K + p.has_shared; ++k) {
        const int at = __shfl_sync(0xffffffffu, mine, k);
        const float g = __shfl_sync(0xffffffffu, my_gate, k);
        float s = 0.f;
        if (dgate && k < p.K && at >= 0) {
#pragma unroll
          for (int j = 0; j < B; ++j)
            if (inside(j)) {
              float a[E], b[E];
              d[j].get(a);
              v[j].get(b);
#pragma unroll
              for (int e = 0; e < E; ++e) s = fmaf(a[e], b[e], s);
            }
        }
        if (k + 1 < p.K) fetch(k + 1);
        if (dgate && k < p.K) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == k) dot += s;
        }
        if (dys && at >= 0) {
          Ts *dst = dys + at * p.ld_dys + (u0 + lane) * E;
#pragma unroll
          for (int j = 0; j < B; ++j)
            if (inside(j)) {
              float a[E];
              d[j].get(a);
#pragma unroll
              for (int e = 0; e < E; ++e) a[e] *= g;
              Unit<Ts, E>::store(dst + j * 32 * E, a);
            }
        }
      }
    };
    int u0 = begin;
    for (; u0 + 32 * B <= end; u0 += 32 * B) chunk(u0, std::true_type{});
    if (u0 < end) chunk(u0, std::false_type{});
  }
  if (!dgate) return;
  if (lane < p.K) partial[warp][lane] = dot;
  __syncthreads();
  if (t64 < p.T && w == 0 && lane < p.K) {
    float s = 0.f;
    for (int j = 0; j < wpt; ++j) s += partial[warp + j][lane];
    dgate[static_cast<int64_t>(t) * p.K + lane] = s;
  }
}

namespace {

bool is_aligned(const void *p, int64_t pitch_bytes, int a) {
  return !p || (reinterpret_cast<uintptr_t>(p) % a == 0 && pitch_bytes % a == 0);
}

struct SortPtrs {
  const void *x;
  const float *x_scale;
  const int32_t *offsets, *sorted;
  int32_t *pos;
  void *xs;
  float *xs_scale;
};

template <typename W>
cudaError_t launch_sort_w(const RowsArgs &p, const SortPtrs &a, int elem, int num_sms, cudaStream_t stream) {
  int wpt = 1;  // warps per token: at least ~32 warps per SM in flight
  while (wpt < 8 && static_cast<int64_t>(p.T) * wpt < num_sms * 32) wpt *= 2;
  const int64_t blocks = (static_cast<int64_t>(p.T) * wpt + 7) / 8, cap = num_sms * 16ll;
  const unsigned grid = static_cast<unsigned>(blocks < cap ? blocks : cap);
  const uint8_t *x = static_cast<const uint8_t *>(a.x);
  uint8_t *xs = static_cast<uint8_t *>(a.xs);
  const int64_t row = static_cast<int64_t>(p.H) * elem;
  if (p.P <= kSmallPositions) {
    return launch_overlapped(rows_sort_small_kernel<W>, grid, 256, 0, stream, p, a.offsets, a.sorted, a.pos, x, xs,
                             a.x_scale, a.xs_scale, row, p.ld_token * elem, p.ld_slot * elem, wpt);
  }
  cudaError_t e = cudaMemsetAsync(a.pos, 0xff, sizeof(int32_t) * static_cast<size_t>(p.P), stream);
  if (e != cudaSuccess) return e;
  const int64_t inv = (p.P + 255ll) / 256, inv_cap = num_sms * 8ll;
  e = launch_overlapped(rows_invert_kernel, static_cast<unsigned>(inv < inv_cap ? inv : inv_cap), 256, 0, stream, p,
                        a.offsets, a.sorted, a.pos);
  if (e != cudaSuccess) return e;
  return launch_overlapped(rows_scatter_kernel<W>, grid, 256, 0, stream, p, a.pos, x, xs, a.x_scale, a.xs_scale,
                           row, p.ld_token * elem, p.ld_slot * elem, wpt);
}

template <typename Tt, typename Ts, int E>
cudaError_t launch_unsort_e(const RowsArgs &p, const void *ys, const float *gate, const int32_t *pos,
                            const void *residual, void *y, cudaStream_t stream) {
  const int units = (p.H + E - 1) / E;
  int log2 = 0;  // threads per token
  while (log2 < 8 && (1 << log2) < units) ++log2;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.T) + (256 >> log2) - 1) >> (8 - log2));
  auto go = [&](auto kern) {
    return launch_overlapped(kern, grid, 256, 0, stream, p, static_cast<const Ts *>(ys), gate, pos,
                             static_cast<const Tt *>(residual), static_cast<Tt *>(y), log2);
  };
  // Straight-line code for the usual numbers of rows a token, 4 or 8 experts with
  // and without a shared one; the others test each row.  What the tests cost (us,
  // straight-line / tested): 16384 tokens x 9 rows of 6144 320 / 642, x 5 178 / 204,
  // 4096 x 9 of 2048 38.0 / 78.5, x 5 20.3 / 24.9, 64 x 9 of 6144 3.2 / 4.9.
  const int n = p.K + p.has_shared;
  if (n == 4) return go(rows_unsort_kernel<Tt, Ts, E, 4, true>);
  if (n == 5) return go(rows_unsort_kernel<Tt, Ts, E, 5, true>);
  if (n == 8) return go(rows_unsort_kernel<Tt, Ts, E, 8, true>);
  if (n == 9) return go(rows_unsort_kernel<Tt, Ts, E, 9, true>);
  if (n < 8) return go(rows_unsort_kernel<Tt, Ts, E, 7, false>);
  return go(rows_unsort_kernel<Tt, Ts, E, 17, false>);
}

template <typename Tt, typename Ts, int E>
cudaError_t launch_grad_e(const RowsArgs &p, const void *dy, const void *ys, const float *gate,
                          const int32_t *pos, void *dys, float *dgate, int num_sms, cudaStream_t stream) {
  int wpt = 1;
  while (wpt < 8 && static_cast<int64_t>(p.T) * wpt < num_sms * 32) wpt *= 2;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.T) + 8 / wpt - 1) / (8 / wpt));
  return launch_overlapped(rows_unsort_grad_kernel<Tt, Ts, E>, grid, 256, 0, stream, p, static_cast<const Tt *>(dy),
                           static_cast<const Ts *>(ys), gate, pos, static_cast<Ts *>(dys), dgate, wpt);
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
  const int64_t row = static_cast<int64_t>(p.H) * elem;
  const SortPtrs a = {x, x_scale, offsets, sorted, pos, xs, xs_scale};
  auto fits = [&](int n) {
    return row % n == 0 && is_aligned(x, p.ld_token * elem, n) && is_aligned(xs, p.ld_slot * elem, n);
  };
  if (fits(16)) return launch_sort_w<uint4>(p, a, elem, num_sms, stream);
  if (fits(8)) return launch_sort_w<uint2>(p, a, elem, num_sms, stream);
  if (fits(4)) return launch_sort_w<uint32_t>(p, a, elem, num_sms, stream);
  if (fits(2)) return launch_sort_w<uint16_t>(p, a, elem, num_sms, stream);
  return launch_sort_w<uint8_t>(p, a, elem, num_sms, stream);
}

cudaError_t launch_rows_unsort(const RowsArgs &p, int dtype, int slot_dtype, const void *ys,
                               const float *gate, const int32_t *pos, const void *residual, void *y,
                               cudaStream_t stream) {
  return by_types(dtype, slot_dtype, [&](auto tt, auto ts) {
    using Tt = decltype(tt);
    using Ts = decltype(ts);
    const int64_t a = sizeof(Tt), b = sizeof(Ts);
    if (p.H % 8 == 0 && is_aligned(ys, p.ld_slot * b, 16) && is_aligned(residual, p.ld_residual * a, 16) &&
        is_aligned(y, p.ld_token * a, 16))
      return launch_unsort_e<Tt, Ts, 8>(p, ys, gate, pos, residual, y, stream);
    return launch_unsort_e<Tt, Ts, 1>(p, ys, gate, pos, residual, y, stream);
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
