// rowio.cuh -- element types of the row kernels (q8_norm.cu, rows.cu,
// q8_gemm.cu): E consecutive elements as loaded and as fp32 values, and stores.
#pragma once

#include "common.cuh"

namespace srm {

// The storage type of each element type: bf16 and fp16 as distinct structs of
// 16 bits, so that overloads tell them apart.
struct Bf16 {
  uint16_t v;
};
struct Fp16 {
  uint16_t v;
};

__device__ __forceinline__ float to_float(Bf16 a) { return bf16_bits_to_float(a.v); }
__device__ __forceinline__ float to_float(Fp16 a) { return __half2float(__ushort_as_half(a.v)); }
__device__ __forceinline__ float to_float(float a) { return a; }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ Bf16 from_float<Bf16>(float v) {
  return Bf16{__bfloat16_as_ushort(__float2bfloat16_rn(v))};
}
template <>
__device__ __forceinline__ Fp16 from_float<Fp16>(float v) {
  return Fp16{__half_as_ushort(__float2half_rn(v))};
}
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}

// Two floats rounded to T in one 32-bit word (16-bit types), low half first.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<Bf16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<Fp16>(float lo, float hi) {
  __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&p);
}

__device__ __forceinline__ void unpack2(Bf16, uint32_t w, float &lo, float &hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack2(Fp16, uint32_t w, float &lo, float &hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  lo = f.x;
  hi = f.y;
}

// (a, b) * (c, d) in one operation
__device__ __forceinline__ void mul2(float &a, float &b, float c, float d) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

// One 16-byte vector of T and its element count; E = 1 is the form for rows
// that are not 16-byte aligned.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

template <typename T, int E>
struct RowIo {  // E = kVec<T>, 16-bit types
  using Raw = uint4;  // the elements as loaded
  static __device__ __forceinline__ void unpack(const uint4 &r, float (&f)[E]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack2(T{}, w[k], f[2 * k], f[2 * k + 1]);
  }
  static __device__ __forceinline__ void store(T *p, const float (&f)[E]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]),
                                               pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
  }
};
template <>
struct RowIo<float, 4> {
  using Raw = uint4;
  static __device__ __forceinline__ void unpack(const uint4 &r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ void store(float *p, const float (&f)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <typename T>
struct RowIo<T, 1> {
  using Raw = T;
  static __device__ __forceinline__ void unpack(const T &r, float (&f)[1]) { f[0] = to_float(r); }
  static __device__ __forceinline__ void store(T *p, const float (&f)[1]) { *p = from_float<T>(f[0]); }
};

}  // namespace srm
