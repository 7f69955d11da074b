// Elements of the tensors that the operators around the cache take: fp32, bf16
// and fp16, eight at a time or single ones.
#pragma once

#include <cstdint>

namespace spec {

constexpr int DT_F32 = 0, DT_BF16 = 1, DT_F16 = 2;  // SPEC_F32, SPEC_BF16, SPEC_F16

// Eight elements of a row as loaded: one 16-byte vector, or two for fp32.
template <int DT>
struct Raw8 {
  uint4 v[DT == DT_F32 ? 2 : 1];
};

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f32_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f32_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DT>
__device__ __forceinline__ float one_element(const void *base, long long i) {
  if (DT == DT_F32) return static_cast<const float *>(base)[i];
  const uint16_t h = static_cast<const uint16_t *>(base)[i];
  if (DT == DT_BF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return f16x2_to_f32(h).x;
}
template <int DT>
__device__ __forceinline__ void put_element(void *base, long long i, float x) {
  if (DT == DT_F32) static_cast<float *>(base)[i] = x;
  else if (DT == DT_BF16) static_cast<uint16_t *>(base)[i] = static_cast<uint16_t>(f32_to_bf16x2(x, 0.f));
  else static_cast<uint16_t *>(base)[i] = static_cast<uint16_t>(f32_to_f16x2(x, 0.f));
}

// The eight elements from element offset i; VEC: 16-byte aligned there.
template <int DT, bool VEC>
__device__ __forceinline__ Raw8<DT> load8(const void *base, long long i) {
  Raw8<DT> r;
  if constexpr (VEC) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + i * (DT == DT_F32 ? 4 : 2));
    r.v[0] = p[0];
    if constexpr (DT == DT_F32) r.v[1] = p[1];
  } else if constexpr (DT == DT_F32) {
    const uint32_t *p = static_cast<const uint32_t *>(base) + i;
    r.v[0] = make_uint4(p[0], p[1], p[2], p[3]);
    r.v[1] = make_uint4(p[4], p[5], p[6], p[7]);
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + i;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = p[2 * j] | static_cast<uint32_t>(p[2 * j + 1]) << 16;
    r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT> &r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  if constexpr (DT == DT_F32) {
    const uint32_t u[4] = {r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = __uint_as_float(w[j]);
      x[4 + j] = __uint_as_float(u[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (DT == DT_BF16) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        const float2 f = f16x2_to_f32(w[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
  }
}
// One rounding, from fp32 to the output's type.
template <int DT>
__device__ __forceinline__ Raw8<DT> pack8(const float (&x)[8]) {
  Raw8<DT> r;
  if constexpr (DT == DT_F32) {
    r.v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    r.v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = DT == DT_BF16 ? f32_to_bf16x2(x[2 * j], x[2 * j + 1]) : f32_to_f16x2(x[2 * j], x[2 * j + 1]);
    r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}
template <int DT, bool VEC>
__device__ __forceinline__ void store8(void *base, long long i, const Raw8<DT> &r) {
  if constexpr (VEC) {
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<char *>(base) + i * (DT == DT_F32 ? 4 : 2));
    p[0] = r.v[0];
    if constexpr (DT == DT_F32) p[1] = r.v[1];
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
    if constexpr (DT == DT_F32) {
      const uint32_t u[4] = {r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
      uint32_t *p = static_cast<uint32_t *>(base) + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = w[j];
        p[4 + j] = u[j];
      }
    } else {
      uint16_t *p = static_cast<uint16_t *>(base) + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[2 * j] = static_cast<uint16_t>(w[j]);
        p[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
      }
    }
  }
}

}  // namespace spec
