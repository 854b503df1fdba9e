// The epilogue of the dense linear (its formulas in float32) and
// the slope its backward multiplies with, shared by every kernel that ends or
// begins with them:
//   u = acc * scale[n] + bias[n],  y = act(u) + residual.
//
// acc, u and act(u) stay in float32; y and the kept u are each rounded once.
//
//   silu(u)      = u p,  p = 1 / (1 + e^-u);          slope p + u p (1 - p)
//   gelu_tanh(u) = u p,  p = (1 + tanh z) / 2 = 1 / (1 + e^-2z),
//                  z = C (u + A u^3);                 slope p + u p (1 - p) 2 z'
//   gelu(u)      = u Phi(u);                          slope Phi(u) + u phi(u)
// Phi(-|u|) = erfc(|u| / sqrt 2) / 2 by the rational approximation 7.1.26 of
// Abramowitz and Stegun's handbook (absolute error 1.5e-7, a float32 rounding
// of the sum 1 + erf it replaces): one exponential, which phi shares, one
// reciprocal and five products, where a library erf costs several times that
// in the epilogue of a matrix product.
// A NaN u stays NaN, +inf stays +inf (-inf gives NaN where the formula is
// -inf times 0); the slopes take |u| > 64 as 64, where they equal their
// limits 0 and 1 in float32 and u^2 cannot overflow.
#pragma once

#include "common.h"
#include "kernels.h"

namespace poetx {

constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;

__device__ __forceinline__ float logistic(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

// Phi(-|u|); *gauss = exp(-u^2 / 2)
__device__ __forceinline__ float normal_tail(float u, float* gauss) {
  const float z = fabsf(u) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, z, 1.0f));
  const float e = __expf(-z * z);
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  *gauss = e;
  return 0.5f * p * t * e;
}

template <Activation ACT> __device__ __forceinline__ float activate(float u) {
  if constexpr (ACT == Activation::Relu) return u < 0.0f ? 0.0f : u;
  if constexpr (ACT == Activation::Silu) return u * logistic(u);
  if constexpr (ACT == Activation::GeluTanh)
    return u * logistic(2.0f * kGeluC * fmaf(kGeluA * u * u, u, u));
  if constexpr (ACT == Activation::Gelu) {
    float e;
    const float q = normal_tail(u, &e);
    return u * (u < 0.0f ? q : 1.0f - q);
  }
  return u;
}

template <Activation ACT> __device__ __forceinline__ float activation_slope(float u) {
  const float v = u > 64.0f ? 64.0f : u < -64.0f ? -64.0f : u;
  if constexpr (ACT == Activation::Silu) {
    const float p = logistic(v);
    return fmaf(v * p, 1.0f - p, p);
  }
  if constexpr (ACT == Activation::GeluTanh) {
    const float w = kGeluA * v * v;
    const float p = logistic(2.0f * kGeluC * fmaf(w, v, v));
    return fmaf(v * p * (1.0f - p), 2.0f * kGeluC * fmaf(3.0f, w, 1.0f), p);
  }
  float e;
  const float q = normal_tail(v, &e);
  return fmaf(v * 0.3989422804014327f, e, v < 0.0f ? q : 1.0f - q);
}

// g times the slope at u; relu's is a choice, not a product, so that an
// infinite g (a loss scale that overflowed) is dropped where the unit is off
template <Activation ACT> __device__ __forceinline__ float activation_gradient(float g, float u) {
  if constexpr (ACT == Activation::Relu) return u <= 0.0f ? 0.0f : g;
  else return g * activation_slope<ACT>(u);
}

// the run-time activation of a wave-uniform `act`, four values at a time
__device__ __forceinline__ void activate4(int act, float v[4]) {
#define POETX_ACTIVATE4(A)                                              \
  case static_cast<int>(Activation::A):                                 \
    for (int e = 0; e < 4; ++e) v[e] = activate<Activation::A>(v[e]);   \
    break;
  switch (act) {
    POETX_ACTIVATE4(Relu)
    POETX_ACTIVATE4(Gelu)
    POETX_ACTIVATE4(GeluTanh)
    POETX_ACTIVATE4(Silu)
    default:
      break;
  }
#undef POETX_ACTIVATE4
}

// four consecutive values, 8 (bf16) or 16 (float32) bytes
template <typename T> struct Quad;
template <> struct Quad<bf16_t> {
  static __device__ __forceinline__ void load(const bf16_t* p, float v[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  static __device__ __forceinline__ uint2 pack(const float v[4]) {
    union { bf16_t h[4]; uint2 w; } o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o.h[e] = f32_to_bf16(v[e]);
    return o.w;
  }
  static __device__ __forceinline__ void store(bf16_t* p, const float v[4]) {
    *reinterpret_cast<uint2*>(p) = pack(v);
  }
};
template <> struct Quad<float> {
  static __device__ __forceinline__ void load(const float* p, float v[4]) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
  static __device__ __forceinline__ void store(float* p, const float v[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

// columns n .. n + 3 (n % 4 == 0, inside the row) of output row m from their
// float32 products
template <typename T>
__device__ __forceinline__ void epilogue4(const Epilogue& ep, int64_t m, int n, float v[4]) {
  if (ep.scale) {
    const float4 s = *reinterpret_cast<const float4*>(ep.scale + n);
    v[0] *= s.x; v[1] *= s.y; v[2] *= s.z; v[3] *= s.w;
  }
  if (ep.bias) {
    const float4 b = *reinterpret_cast<const float4*>(ep.bias + n);
    v[0] += b.x; v[1] += b.y; v[2] += b.z; v[3] += b.w;
  }
  const int64_t at = m * ep.ld + n;
  if (ep.u) Quad<T>::store(static_cast<T*>(ep.u) + at, v);
  activate4(ep.act, v);
  if (ep.residual) {
    float r[4];
    Quad<T>::load(static_cast<const T*>(ep.residual) + at, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += r[e];
  }
  Quad<T>::store(static_cast<T*>(ep.y) + at, v);
}

}  // namespace poetx
