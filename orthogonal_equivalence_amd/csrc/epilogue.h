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
//
// float32 tensors (kPrecise): the exponential, the complementary error function
// and the quotient to float32's last place, and 1 - p as e^-v p where it is
// small: within about one rounding a step of the formula. 2048 x 2048 g_bias
// (the slopes alone) gelu 14.7 us, gelu_tanh 12.9, silu 12.7, in the bf16 forms
// 12.5, 12.0 and 11.8; a forward takes 0 to 3% longer.
//
// bf16 tensors: their last place is 2^16 times float32's, so the cheapest
// forms that are good to 1.5e-7: the hardware's exponential and reciprocal, and
// Phi(-|u|) = erfc(|u| / sqrt 2) / 2 by the rational approximation 7.1.26 of
// Abramowitz and Stegun's handbook (absolute error 1.5e-7): one exponential,
// which phi shares, one reciprocal and five products in the epilogue of a
// matrix product, where erfc costs several times that.
//
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

// 2 z of gelu_tanh
__device__ __forceinline__ float tanh_argument(float u) {
  return 2.0f * kGeluC * fmaf(kGeluA * u * u, u, u);
}

// whether the activations of T tensors take the forms for float32
template <typename T> constexpr bool kPrecise = sizeof(T) == 4;

template <typename T, Activation ACT> __device__ __forceinline__ float activate(float u) {
  if constexpr (ACT == Activation::Relu) return u < 0.0f ? 0.0f : u;
  if constexpr (ACT == Activation::Silu)
    return kPrecise<T> ? u / (1.0f + expf(-u)) : u * logistic(u);
  if constexpr (ACT == Activation::GeluTanh)
    return kPrecise<T> ? u / (1.0f + expf(-tanh_argument(u))) : u * logistic(tanh_argument(u));
  if constexpr (ACT == Activation::Gelu) {
    if constexpr (kPrecise<T>) return u * (0.5f * erfcf(u * -0.70710678118654752f));
    float e;
    const float q = normal_tail(u, &e);
    return u * (u < 0.0f ? q : 1.0f - q);
  }
  return u;
}

// e^v for v <= 88 within about one step of float32: what v / ln 2 loses by its
// rounding, times ln 2, corrects the hardware's 2^x
__device__ __forceinline__ float exp_below(float v) {
  constexpr float kHi = 1.44269504f, kLo = 1.92596299e-8f;  // 1 / ln 2
  const float t = v * kHi, rest = fmaf(v, kLo, fmaf(v, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, rest * 0.69314718f, e);
}

// the slope of v p(s(v)), p the logistic function and ds the slope of s. In the
// precise form |s| is cut at 87, where p is 0 or 1 to 2e-38, for exp_below and
// the reciprocal, a Newton step of the hardware's: 2048 x 2048 silu 12.7 us, with
// expf and a division 14.2, in the bf16 form 11.8.
template <typename T>
__device__ __forceinline__ float logistic_slope(float v, float s, float ds) {
  if constexpr (kPrecise<T>) {
    const float c = s > 87.0f ? 87.0f : s < -87.0f ? -87.0f : s;
    const float e = exp_below(-c), d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
    const float p = fmaf(r, fmaf(-d, r, 1.0f), r);
    return fmaf(v * p * (s > 0.0f ? e * p : 1.0f - p), ds, p);
  } else {
    const float p = logistic(s);
    return fmaf(v * p * (1.0f - p), ds, p);
  }
}

template <typename T, Activation ACT> __device__ __forceinline__ float activation_slope(float u) {
  const float v = u > 64.0f ? 64.0f : u < -64.0f ? -64.0f : u;
  if constexpr (ACT == Activation::Silu) return logistic_slope<T>(v, v, 1.0f);
  if constexpr (ACT == Activation::GeluTanh)
    return logistic_slope<T>(v, tanh_argument(v),
                             2.0f * kGeluC * fmaf(3.0f, kGeluA * v * v, 1.0f));
  if constexpr (kPrecise<T>)
    return fmaf(v * 0.3989422804014327f, exp_below(-0.5f * v * v),
                0.5f * erfcf(v * -0.70710678118654752f));
  float e;
  const float q = normal_tail(v, &e);
  return fmaf(v * 0.3989422804014327f, e, v < 0.0f ? q : 1.0f - q);
}

// g times the slope at u; relu's is a choice, not a product, so that an
// infinite g (a loss scale that overflowed) is dropped where the unit is off
template <typename T, Activation ACT>
__device__ __forceinline__ float activation_gradient(float g, float u) {
  if constexpr (ACT == Activation::Relu) return u <= 0.0f ? 0.0f : g;
  else return g * activation_slope<T, ACT>(u);
}

// the run-time activation of a wave-uniform `act`, four values at a time
template <typename T> __device__ __forceinline__ void activate4(int act, float v[4]) {
#define POETX_ACTIVATE4(A)                                                \
  case static_cast<int>(Activation::A):                                   \
    for (int e = 0; e < 4; ++e) v[e] = activate<T, Activation::A>(v[e]);  \
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
  if (ep.add) {
    float a[4];
    Quad<float>::load(ep.add + at, a);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += a[e];
  }
  if (ep.sum) {
    Quad<float>::store(ep.sum + at, v);
    return;
  }
  if (ep.u) Quad<T>::store(static_cast<T*>(ep.u) + at, v);
  activate4<T>(ep.act, v);
  if (ep.residual) {
    float r[4];
    Quad<T>::load(static_cast<const T*>(ep.residual) + at, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += r[e];
  }
  Quad<T>::store(static_cast<T*>(ep.y) + at, v);
}

}  // namespace poetx
