// What the kernels of the gated linear layer share (fm_ops.h).
#pragma once

#include <cuda_fp8.h>

#include "fm_ops.cuh"

namespace fm {

struct E4M3 {
  uint8_t bits;
};
template <>
__device__ __forceinline__ float to_f<E4M3>(E4M3 x) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(x.bits, __NV_E4M3);
  return __half2float(__half(h));
}

struct GatedParams {
  long long rows;
  int width, hidden;
  int act;
  long long xs, gs, us, hs, dhs, dxs, dgs, dus;
  const void *x, *wg, *wu, *dh;
  const float *x_scales, *g_scales, *u_scales;  // NULL: ones
  void *h, *dx, *dwg, *dwu;
};

// 1 / (1 + e^-g) and what it lacks of one, each to a few of its last places on both sides:
// by e^-|g|, which does not overflow, and an exponential that rounds its argument once
// (the fast one is off by 50 last places at g = -40).
__device__ __forceinline__ float sigmoid_of(float g) {
  const float e = expf(-fabsf(g));
  return (g < 0.f ? e : 1.f) / (1.f + e);
}
__device__ __forceinline__ float sigmoid_of(float g, float& rest) {
  const float e = expf(-fabsf(g)), one = 1.f / (1.f + e);
  rest = g < 0.f ? one : e * one;
  return g < 0.f ? e * one : one;
}
// The normal distribution's integral up to g, by erfc: 1 + erf of a g far below zero would
// leave none of its digits (g = -5.5: half of it, -6: nothing).
__device__ __forceinline__ float normal_integral(float g) { return 0.5f * erfcf(g * -0.70710678118654752f); }
template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if (ACT == FM_ACT_SILU) return g * sigmoid_of(g);
  if (ACT == FM_ACT_GELU) return g * normal_integral(g);
  if (ACT == FM_ACT_SIGMOID) return sigmoid_of(g);
  return g > 0.f || g != g ? g : 0.f;
}
// act(g) and its slope
template <int ACT>
__device__ __forceinline__ void act_and_slope(float g, float& a, float& slope) {
  if (ACT == FM_ACT_SILU) {
    float rest;
    const float s = sigmoid_of(g, rest);
    a = g * s;
    slope = s * (1.f + g * rest);
  } else if (ACT == FM_ACT_GELU) {
    const float c = normal_integral(g);
    a = g * c;
    slope = fmaf(g * 0.39894228040143268f, expf(-0.5f * g * g), c);
  } else if (ACT == FM_ACT_SIGMOID) {
    float rest;
    a = sigmoid_of(g, rest);
    slope = a * rest;
  } else {
    a = g > 0.f || g != g ? g : 0.f;
    slope = g > 0.f ? 1.f : 0.f;
  }
}
// f(act) with the activation as a constant
template <typename F>
void with_act(int act, F f) {
  if (act == FM_ACT_SILU) f(std::integral_constant<int, FM_ACT_SILU>());
  else if (act == FM_ACT_GELU) f(std::integral_constant<int, FM_ACT_GELU>());
  else if (act == FM_ACT_SIGMOID) f(std::integral_constant<int, FM_ACT_SIGMOID>());
  else f(std::integral_constant<int, FM_ACT_RELU>());
}

}  // namespace fm
