// Activations of the FP8 layers and their slopes (fp8_matmul.cu, fp8_linear_backward.cu),
// two values at a time in packed fp32:
//
//   GELU       x Phi(x)                        Phi(x) + x phi(x)
//   GELU_TANH  x s, s = sigmoid(c (x + a x^3)) s + x s (1 - s) c (1 + 3 a x^2),
//              c = sqrt(8 / pi), a = 0.044715: the form with tanh, (1 + tanh(u)) / 2 = sigmoid(2 u)
//   SILU       x s, s = sigmoid(x)             s (1 + x (1 - s))
//   RELU       max(x, 0)                       1 where x > 0, else 0
//
// Phi's error function is Abramowitz and Stegun's 7.1.26, whose absolute error of
// 1.5e-7 is that of fp32 near 1. An exponential that is infinite gives a quotient
// of zero, as it should.
#pragma once

#include "fp8_block.cuh"

namespace taco {

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return f2{v, v}; }
__device__ __forceinline__ f2 ex2_2(f2 x) { return f2{ex2(x.x), ex2(x.y)}; }
// 1 / (1 + 2^t)
__device__ __forceinline__ f2 logistic2(f2 t) {
  const f2 d = add2(ex2_2(t), both(1.0f));
  return f2{reciprocal(d.x), reciprocal(d.y)};
}
constexpr float kLog2e = 1.44269504f;
constexpr float kTanhC = 1.59576912f;    // sqrt(8 / pi)
constexpr float kTanhA = 0.044715f;

// (1 - erf(z / sqrt 2)) / 2 of z = |x|, and e = exp(-x^2 / 2). From 64 on both are
// zero, and z may be held there.
__device__ __forceinline__ f2 upper_tail(f2 x, f2 z, f2& e) {
  const f2 d = fma2(z, both(0.3275911f * 0.70710678f), both(1.0f));
  const f2 t{reciprocal(d.x), reciprocal(d.y)};
  f2 p = fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
  p = fma2(p, t, both(0.5f * 1.421413741f));
  p = fma2(p, t, both(0.5f * -0.284496736f));
  p = fma2(p, t, both(0.5f * 0.254829592f));
  e = ex2_2(mul2(mul2(x, x), both(-0.5f * kLog2e)));
  return mul2(mul2(p, t), e);
}

template <int ACT>
__device__ __forceinline__ f2 activate2(f2 x) {
  if constexpr (ACT == TACO_ACT_GELU) {
    f2 e;
    const f2 z{fminf(fabsf(x.x), 64.0f), fminf(fabsf(x.y), 64.0f)}, h = upper_tail(x, z, e);
    const f2 top{x.x < 0.0f ? 0.0f : x.x, x.y < 0.0f ? 0.0f : x.y};
    // -|x| h, but no infinity times 0 at +infinity, which stays what it is (-infinity gives NaN, as the formula)
    return fma2(f2{fminf(x.x, -z.x), fminf(x.y, -z.y)}, h, top);
  } else if constexpr (ACT == TACO_ACT_GELU_TANH) {
    const f2 t = fma2(mul2(x, x), both(-kTanhC * kTanhA * kLog2e), both(-kTanhC * kLog2e));
    return mul2(x, logistic2(mul2(x, t)));
  } else if constexpr (ACT == TACO_ACT_SILU) {
    return mul2(x, logistic2(mul2(x, both(-kLog2e))));
  } else if constexpr (ACT == TACO_ACT_RELU) {
    return f2{x.x < 0.0f ? 0.0f : x.x, x.y < 0.0f ? 0.0f : x.y};   // a NaN stays one
  } else {
    return x;
  }
}

// Slopes take values up to 448 * 2^10 as they are (x^3 is far from fp32's end);
// larger ones are brought within [-64, 64] first, where every slope is 0 or 1 to
// fp32's last bit already, a NaN as it is. Whole blocks share the check, by their
// scale: above 2^kSlopeBinades.
constexpr uint32_t kSlopeBinades = 10;
template <int ACT, int N>
__device__ __forceinline__ void limit_for_slope(float (&x)[N]) {
  if (ACT == TACO_ACT_RELU) return;
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm("{ .reg .f32 t;\n min.NaN.f32 t, %0, 0f42800000;\n max.NaN.f32 %0, t, 0fC2800000; }" : "+f"(x[i]));
}
// s (1 + w (1 - s)) of s = 1 / (1 + 2^t), with 1 - s = 2^t s to its own
// precision. 2^t is held at 2^100, where s is small enough for any w (below 2^60).
__device__ __forceinline__ f2 logistic_slope(f2 t, f2 w) {
  const f2 e = ex2_2(f2{fminf(t.x, 100.0f), fminf(t.y, 100.0f)});
  const f2 d = add2(e, both(1.0f)), s{reciprocal(d.x), reciprocal(d.y)};
  return mul2(s, fma2(w, mul2(e, s), both(1.0f)));
}

template <int ACT>
__device__ __forceinline__ f2 slope2(f2 x) {
  if constexpr (ACT == TACO_ACT_GELU) {
    f2 e;
    const f2 h = upper_tail(x, f2{fabsf(x.x), fabsf(x.y)}, e);
    const f2 phi{x.x < 0.0f ? h.x : 1.0f - h.x, x.y < 0.0f ? h.y : 1.0f - h.y};
    return fma2(mul2(x, e), both(0.39894228f), phi);
  } else if constexpr (ACT == TACO_ACT_GELU_TANH) {
    const f2 q = mul2(x, x);
    const f2 t = mul2(x, fma2(q, both(-kTanhC * kTanhA * kLog2e), both(-kTanhC * kLog2e)));
    return logistic_slope(t, mul2(x, fma2(q, both(3.0f * kTanhC * kTanhA), both(kTanhC))));
  } else if constexpr (ACT == TACO_ACT_SILU) {
    return logistic_slope(mul2(x, both(-kLog2e)), x);
  } else if constexpr (ACT == TACO_ACT_RELU) {
    const auto step = [](float v) { return v > 0.0f ? 1.0f : v <= 0.0f ? 0.0f : v; };   // a NaN stays one
    return f2{step(x.x), step(x.y)};
  } else {
    return both(1.0f);
  }
}

// f(integral_constant) for the activation `act`.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case TACO_ACT_GELU: return f(std::integral_constant<int, TACO_ACT_GELU>{});
    case TACO_ACT_GELU_TANH: return f(std::integral_constant<int, TACO_ACT_GELU_TANH>{});
    case TACO_ACT_SILU: return f(std::integral_constant<int, TACO_ACT_SILU>{});
    case TACO_ACT_RELU: return f(std::integral_constant<int, TACO_ACT_RELU>{});
    default: return;
  }
}
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  with_act(act, [&](auto kind) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const f2 y = activate2<decltype(kind)::value>(f2{v[i], v[i + 1]});
      v[i] = y.x;
      v[i + 1] = y.y;
    }
  });
}

}  // namespace taco
