// glu_grad.cuh -- the gate of a block that is trained, for the endings that store h beside
// g and u, and a gate's activation and derivative, for those that make dg and du from dh
// (mlp_train.cu, gemm_tc.cu).
#pragma once

#include <cstdint>

#include "common.cuh"

namespace gbf {

__device__ __forceinline__ float mb_pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float mb_rcp(float x) {  // 0 for infinity
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float mb_clamp(float v, float most) {  // a NaN stays one
  float y;
  asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}"
      : "=f"(y) : "f"(v), "f"(most), "f"(-most));
  return y;
}

__device__ __forceinline__ float mb_relu(float v) {  // a NaN stays one
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(v));
  return y;
}

// h = act(g) u of 32 columns.  A NaN in g is one in h, with every gate.
template <int ACT>
__device__ __forceinline__ float gate(float g) {
  if constexpr (ACT == kActRelu) return mb_relu(g);
  else return act_apply<ACT>(g);
}
template <int ACT>
__device__ __forceinline__ void glu_pack_act(const uint32_t (&g)[32], const uint32_t (&u)[32],
                                             uint32_t (&w)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k)
    w[k] = pack_bf16x2(
        gate<ACT>(__uint_as_float(g[2 * k])) * __uint_as_float(u[2 * k]),
        gate<ACT>(__uint_as_float(g[2 * k + 1])) * __uint_as_float(u[2 * k + 1]));
}
__device__ __forceinline__ void glu_pack(int act, const uint32_t (&g)[32], const uint32_t (&u)[32],
                                         uint32_t (&w)[16]) {
  switch (act) {
    case kActRelu: glu_pack_act<kActRelu>(g, u, w); break;
    case kActSilu: glu_pack_act<kActSilu>(g, u, w); break;
    case kActGeluTanh: glu_pack_act<kActGeluTanh>(g, u, w); break;
    default: glu_pack_act<kActIdentity>(g, u, w); break;
  }
}

// Two fp32 values at a time, each operation rounded as the scalar one.
struct f2 {
  uint64_t v;
};
__device__ __forceinline__ f2 f2_of(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 f2_all(float x) { return f2_of(x, x); }
__device__ __forceinline__ void f2_get(f2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v));
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// 1 / (1 + 2^x)
__device__ __forceinline__ f2 f2_sigmoid2(f2 x) {
  float a, b;
  f2_get(x, a, b);
  return f2_of(mb_rcp(1.0f + mb_pow2(a)), mb_rcp(1.0f + mb_pow2(b)));
}

// Activation and derivative, in as few operations as it takes: they run on every
// element of dh, and with a short K (D = 1000) the ending is what a unit waits for.
template <int ACT>
__device__ __forceinline__ void act_both(f2 v, f2& y, f2& dy) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (ACT == kActRelu) {
    float a, b;
    f2_get(v, a, b);
    y = f2_of(mb_relu(a), mb_relu(b));
    dy = f2_of(a > 0.0f ? 1.0f : 0.0f, b > 0.0f ? 1.0f : 0.0f);
  } else if constexpr (ACT == kActSilu) {
    const f2 s = f2_sigmoid2(f2_mul(v, f2_all(-kLog2e)));
    y = f2_mul(v, s);
    dy = f2_mul(s, f2_fma(v, f2_fma(s, f2_all(-1.0f), f2_all(1.0f)), f2_all(1.0f)));
  } else if constexpr (ACT == kActGeluTanh) {
    // y = v s(2 z), z = c (v + k v^3);  y' = s + s (1 - s) v 2 c (1 + 3 k v^2).  From
    // |v| = 30 on s is 0 or 1 and the second term 0; v^2 stays in range.
    constexpr float c = 0.7978845608028654f, k = 0.044715f;
    float a, b;
    f2_get(v, a, b);
    const f2 x = f2_of(mb_clamp(a, 30.0f), mb_clamp(b, 30.0f));
    const f2 x2 = f2_mul(x, x);
    const f2 s = f2_sigmoid2(f2_mul(
        x, f2_fma(x2, f2_all(-2.0f * kLog2e * c * k), f2_all(-2.0f * kLog2e * c))));
    y = f2_mul(v, s);
    const f2 t = f2_mul(f2_fma(f2_mul(s, f2_all(-1.0f)), s, s), x);
    dy = f2_fma(t, f2_fma(x2, f2_all(6.0f * c * k), f2_all(2.0f * c)), s);
  } else {
    y = v;
    dy = f2_all(1.0f);
  }
}

}  // namespace gbf
