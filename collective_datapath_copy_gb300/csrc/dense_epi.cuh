// Scalar pieces of the dense operators: conversions, activations with their slopes, and the
// epilogue of one run of eight columns of one row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dense.h"

namespace coll {

__device__ __forceinline__ float h2f(uint16_t v, int type) {
  return type == COLL_BF16 ? __uint_as_float((uint32_t)v << 16)
                           : __half2float(__ushort_as_half(v));
}

__device__ __forceinline__ uint16_t f2h(float v, int type) {
  return type == COLL_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                           : __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ uint32_t f2h2(float lo, float hi, int type) {
  if (type == COLL_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void h2f2(uint32_t w, int type, float &lo, float &hi) {
  lo = h2f((uint16_t)(w & 0xFFFFu), type);
  hi = h2f((uint16_t)(w >> 16), type);
}

__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kRsqrt2 = 0.70710678118654752f;
constexpr float kRsqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case COLL_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case COLL_ACT_GELU: return 0.5f * z * (1.0f + erff(z * kRsqrt2));
    case COLL_ACT_GELU_TANH:
      // (1 + tanh(a)) / 2 = logistic(2 a)
      return z * logistic(2.0f * kTanhScale * fmaf(kTanhCubic * z * z, z, z));
    case COLL_ACT_SILU: return z * logistic(z);
    case COLL_ACT_SIGMOID: return logistic(z);
    default: return z;
  }
}

// value and slope together (the backward calls' elementwise step)
__device__ __forceinline__ void act_value_slope(float z, int act, float &v, float &d) {
  switch (act) {
    case COLL_ACT_RELU:
      v = z > 0.0f ? z : (z != z ? z : 0.0f);
      d = z > 0.0f ? 1.0f : 0.0f;
      return;
    case COLL_ACT_GELU: {
      const float c = 0.5f * (1.0f + erff(z * kRsqrt2));
      v = z * c;
      d = fmaf(z * kRsqrt2Pi, __expf(-0.5f * z * z), c);
      return;
    }
    case COLL_ACT_GELU_TANH: {
      const float s = logistic(2.0f * kTanhScale * fmaf(kTanhCubic * z * z, z, z));
      v = z * s;
      d = fmaf(v * (1.0f - s), 2.0f * kTanhScale * fmaf(3.0f * kTanhCubic * z, z, 1.0f), s);
      return;
    }
    case COLL_ACT_SILU: {
      const float s = logistic(z);
      v = z * s;
      d = fmaf(v, 1.0f - s, s);
      return;
    }
    case COLL_ACT_SIGMOID: {
      const float s = logistic(z);
      v = s;
      d = s * (1.0f - s);
      return;
    }
    default:
      v = z;
      d = 1.0f;
  }
}

__device__ __forceinline__ float ld_elem(const void *p, int64_t i, int type) {
  return type == COLL_F32 ? static_cast<const float *>(p)[i]
                          : h2f(static_cast<const uint16_t *>(p)[i], type);
}

__device__ __forceinline__ void st_elem(void *p, int64_t i, float v, int type) {
  if (type == COLL_F32) static_cast<float *>(p)[i] = v;
  else static_cast<uint16_t *>(p)[i] = f2h(v, type);
}

__device__ __forceinline__ void act_run8(float (&v)[8], int act) {
  switch (act) {
#define COLL_ACT_CASE(a)                                   \
  case a:                                                  \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] = act_value(v[i], a); \
    return;
    COLL_ACT_CASE(COLL_ACT_RELU)
    COLL_ACT_CASE(COLL_ACT_GELU)
    COLL_ACT_CASE(COLL_ACT_GELU_TANH)
    COLL_ACT_CASE(COLL_ACT_SILU)
    COLL_ACT_CASE(COLL_ACT_SIGMOID)
#undef COLL_ACT_CASE
    default: return;
  }
}

__device__ __forceinline__ void ld_run8(const void *p, int64_t i, int type, float (&v)[8]) {
  if (type == COLL_F32) {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
  const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  if (type == COLL_BF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) h2f2(w[q], COLL_BF16, v[2 * q], v[2 * q + 1]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) h2f2(w[q], COLL_F16, v[2 * q], v[2 * q + 1]);
  }
}

__device__ __forceinline__ void st_run8(void *p, int64_t i, int type, const float (&v)[8]) {
  if (type == COLL_F32) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t w[4];
  if (type == COLL_BF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = f2h2(v[2 * q], v[2 * q + 1], COLL_BF16);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = f2h2(v[2 * q], v[2 * q + 1], COLL_F16);
  }
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Columns [col, col + 8) of one row; `left` = columns of the row from col on (>= 1). g holds the
// product (gated: the gate's), u the up product.
template <bool GATED>
__device__ __forceinline__ void epilogue_run8(const DenseEpi &e, int batch, int64_t row,
                                              int64_t col, int64_t left, float (&g)[8],
                                              float (&u)[8]) {
  const int64_t o = row * e.out_rs[batch] + col;
  if (e.vec && left >= 8) {
    if (GATED) {
      if (e.gate) {
        st_run8(e.gate, row * e.gate_rs + col, e.type, g);
        st_run8(e.up, row * e.up_rs + col, e.type, u);
      }
      act_run8(g, e.act);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= u[i];
    } else {
      float t[8];
      if (e.bias) {
        ld_run8(e.bias, col, e.type, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += t[i];
      }
      if (e.pre) st_run8(e.pre, row * e.pre_rs + col, e.type, g);
      act_run8(g, e.act);
      if (e.res) {
        ld_run8(e.res, row * e.res_rs + col, e.out_type, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += t[i];
      }
    }
    st_run8(e.out[batch], o, e.out_type, g);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= left) break;
    const int64_t c = col + i;
    float v = g[i];
    if (GATED) {
      if (e.gate) {
        st_elem(e.gate, row * e.gate_rs + c, v, e.type);
        st_elem(e.up, row * e.up_rs + c, u[i], e.type);
      }
      v = act_value(v, e.act) * u[i];
    } else {
      if (e.bias) v += ld_elem(e.bias, c * e.bias_stride, e.type);
      if (e.pre) st_elem(e.pre, row * e.pre_rs + c, v, e.type);
      v = act_value(v, e.act);
      if (e.res) v += ld_elem(e.res, row * e.res_rs + c * e.res_cs, e.out_type);
    }
    st_elem(e.out[batch], o + i, v, e.out_type);
  }
}

}  // namespace coll
