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

// The hardware's approximations of 1 / x and 2^x, an instruction each: results too small for a
// normal number are zero, which takes the steps that would save them out of every element (gelu
// over 8192 x 8192 outputs: 75 us, with __fdividef and __expf 99).
__device__ __forceinline__ float recip(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRsqrt2 = 0.70710678118654752f;
constexpr float kRsqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float logistic(float z) {
  return recip(1.0f + exp2_fast(-kLog2e * z));
}

// (1 + tanh(a)) / 2 = logistic(2 a) for a = sqrt(2 / pi) (z + kTanhCubic z^3)
__device__ __forceinline__ float tanh_gate(float z) {
  const float c = fmaf(-2.0f * kTanhScale * kTanhCubic * kLog2e, z * z,
                       -2.0f * kTanhScale * kLog2e);
  return recip(1.0f + exp2_fast(z * c));
}

// Phi(z), the standard normal distribution function, and exp(-z^2 / 2), by the polynomial
// 7.1.26 of Abramowitz and Stegun for erfc(|z| / sqrt 2): a reciprocal, an exponential and eight
// multiply-adds. Its absolute error is below 1e-7, 2e-7 as evaluated here, which is what an output
// that adds up with others sees. Against Phi itself it grows for negative z: 3e-6 at -2, 5e-5 at
// -3, 5e-4 at -4, 1.6e-3 at -5, 1e-2 at -8. (The sum 1 + erf in binary32 is off by 4e-4 at -4, by
// a twentieth at -5, and zero from -5.6 on.)
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float t = recip(fmaf(0.3275911f * kRsqrt2, fabsf(z), 1.0f));
  e = exp2_fast(z * z * (-0.5f * kLog2e));
  float p = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  p = fmaf(p, t, 0.5f * 1.421413741f);
  p = fmaf(p, t, 0.5f * -0.284496736f);
  p = fmaf(p, t, 0.5f * 0.254829592f);
  const float half = p * t * e;
  return z < 0.0f ? half : 1.0f - half;
}

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case COLL_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case COLL_ACT_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case COLL_ACT_GELU_TANH: return z * tanh_gate(z);
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
      float e;
      const float c = normal_cdf(z, e);
      v = z * c;
      d = fmaf(z * kRsqrt2Pi, e, c);
      return;
    }
    case COLL_ACT_GELU_TANH: {
      const float s = tanh_gate(z);
      v = z * s;
      // far out s is 0 or 1 and the first factor 0: the square is kept from overflowing beside it
      const float zz = fminf(z * z, 4096.0f);
      d = fmaf(v * (1.0f - s), 2.0f * kTanhScale * fmaf(3.0f * kTanhCubic, zz, 1.0f), s);
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

template <int N>
__device__ __forceinline__ void act_run(float (&v)[N], int act) {
  switch (act) {
#define COLL_ACT_CASE(a)                                                     \
  case a:                                                                    \
    _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = act_value(v[i], a); \
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

// ---- 32-byte accesses (sm_100 and later): one whole sector a lane

__device__ __forceinline__ void ld_32b(const void *p, uint32_t *r) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}

__device__ __forceinline__ void st_32b(void *p, const uint32_t *r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void ld_16b(const void *p, uint32_t *r) {
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "l"(p)
               : "memory");
}

__device__ __forceinline__ void st_16b(void *p, const uint32_t *r) {
  asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// WORDS 32-bit words of a row from a 16-byte boundary on, whole sectors at a time where the row
// starts on one. Where every other row starts in the middle of a sector, stores write the first
// and last 16 bytes alone (8192 x 8200 written in 16-byte accesses: 69 us, so: 62); loads are 16
// bytes each, whose registers lie the same way in both forms, so that what was asked for ahead
// need not be moved, and waited for, before its use.
template <int WORDS>
__device__ __forceinline__ void ld_row(const void *p, uint32_t *r) {
  const char *q = static_cast<const char *>(p);
  if ((uintptr_t)p & 16u) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) ld_16b(q + 4 * i, r + i);
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 8) ld_32b(q + 4 * i, r + i);
  }
}

template <int WORDS>
__device__ __forceinline__ void st_row(void *p, const uint32_t *r) {
  char *q = static_cast<char *>(p);
  if ((uintptr_t)p & 16u) {
    st_16b(q, r);
#pragma unroll
    for (int i = 4; i < WORDS - 4; i += 8) st_32b(q + 4 * i, r + i);
    st_16b(q + 4 * (WORDS - 4), r + WORDS - 4);
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 8) st_32b(q + 4 * i, r + i);
  }
}

// v[0..32) += 32 neighbouring 16-bit elements held in r[16]
__device__ __forceinline__ void add_halves(float (&v)[32], const uint32_t *r, int type) {
  if (type == COLL_BF16) {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float lo, hi;
      h2f2(r[q], COLL_BF16, lo, hi);
      v[2 * q] += lo, v[2 * q + 1] += hi;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float lo, hi;
      h2f2(r[q], COLL_F16, lo, hi);
      v[2 * q] += lo, v[2 * q + 1] += hi;
    }
  }
}

__device__ __forceinline__ void ld_halves(const void *p, int64_t i, uint32_t *r) {
  ld_row<16>(static_cast<const uint16_t *>(p) + i, r);
}

// 32 neighbouring elements from element i on
__device__ __forceinline__ void st_run32(void *p, int64_t i, int type, const float (&v)[32]) {
  if (type == COLL_F32) {
    uint32_t r[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) r[q] = __float_as_uint(v[q]);
    st_row<32>(static_cast<float *>(p) + i, r);
    return;
  }
  uint32_t r[16];
  if (type == COLL_BF16) {
#pragma unroll
    for (int q = 0; q < 16; ++q) r[q] = f2h2(v[2 * q], v[2 * q + 1], COLL_BF16);
  } else {
#pragma unroll
    for (int q = 0; q < 16; ++q) r[q] = f2h2(v[2 * q], v[2 * q + 1], COLL_F16);
  }
  st_row<16>(static_cast<uint16_t *>(p) + i, r);
}

// ---- rows that start anywhere: 32 x 32 blocks through shared memory, so that neighbouring lanes
// access neighbouring columns. `st` is the warp's own 32 x kPitch words (an odd pitch: a lane's
// row and a row across the lanes are both free of bank conflicts); lane l holds row l of the
// block; `rows` and `cols` say how much of the block there is. Elements are accessed in pairs
// where rows start on 4 bytes.

constexpr int kPitch = 17;

__device__ __forceinline__ bool in_pairs(const void *p, int64_t rs) {
  return ((uintptr_t)p & 3u) == 0 && (rs & 1) == 0;
}

// block element (r, c) at p[r * rs + c]
__device__ __forceinline__ void staged_store(uint32_t *st, void *p, int64_t rs, int type, int rows,
                                             int cols, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  if (type == COLL_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) st[lane * kPitch + i] = __float_as_uint(v[16 * h + i]);
      __syncwarp();
      const int c = lane & 15;
      if (16 * h + c < cols)
#pragma unroll 4
        for (int r = lane >> 4; r < rows; r += 2)
          static_cast<uint32_t *>(p)[r * rs + 16 * h + c] = st[r * kPitch + c];
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 16; ++i)
    st[lane * kPitch + i] = type == COLL_BF16 ? f2h2(v[2 * i], v[2 * i + 1], COLL_BF16)
                                              : f2h2(v[2 * i], v[2 * i + 1], COLL_F16);
  __syncwarp();
  uint16_t *o = static_cast<uint16_t *>(p);
  if (in_pairs(p, rs)) {
    const int c = 2 * (lane & 15);
    if (rows == 32 && cols == 32) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = st[(2 * i + (lane >> 4)) * kPitch + (lane & 15)];
      o += (lane >> 4) * rs + c;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        *reinterpret_cast<uint32_t *>(o) = w[i];
        o += 2 * rs;
      }
      return;
    }
#pragma unroll 4
    for (int r = lane >> 4; r < rows; r += 2) {
      const uint32_t w = st[r * kPitch + (lane & 15)];
      if (c + 1 < cols) *reinterpret_cast<uint32_t *>(o + r * rs + c) = w;
      else if (c < cols) o[r * rs + c] = (uint16_t)w;
    }
  } else if (rows == 32 && cols == 32) {
    o += lane;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      *o = reinterpret_cast<const uint16_t *>(st + r * kPitch)[lane];
      o += rs;
    }
  } else if (lane < cols) {
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      o[r * rs + lane] = reinterpret_cast<const uint16_t *>(st + r * kPitch)[lane];
  }
}

// v += the block with element (r, c) at p[r * rs + c * cs]
__device__ __forceinline__ void staged_add(uint32_t *st, const void *p, int64_t rs, int64_t cs,
                                           int type, int rows, int cols, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  if (type == COLL_F32) {
    const float *q = static_cast<const float *>(p);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = lane & 15, r0 = lane >> 4;
      const float *o = q + r0 * rs + (16 * h + c) * cs;
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i, o += 2 * rs)
        w[i] = r0 + 2 * i < rows && 16 * h + c < cols ? *o : 0.0f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) st[(r0 + 2 * i) * kPitch + c] = __float_as_uint(w[i]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[16 * h + i] += __uint_as_float(st[lane * kPitch + i]);
    }
    return;
  }
  // all loads in flight before the first is used
  const uint16_t *q = static_cast<const uint16_t *>(p);
  if (cs == 1 && in_pairs(p, rs) && cols == 32) {
    uint32_t w[16];
    const int r0 = lane >> 4;
    const uint16_t *o = q + r0 * rs + 2 * (lane & 15);
#pragma unroll
    for (int i = 0; i < 16; ++i, o += 2 * rs)
      w[i] = r0 + 2 * i < rows ? *reinterpret_cast<const uint32_t *>(o) : 0u;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) st[(r0 + 2 * i) * kPitch + (lane & 15)] = w[i];
  } else {
    uint16_t w[32];
    const uint16_t *o = q + lane * cs;
#pragma unroll
    for (int r = 0; r < 32; ++r, o += rs) w[r] = r < rows && lane < cols ? *o : (uint16_t)0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; ++r) reinterpret_cast<uint16_t *>(st + r * kPitch)[lane] = w[r];
  }
  __syncwarp();
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = st[lane * kPitch + i];
  add_halves(v, w, type);
}

// v[i] += b of lane i, through the warp's block
__device__ __forceinline__ void add_lanes(uint32_t *st, float b, float (&v)[32]) {
  __syncwarp();
  st[threadIdx.x & 31] = __float_as_uint(b);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 w = *reinterpret_cast<const float4 *>(st + i);
    v[i] += w.x, v[i + 1] += w.y, v[i + 2] += w.z, v[i + 3] += w.w;
  }
}

// What the epilogue of one element adds, as it lies in memory: asked for before the sums it is
// added to are there (one token, 4096 x 1792 with bias and residual: 4.6 us, asked for after: 5.4).
struct Addends {
  uint32_t bias, res;
};

template <bool GATED>
__device__ __forceinline__ Addends ask_addends(const DenseEpi &e, int64_t row, int64_t col) {
  Addends a = {0u, 0u};
  if (GATED) return a;
  if (e.bias) a.bias = static_cast<const uint16_t *>(e.bias)[col * e.bias_stride];
  if (e.res) {
    const int64_t at = row * e.res_rs + col * e.res_cs;
    if (e.out_type == COLL_F32) a.res = static_cast<const uint32_t *>(e.res)[at];
    else a.res = static_cast<const uint16_t *>(e.res)[at];
  }
  return a;
}

// One element: g holds the product (gated: the gate's), u the up product.
template <bool GATED>
__device__ __forceinline__ void epilogue_one(const DenseEpi &e, int batch, int64_t row, int64_t col,
                                             float g, float u, Addends a) {
  if (GATED) {
    if (e.gate) {
      st_elem(e.gate, row * e.gate_rs + col, g, e.type);
      st_elem(e.up, row * e.up_rs + col, u, e.type);
    }
    g = act_value(g, e.act) * u;
  } else {
    if (e.bias) g += h2f((uint16_t)a.bias, e.type);
    if (e.pre) st_elem(e.pre, row * e.pre_rs + col, g, e.type);
    g = act_value(g, e.act);
    if (e.res)
      g += e.out_type == COLL_F32 ? __uint_as_float(a.res) : h2f((uint16_t)a.res, e.out_type);
  }
  st_elem(e.out[batch], row * e.out_rs[batch] + col, g, e.out_type);
}

__device__ __forceinline__ void join_column(const DenseJoin &j, int64_t c) {
  float s = 0.0f;
  int64_t b = 0;
  for (; b + 8 <= j.blocks; b += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = j.part[(b + i) * j.n + c];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  for (; b < j.blocks; ++b) s += j.part[b * j.n + c];
  st_elem(j.db, c, s, j.type);
}

__device__ __forceinline__ float bias_at(const DenseEpi &e, int64_t col) {
  return e.bias ? ld_elem(e.bias, col * e.bias_stride, e.type) : 0.0f;
}

}  // namespace coll
