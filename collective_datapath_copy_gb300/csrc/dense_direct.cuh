// Loads from global memory straight into the fragments of mma.m16n8k16, from rows that start
// anywhere: the kernels for a few tokens.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "coll.h"

namespace coll {

// Plain loads that stay behind the wait for the predecessor; not the read-only path, whose data
// may not change while the kernel runs, and this one starts before its predecessor has finished.
__device__ __forceinline__ void ld_stream32(const void *p, uint32_t (&r)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}
__device__ __forceinline__ uint4 ld_word16(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_word8(const void *p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_word4(const void *p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_word2(const void *p) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}

// 16 elements from p (element k of its row of `len`), zeros past the row's end. ALIGN: bytes that
// every row start and hence p is a multiple of.
template <int ALIGN>
__device__ __forceinline__ void load16(const uint16_t *p, int k, int len, uint32_t (&r)[8]) {
  if (ALIGN == 32) {  // len is a multiple of 16
    if (k < len) {
      ld_stream32(p, r);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0u;
  } else if (ALIGN == 16) {  // len is a multiple of 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (k + 8 * h < len) v = ld_word16(p + 8 * h);
      r[4 * h] = v.x, r[4 * h + 1] = v.y, r[4 * h + 2] = v.z, r[4 * h + 3] = v.w;
    }
  } else if (ALIGN == 4) {  // len is even
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r[i] = k + 2 * i < len ? ld_word4(p + 2 * i) : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t lo = k + 2 * i < len ? ld_word2(p + 2 * i) : 0u;
      const uint32_t hi = k + 2 * i + 1 < len ? ld_word2(p + 2 * i + 1) : 0u;
      r[i] = lo | hi << 16;
    }
  }
}

// The same from anywhere, in two halves so that the loads of several calls are in flight together:
// the three aligned 16-byte words around the elements, if all their bytes are the row's, ...
struct Around {
  uint32_t w[12];
  bool whole;
};

__device__ __forceinline__ void ask16(const uint16_t *p, int k, int len, Around &a) {
  const int off = (int)((uintptr_t)p & 15u);
  a.whole = k >= off / 2 && k + (48 - off) / 2 <= len;
  const char *q = reinterpret_cast<const char *>(p) - off;
#pragma unroll
  for (int h = 0; h < 3; ++h) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (a.whole) v = ld_word16(q + 16 * h);
    a.w[4 * h] = v.x, a.w[4 * h + 1] = v.y, a.w[4 * h + 2] = v.z, a.w[4 * h + 3] = v.w;
  }
}

// ... then the elements out of them; single ones at the row's ends, zeros past them.
__device__ __forceinline__ void take16(const uint16_t *p, int k, int len, Around &a,
                                       uint32_t (&r)[8]) {
  const int off = (int)((uintptr_t)p & 15u);
  if (!a.whole && k < len) {
    load16<2>(p, k, len, r);
    return;
  }
  uint32_t *w = a.w;
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = w[i + 1];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
}

template <int TYPE>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (TYPE == COLL_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace coll
