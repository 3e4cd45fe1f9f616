// The products of the dense operators for one to a few tokens.
//
// Bound by HBM (the weights, read once) and by latency, so there is no staging, no barrier in the
// loop and one launch: every warp loads weights straight into the fragments of mma.m16n8k16, 16
// weight rows by 64 of k a step (gated: eight rows of each matrix, so a lane ends up with g and u
// of the same output), the tokens are the eight columns. The order of k inside a step is the same
// for both operands and otherwise free, so a lane takes 16 neighbouring elements of its row, 32
// bytes, and four lanes a whole 128-byte line. The warps of a CTA take the steps of its rows in
// turn and join once, in order, through shared memory. Several steps of loads per lane are in
// flight before the first is used.
//
// Measured for one token, weights from HBM: 4096 x 1792 4.6 us, gated 14336 x 4096 37 us (6.3
// TB/s).
//
// tcgen05 is the wrong tool here: an instruction of 128 rows by 16 tokens takes about 27 ns to
// issue whatever the batch, 7 us for k = 4096, and sharing k between CTAs costs a cluster
// launch and two cluster barriers, 2 to 3 us.
#include <type_traits>

#include "dense.h"
#include "dense_epi.cuh"
#include "dense_tc.h"
#include "tma.cuh"

namespace coll {
namespace {

constexpr int kStep = 64;      // elements of k a warp takes at a time
// warps of a CTA: shared memory for their sums is 32 KiB at most
template <int NT>
constexpr int kMostWarps = NT == 8 ? 8 : 16;

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
  a.whole = 2 * k >= off && k + (48 - off) / 2 <= len;
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

// NT: columns of eight tokens.
template <bool GATED, int TYPE, int NT, int ALIGN>
__global__ void __launch_bounds__(kMostWarps<NT> * 32, 1)
    gemv_kernel(const __grid_constant__ GemvParams p) {
  griddep_launch();
  constexpr int FEAT = GATED ? 8 : 16;   // outputs of a CTA
  constexpr int AHEAD = NT == 1 && ALIGN > 2 ? 4 : NT <= 2 ? 2 : 1;
  __shared__ float part[kMostWarps<NT>][8 * NT][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int64_t f0 = (int64_t)blockIdx.x * FEAT;
  const int len = (int)p.k;
  const int64_t fa = f0 + g, fb = GATED ? fa : fa + 8;
  const int la = fa < p.n ? len : 0, lb = fb < p.n ? len : 0;  // rows that are not there are empty
  const uint16_t *wa = static_cast<const uint16_t *>(p.w[0]) + (la ? fa : 0) * p.ld[0] + 16 * t;
  const uint16_t *wb =
      static_cast<const uint16_t *>(p.w[GATED ? 1 : 0]) + (lb ? fb : 0) * p.ld[GATED ? 1 : 0] +
      16 * t;
  const uint16_t *xt[NT];
  int lx[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int tok = c * 8 + g;
    lx[c] = tok < (int)p.m ? len : 0;
    xt[c] = static_cast<const uint16_t *>(p.x) + (lx[c] ? tok : 0) * p.x_ld + 16 * t;
  }
  float acc[NT][4] = {};
  griddep_wait();
  // the first of the outputs that this thread finishes
  Addends ahead = {0u, 0u};
  if ((int)threadIdx.x < FEAT * (int)p.m && f0 + threadIdx.x % FEAT < p.n)
    ahead = ask_addends<GATED>(p.e, threadIdx.x / FEAT, f0 + threadIdx.x % FEAT);
  const int steps = (len + kStep - 1) / kStep;
  for (int s = warp; s < steps; s += AHEAD * warps) {
    uint32_t a[AHEAD][8], b[AHEAD][8], x[AHEAD][NT][8];
    if constexpr (ALIGN == 2) {
      Around ra[AHEAD], rb[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = (s + i * warps) * kStep;
        ask16(wa + k, k + 16 * t, la, ra[i]);
        ask16(wb + k, k + 16 * t, lb, rb[i]);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = (s + i * warps) * kStep;
        take16(wa + k, k + 16 * t, la, ra[i], a[i]);
        take16(wb + k, k + 16 * t, lb, rb[i], b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = (s + i * warps) * kStep;
        load16<ALIGN>(wa + k, k + 16 * t, la, a[i]);
        load16<ALIGN>(wb + k, k + 16 * t, lb, b[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int k = (s + i * warps) * kStep;
      if constexpr (ALIGN == 2) {
        Around rx[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) ask16(xt[c] + k, k + 16 * t, lx[c], rx[c]);
#pragma unroll
        for (int c = 0; c < NT; ++c) take16(xt[c] + k, k + 16 * t, lx[c], rx[c], x[i][c]);
      } else {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (p.x_align >= ALIGN) load16<ALIGN>(xt[c] + k, k + 16 * t, lx[c], x[i][c]);
          else load16<2>(xt[c] + k, k + 16 * t, lx[c], x[i][c]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma16816<TYPE>(acc[c], a[i][2 * q], b[i][2 * q], a[i][2 * q + 1], b[i][2 * q + 1],
                         x[i][c][2 * q], x[i][c][2 * q + 1]);
  }
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    part[warp][c * 8 + 2 * t][g] = acc[c][0];
    part[warp][c * 8 + 2 * t + 1][g] = acc[c][1];
    part[warp][c * 8 + 2 * t][g + 8] = acc[c][2];
    part[warp][c * 8 + 2 * t + 1][g + 8] = acc[c][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < FEAT * (int)p.m; i += blockDim.x) {
    const int tok = i / FEAT, f = i % FEAT;
    if (f0 + f >= p.n) continue;
    float v = part[0][tok][f], u = GATED ? part[0][tok][(f + 8) & 15] : 0.0f;
    for (int w = 1; w < warps; ++w) {
      v += part[w][tok][f];
      if (GATED) u += part[w][tok][(f + 8) & 15];
    }
    if (i != (int)threadIdx.x) ahead = ask_addends<GATED>(p.e, tok, f0 + f);
    epilogue_one<GATED>(p.e, 0, tok, f0 + f, v, u, ahead);
  }
}

template <bool GATED, int TYPE, int NT>
cudaError_t launch(const GemvParams &p, int align, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.n + (GATED ? 8 : 16) - 1) / (GATED ? 8 : 16));
  const unsigned threads = 32u * (p.warps < kMostWarps<NT> ? p.warps : kMostWarps<NT>);
  auto kernel = align == 32   ? gemv_kernel<GATED, TYPE, NT, 32>
                : align == 16 ? gemv_kernel<GATED, TYPE, NT, 16>
                : align == 4  ? gemv_kernel<GATED, TYPE, NT, 4>
                              : gemv_kernel<GATED, TYPE, NT, 2>;
  return dense_launch(kernel, dim3(grid), threads, 0, 1, s, p);
}

template <bool GATED, int TYPE>
cudaError_t launch(const GemvParams &p, int align, cudaStream_t s) {
  return p.m <= 8    ? launch<GATED, TYPE, 1>(p, align, s)
         : p.m <= 16 ? launch<GATED, TYPE, 2>(p, align, s)
         : p.m <= 32 ? launch<GATED, TYPE, 4>(p, align, s)
                     : launch<GATED, TYPE, 8>(p, align, s);
}

// ---- weights that lie the other way: stored as k rows of n
//
// The tokens are the 16 rows, the outputs the columns. A lane reads four neighbouring outputs of
// four neighbouring rows of k and pairs the rows up with byte permutes; which output is which
// column of which fragment is free, so those four serve four fragments, and the eight lanes of a
// row of k read 64 neighbouring bytes. Rows of k in turn go to the warps, which join as above.

constexpr int kFeat = 32;  // outputs of a CTA

// Four elements from p, `left` of them there. ALIGN 8: all or none are, on 8 bytes.
template <int ALIGN>
__device__ __forceinline__ uint2 load4(const uint16_t *p, int left) {
  if (ALIGN == 8) {
    uint2 v = make_uint2(0u, 0u);
    if (left > 0) v = ld_word8(p);
    return v;
  }
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < left ? ld_word2(p + i) : 0u;
  return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
}

template <bool GATED, int TYPE, int ALIGN>
__global__ void __launch_bounds__(GATED ? 256 : 512, 1) gemv_t_kernel(
    const __grid_constant__ GemvTParams p) {
  griddep_launch();
  constexpr int W = GATED ? 2 : 1, WARPS = GATED ? 8 : 16, AHEAD = GATED ? 2 : 4;
  __shared__ float part[WARPS][W][16][kFeat + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3, m = (int)p.m, len = (int)p.k;
  const int64_t f0 = (int64_t)blockIdx.x * kFeat, fl = f0 + 4 * g;
  const int left = (int)(p.n - fl < 4 ? p.n - fl : 4);  // outputs of this lane, may be negative
  float acc[W][4][4] = {};
  griddep_wait();
  Addends ahead = {0u, 0u};  // the first of the outputs that this thread finishes
  if ((int)threadIdx.x < kFeat * m && f0 + threadIdx.x % kFeat < p.n)
    ahead = ask_addends<GATED>(p.e, threadIdx.x / kFeat, f0 + threadIdx.x % kFeat);
  const int steps = (len + 15) / 16;
  for (int s0 = warp; s0 < steps; s0 += AHEAD * warps) {
    uint2 w[AHEAD][W][4], x[AHEAD][2];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int k = (s0 + i * warps) * 16 + 4 * t;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const uint16_t *row = static_cast<const uint16_t *>(p.w[q]) + (int64_t)k * p.ld[q] + fl;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          w[i][q][r] = k + r < len && left > 0 ? load4<ALIGN>(row + r * p.ld[q], left)
                                               : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = g + 8 * h;
        const uint16_t *row = static_cast<const uint16_t *>(p.x) + tok * p.x_ld + k;
        x[i][h] = make_uint2(0u, 0u);
        if (tok < m && k < len) {
          if (p.x_align == 8) x[i][h] = ld_word8(row);
          else x[i][h] = load4<2>(row, len - k < 4 ? len - k : 4);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int q = 0; q < W; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // output j of the lane's four: rows k, k + 1 and k + 2, k + 3
          const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
          const uint2 *r = w[i][q];
          const uint32_t b0 = j < 2 ? __byte_perm(r[0].x, r[1].x, sel)
                                    : __byte_perm(r[0].y, r[1].y, sel);
          const uint32_t b1 = j < 2 ? __byte_perm(r[2].x, r[3].x, sel)
                                    : __byte_perm(r[2].y, r[3].y, sel);
          mma16816<TYPE>(acc[q][j], x[i][0].x, x[i][1].x, x[i][0].y, x[i][1].y, b0, b1);
        }
  }
#pragma unroll
  for (int q = 0; q < W; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // column c of fragment j is output 4 c + j
      part[warp][q][g][8 * t + j] = acc[q][j][0];
      part[warp][q][g][8 * t + 4 + j] = acc[q][j][1];
      part[warp][q][g + 8][8 * t + j] = acc[q][j][2];
      part[warp][q][g + 8][8 * t + 4 + j] = acc[q][j][3];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kFeat * m; i += blockDim.x) {
    const int tok = i / kFeat, f = i % kFeat;
    if (f0 + f >= p.n) continue;
    float v = part[0][0][tok][f], u = GATED ? part[0][W - 1][tok][f] : 0.0f;
    for (int c = 1; c < warps; ++c) {
      v += part[c][0][tok][f];
      if (GATED) u += part[c][W - 1][tok][f];
    }
    if (i != (int)threadIdx.x) ahead = ask_addends<GATED>(p.e, tok, f0 + f);
    epilogue_one<GATED>(p.e, 0, tok, f0 + f, v, u, ahead);
  }
}

// The widest access that every row of the matrix starts on.
int row_align(const void *p, int64_t rows, int64_t ld, int64_t k) {
  const uint64_t bits = (uintptr_t)p | (rows > 1 ? (uint64_t)ld * 2 : 0) | (uint64_t)k * 2;
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

}  // namespace

cudaError_t gemv_run(const DenseJob &j, cudaStream_t s) {
  GemvParams p = {};
  p.e = j.e;
  p.m = j.m;
  p.n = j.n;
  p.k = j.k;
  p.x = j.a[0].p;
  p.x_ld = j.a[0].rs;
  p.x_align = row_align(p.x, j.m, p.x_ld, j.k);
  int align = 32;
  for (int i = 0; i < (j.gated ? 2 : 1); ++i) {
    p.w[i] = j.b[i].p;
    p.ld[i] = j.b[i].rs;
    const int a = row_align(p.w[i], j.n, p.ld[i], j.k);
    if (a < align) align = a;
  }
  // Warps of a CTA: 16, one CTA an SM, where there are no more CTAs than SMs, else 8 and two CTAs
  // an SM (128 registers a thread); no more than there are steps of k.
  const int64_t ctas = (j.n + (j.gated ? 7 : 15)) / (j.gated ? 8 : 16);
  const int64_t steps = (j.k + kStep - 1) / kStep;
  p.warps = ctas <= (int64_t)kSms ? 16 : 8;
  while (p.warps > 1 && p.warps > steps) p.warps /= 2;
  if (j.e.type == COLL_BF16)
    return j.gated ? launch<true, COLL_BF16>(p, align, s) : launch<false, COLL_BF16>(p, align, s);
  return j.gated ? launch<true, COLL_F16>(p, align, s) : launch<false, COLL_F16>(p, align, s);
}

cudaError_t gemv_t_run(const DenseJob &j, cudaStream_t s) {
  GemvTParams p = {};
  p.e = j.e;
  p.m = j.m;
  p.n = j.n;
  p.k = j.k;
  p.x = j.a[0].p;
  p.x_ld = j.a[0].rs;
  // bits of what the four-element accesses start on
  const uint64_t xb =
      (uint64_t)j.k * 2 | (uintptr_t)p.x | (j.m > 1 ? (uint64_t)p.x_ld * 2 : 0);
  uint64_t wb = (uint64_t)j.n * 2;
  for (int i = 0; i < (j.gated ? 2 : 1); ++i) {
    p.w[i] = j.b[i].p;
    p.ld[i] = j.b[i].cs;
    wb |= (uintptr_t)p.w[i] | (j.k > 1 ? (uint64_t)p.ld[i] * 2 : 0);
  }
  p.x_align = xb % 8 ? 2 : 8;
  const int64_t steps = (j.k + 15) / 16;
  // all the warps the sums have room for, no more than there are steps
  unsigned warps = j.gated ? 8 : 16;
  while (warps > 1 && warps > steps) warps /= 2;
  const dim3 grid((unsigned)((j.n + kFeat - 1) / kFeat));
  const bool bf = j.e.type == COLL_BF16, wide = wb % 8 == 0;
  auto kernel =
      j.gated ? (bf ? (wide ? gemv_t_kernel<true, COLL_BF16, 8> : gemv_t_kernel<true, COLL_BF16, 2>)
                    : (wide ? gemv_t_kernel<true, COLL_F16, 8> : gemv_t_kernel<true, COLL_F16, 2>))
              : (bf ? (wide ? gemv_t_kernel<false, COLL_BF16, 8>
                            : gemv_t_kernel<false, COLL_BF16, 2>)
                    : (wide ? gemv_t_kernel<false, COLL_F16, 8>
                            : gemv_t_kernel<false, COLL_F16, 2>));
  return dense_launch(kernel, grid, 32 * warps, 0, 1, s, p);
}

}  // namespace coll
