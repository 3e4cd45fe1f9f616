// The products of the dense operators in their simplest form: a 64 x 64 tile per CTA, operands
// widened to binary32 in shared memory, one fused multiply-add per term in order of k. Takes any
// strides and sizes. Bound by the binary32 pipes.
#include "dense.h"
#include "dense_epi.cuh"

namespace coll {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;

template <bool GATED>
__global__ void __launch_bounds__(256) simple_kernel(const DenseJob j) {
  __shared__ float sa[TK][TM + 1], sb[GATED ? 2 : 1][TK][TN + 1];
  const int batch = blockIdx.z, t = threadIdx.x;
  const int64_t m0 = (int64_t)blockIdx.y * TM, n0 = (int64_t)blockIdx.x * TN;
  const int r = t / 8 * 2, c = t % 8 * 8;  // two rows, eight columns
  float acc[2][8] = {}, acc2[2][8] = {};
  for (int seg = 0; seg < j.nseg; ++seg) {
    const DenseMat &a = j.a[j.nbatch == 2 ? batch : seg];
    for (int64_t k0 = 0; k0 < j.k; k0 += TK) {
      for (int i = t; i < TM * TK; i += 256) {
        // neighbouring threads along the contiguous axis
        const int mm = a.cs == 1 ? i / TK : i % TM, kk = a.cs == 1 ? i % TK : i / TM;
        const int64_t m = m0 + mm, k = k0 + kk;
        sa[kk][mm] =
            m < j.m && k < j.k
                ? h2f(static_cast<const uint16_t *>(a.p)[m * a.rs + k * a.cs], j.e.type)
                : 0.0f;
      }
#pragma unroll
      for (int w = 0; w < (GATED ? 2 : 1); ++w) {
        const DenseMat &b = j.b[GATED ? w : seg];
        for (int i = t; i < TN * TK; i += 256) {
          const int nn = b.cs == 1 ? i / TK : i % TN, kk = b.cs == 1 ? i % TK : i / TN;
          const int64_t n = n0 + nn, k = k0 + kk;
          sb[w][kk][nn] =
              n < j.n && k < j.k
                  ? h2f(static_cast<const uint16_t *>(b.p)[n * b.rs + k * b.cs], j.e.type)
                  : 0.0f;
        }
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < TK; ++kk)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            acc[x][y] = fmaf(sa[kk][r + x], sb[0][kk][c + y], acc[x][y]);
            if (GATED) acc2[x][y] = fmaf(sa[kk][r + x], sb[GATED ? 1 : 0][kk][c + y], acc2[x][y]);
          }
      __syncthreads();
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (m0 + r + x < j.m && n0 + c < j.n)
      epilogue_run8<GATED>(j.e, batch, m0 + r + x, n0 + c, j.n - n0 - c, acc[x], acc2[x]);
}

}  // namespace

cudaError_t dense_simple(const DenseJob &j, cudaStream_t s) {
  const dim3 grid((unsigned)((j.n + TN - 1) / TN), (unsigned)((j.m + TM - 1) / TM),
                  (unsigned)j.nbatch);
  if (grid.y > 65535u) return cudaErrorInvalidConfiguration;
  if (j.gated) simple_kernel<true><<<grid, 256, 0, s>>>(j);
  else simple_kernel<false><<<grid, 256, 0, s>>>(j);
  return cudaGetLastError();
}

}  // namespace coll
