// Elementwise steps of the dense backward calls.
//
//   one product:  dz = dy act'(z), and db = the column sums of dz
//   gated:        dg = dh u act'(g), du = dh act(g)
// Bound by HBM: each input is read once, dz (dg, du) written once, rounded to the operands' type
// for the tensor-core products that follow (their sums over rows or columns average the
// rounding, which is that of any stored activation). db sums the unrounded binary32 dz: a thread
// adds its rows in order, row groups of a CTA join in order in shared memory, and row blocks in
// order in a second launch, so the result does not depend on timing.
#include "dense.h"
#include "dense_epi.cuh"

namespace coll {
namespace {

constexpr int COLS = 256;   // columns per CTA: 32 runs of eight
constexpr int GROUPS = 8;   // row groups per CTA

__device__ __forceinline__ void load8(const DenseMat &m, int64_t row, int64_t col, int64_t left,
                                      int type, float (&v)[8]) {
  const uint16_t *p = static_cast<const uint16_t *>(m.p) + row * m.rs + col * m.cs;
  if (m.cs == 1 && left >= 8 && ((uintptr_t)p & 15u) == 0) {
    ld_run8(p, 0, type, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < left ? h2f(p[i * m.cs], type) : 0.0f;
}

__device__ __forceinline__ void store8(void *base, int64_t off, int64_t left, int type,
                                       const float (&v)[8]) {
  if (left >= 8) {  // ld is a multiple of eight and the base 16-byte aligned
    st_run8(base, off, type, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) static_cast<uint16_t *>(base)[off + i] = f2h(v[i], type);
}

template <bool GATED>
__global__ void __launch_bounds__(256) act_bwd_kernel(const DenseActBwd a, int64_t rows_per_block) {
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * COLS + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < a.m ? r0 + rows_per_block : a.m;
  const int64_t left = a.n - col;
  float sum[8] = {};
  if (left > 0) {
    for (int64_t r = r0 + grp; r < r1; r += GROUPS) {
      float dy[8], z[8], u[8], dz[8];
      load8(a.dy, r, col, left, a.type, dy);
      if (a.pre.p) load8(a.pre, r, col, left, a.type, z);
      if (GATED) load8(a.up, r, col, left, a.type, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (GATED) {
          float v, d;
          act_value_slope(z[i], a.act, v, d);
          dz[i] = dy[i] * u[i] * d;
          u[i] = dy[i] * v;
        } else {
          float v, d = 1.0f;
          if (a.pre.p) act_value_slope(z[i], a.act, v, d);
          dz[i] = dy[i] * d;
          sum[i] += dz[i];
        }
      }
      if (a.dz) store8(a.dz, r * a.ld + col, left, a.type, dz);
      if (GATED) store8(a.du, r * a.ld + col, left, a.type, u);
    }
  }
  __shared__ float part[GROUPS][COLS];
  if (!a.db) return;  // gated calls have none
#pragma unroll
  for (int i = 0; i < 8; ++i) part[grp][lane * 8 + i] = sum[i];
  __syncthreads();
  const int64_t c = (int64_t)blockIdx.x * COLS + threadIdx.x;
  if (c >= a.n) return;
  float s = part[0][threadIdx.x];
#pragma unroll
  for (int g = 1; g < GROUPS; ++g) s += part[g][threadIdx.x];
  if (gridDim.y == 1) st_elem(a.db, c, s, a.db_type);
  else a.part[(int64_t)blockIdx.y * a.n + c] = s;
}

__global__ void __launch_bounds__(256) join_kernel(const float *part, int64_t blocks, int64_t n,
                                                   void *db, int type) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.0f;
  for (int64_t b = 0; b < blocks; ++b) s += part[b * n + c];
  st_elem(db, c, s, type);
}

// A thread moves eight neighbouring elements: plain 2-byte loads (the rows start anywhere), one
// 16-byte store.
__global__ void __launch_bounds__(256) pack_kernel(const DenseMat src, int64_t rows, int64_t cols,
                                                   uint16_t *dst, int64_t ld) {
  const int64_t runs = ld / 8, total = rows * runs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / runs, c = (i - r * runs) * 8;
    const uint16_t *p = static_cast<const uint16_t *>(src.p) + r * src.rs + c * src.cs;
    uint32_t v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = c + q < cols ? p[q * src.cs] : 0u;
    *reinterpret_cast<uint4 *>(dst + r * ld + c) =
        make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

template <bool GATED>
__global__ void __launch_bounds__(256) empty_sum_kernel(const DenseJob j) {
  const int64_t runs = (j.n + 7) / 8, total = j.m * runs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / runs, c = (i - r * runs) * 8;
    float g[8] = {}, u[8] = {};
    epilogue_run8<GATED>(j.e, blockIdx.y, r, c, j.n - c, g, u);
  }
}

unsigned grid_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return (unsigned)(b < 4864 ? b : 4864);  // four CTAs of eight warps on each of 152 SMs, 8 deep
}

}  // namespace

cudaError_t dense_pack(const DenseMat &src, int64_t rows, int64_t cols, void *dst, int64_t ld,
                       cudaStream_t s) {
  pack_kernel<<<grid_for(rows * (ld / 8)), 256, 0, s>>>(src, rows, cols,
                                                        static_cast<uint16_t *>(dst), ld);
  return cudaGetLastError();
}

cudaError_t dense_empty_sum(const DenseJob &j, cudaStream_t s) {
  const dim3 grid(grid_for(j.m * ((j.n + 7) / 8)), (unsigned)j.nbatch);
  if (j.gated) empty_sum_kernel<true><<<grid, 256, 0, s>>>(j);
  else empty_sum_kernel<false><<<grid, 256, 0, s>>>(j);
  return cudaGetLastError();
}

// Row blocks: enough CTAs for two waves of eight a multiprocessor, 64 rows a block at least.
int64_t dense_act_bwd_row_blocks(int64_t m, int64_t n) {
  const int64_t cols = (n + COLS - 1) / COLS;
  int64_t want = (2432 + cols - 1) / cols;
  const int64_t most = (m + 63) / 64;
  if (want > most) want = most;
  if (want < 1) want = 1;
  if (want > 65535) want = 65535;
  const int64_t per = (m + want - 1) / want;
  return per ? (m + per - 1) / per : 1;
}

cudaError_t dense_act_bwd(const DenseActBwd &a, cudaStream_t s) {
  const int64_t blocks = dense_act_bwd_row_blocks(a.m, a.n);
  const int64_t per = (a.m + blocks - 1) / blocks;
  const dim3 grid((unsigned)((a.n + COLS - 1) / COLS), (unsigned)blocks);
  if (a.gated) act_bwd_kernel<true><<<grid, 256, 0, s>>>(a, per);
  else act_bwd_kernel<false><<<grid, 256, 0, s>>>(a, per);
  if (!a.gated && a.db && blocks > 1)
    join_kernel<<<(unsigned)((a.n + 255) / 256), 256, 0, s>>>(a.part, blocks, a.n, a.db,
                                                              a.db_type);
  return cudaGetLastError();
}

}  // namespace coll
