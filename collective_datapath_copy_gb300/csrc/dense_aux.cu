// Elementwise steps of the dense backward calls.
//
//   one product:  dz = dy act'(z), and db = the column sums of dz
//   gated:        dg = dh u act'(g), du = dh act(g)
// Bound by HBM (gated, 4096 x 14336: 92 us for 587 MB, 6.4 TB/s): each input is read once, dz (dg,
// du) written once, rounded to the operands' type for the tensor-core products that follow (their
// sums over rows or columns average the rounding, which is that of any stored activation; the
// gradients' error against 64 bits is 1.4 times that of rounding them alone, 0.0023 for 0.0017 in
// bf16). In f16 that also bounds dz: past 65504 it is infinite, and with it the rows of dx and dW
// that it enters, where a binary32 dz would have stayed finite; below 2^-25 it is zero. A caller
// scales its loss for that, as for its stored activations. db sums the unrounded binary32 dz: a
// thread adds its rows in order, row groups of a CTA join in order in shared memory, and row blocks
// in order in a second launch, so the result does not depend on timing.
#include "dense.h"
#include "dense_epi.cuh"
#include "tma.cuh"

namespace coll {
namespace {

constexpr int COLS = 256;   // columns per CTA: 32 lanes of eight
constexpr int GROUPS = 8;   // row groups per CTA, a warp each

// Eight columns of one row, zeros past its end. ALIGN 16: rows of whole 16-byte runs; 4: rows of
// whole pairs; 0: any strides.
template <int ALIGN>
__device__ __forceinline__ uint4 load8(const DenseMat &m, int64_t row, int64_t col, int64_t left) {
  const uint16_t *p = static_cast<const uint16_t *>(m.p) + row * m.rs + col * m.cs;
  if constexpr (ALIGN == 16) {
    return __ldcs(reinterpret_cast<const uint4 *>(p));
  } else if constexpr (ALIGN == 4) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
    return make_uint4(q[0], left > 2 ? q[1] : 0u, left > 4 ? q[2] : 0u, left > 6 ? q[3] : 0u);
  } else {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i * m.cs] : 0u;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

__device__ __forceinline__ void widen8(const uint4 &a, int type, float (&v)[8]) {
  h2f2(a.x, type, v[0], v[1]);
  h2f2(a.y, type, v[2], v[3]);
  h2f2(a.z, type, v[4], v[5]);
  h2f2(a.w, type, v[6], v[7]);
}

// The scratch rows are padded to a multiple of eight columns, so a run is stored whole.
__device__ __forceinline__ void store8(void *base, int64_t off, int type, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off) =
      make_uint4(f2h2(v[0], v[1], type), f2h2(v[2], v[3], type), f2h2(v[4], v[5], type),
                 f2h2(v[6], v[7], type));
}

// Eight elements that start at p, on any 2-byte boundary, out of the two aligned 16-byte words
// that hold them.
__device__ __forceinline__ uint4 shifted8(const uint16_t *p, const uint4 &a, const uint4 &b) {
  const uint32_t off = (uint32_t)((uintptr_t)p & 15u), word = off >> 2, bits = (off & 2u) * 8u;
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (word & 2) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (word & 1) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// One of `ctas` CTAs that lay out operand o. A thread takes kRuns runs of eight elements, counted
// through the rows, all in flight together. Inside a row that is contiguous the loads are 16-byte
// words (all of whose bytes are the row's); elsewhere single elements. 8183 x 10167: 48 us for
// 333 MB, 7.0 TB/s (two runs in flight 54, a warp for each row 68).
constexpr int kRuns = 4;

__device__ __forceinline__ void pack_rows(const DensePack &a, int o, int64_t cta, int64_t ctas) {
  const DenseMat src = a.src[o];
  const uint32_t runs = (uint32_t)(a.ld[o] / 8), cols = (uint32_t)a.cols[o];
  const int64_t total = a.rows[o] * runs;
  for (int64_t at = cta * (256 * kRuns); at < total; at += ctas * (256 * kRuns)) {
    const int64_t row0 = at / runs;
    const uint32_t q0 = (uint32_t)(at - row0 * runs);
    uint4 w[kRuns][2];
    const uint16_t *p[kRuns];
    uint32_t c[kRuns];
    bool whole[kRuns], there[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const uint32_t l = q0 + i * 256 + threadIdx.x, r = l / runs;
      c[i] = (l - r * runs) * 8;
      there[i] = at + i * 256 + threadIdx.x < total;
      p[i] = static_cast<const uint16_t *>(src.p) + (row0 + r) * src.rs + c[i] * src.cs;
      whole[i] = there[i] && src.cs == 1 && c[i] >= 8 && c[i] + 16 <= cols;
      if (whole[i]) {
        const uint4 *q = reinterpret_cast<const uint4 *>((uintptr_t)p[i] & ~(uintptr_t)15u);
        w[i][0] = q[0];
        w[i][1] = q[1];
      }
    }
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      if (!there[i]) continue;
      uint4 out;
      if (whole[i]) {
        out = shifted8(p[i], w[i][0], w[i][1]);
      } else {
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = c[i] + k < cols ? p[i][k * src.cs] : 0u;
        out = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                         v[6] | v[7] << 16);
      }
      // rows of the copy follow one another
      reinterpret_cast<uint4 *>(a.dst[o])[at + i * 256 + threadIdx.x] = out;
    }
  }
}

__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ DensePack a) {
  griddep_launch();
  griddep_wait();
  pack_rows(a, blockIdx.y, blockIdx.x, gridDim.x);
}

// Two rows a turn keep six 16-byte loads of a lane in flight (one row where loads are single
// elements, which are many already). CTAs past the row blocks lay out the products' operands: a
// launch of its own for that costs 2 to 4 us (777 x 1530 x 1016: 21 us, so: 17).
template <bool GATED, int ACT, int TYPE, int ALIGN>
__global__ void __launch_bounds__(256, ALIGN == 16 ? 4 : 2)
    act_bwd_kernel(const DenseActBwd a, int64_t rows_per_block, unsigned row_blocks,
                   const __grid_constant__ DensePack pack) {
  griddep_launch();
  griddep_wait();
  if (blockIdx.y >= row_blocks) {
    const unsigned i = (blockIdx.y - row_blocks) * gridDim.x + blockIdx.x, o = i / pack.ctas;
    if (o < (unsigned)pack.count) pack_rows(pack, (int)o, i - o * pack.ctas, pack.ctas);
    return;
  }
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * COLS + lane * 8;
  const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < a.m ? r0 + rows_per_block : a.m;
  const int64_t left = a.n - col;
  float sum[8] = {};
  auto one = [&](int64_t r, const uint4 &wy, const uint4 &wz, const uint4 &wu) {
    float dy[8], z[8], u[8];
    widen8(wy, TYPE, dy);
    if (ACT != COLL_ACT_NONE) widen8(wz, TYPE, z);
    if (GATED) widen8(wu, TYPE, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v, d = 1.0f;
      if (ACT != COLL_ACT_NONE) act_value_slope(z[i], ACT, v, d);
      if (GATED) {
        z[i] = dy[i] * v;
        dy[i] = dy[i] * u[i] * d;
      } else {
        if (ACT != COLL_ACT_NONE) dy[i] *= d;
        sum[i] += dy[i];
      }
    }
    if (a.dz) store8(a.dz, r * a.ld + col, TYPE, dy);
    if (GATED) store8(a.du, r * a.ld + col, TYPE, z);
  };
  if (left > 0) {
    constexpr int AHEAD = ALIGN ? 2 : 1;
    uint4 y[AHEAD], z[AHEAD] = {}, u[AHEAD] = {};
    auto fetch = [&](int i, int64_t r) {
      y[i] = load8<ALIGN>(a.dy, r, col, left);
      if (ACT != COLL_ACT_NONE) z[i] = load8<ALIGN>(a.pre, r, col, left);
      if (GATED) u[i] = load8<ALIGN>(a.up, r, col, left);
    };
    for (int64_t r = r0 + grp; r < r1; r += AHEAD * GROUPS) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (r + i * GROUPS < r1) fetch(i, r + i * GROUPS);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (r + i * GROUPS < r1) one(r + i * GROUPS, y[i], z[i], u[i]);
    }
  }
  if constexpr (!GATED) {
    if (!a.db) return;
    __shared__ float part[GROUPS][COLS];
#pragma unroll
    for (int i = 0; i < 8; ++i) part[grp][lane * 8 + i] = sum[i];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * COLS + threadIdx.x;
    if (c >= a.n) return;
    float s = part[0][threadIdx.x];
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) s += part[g][threadIdx.x];
    if (row_blocks == 1) st_elem(a.db, c, s, a.db_type);
    else a.part[(int64_t)blockIdx.y * a.n + c] = s;
  }
}

// Bits of the rows' addresses; all set where columns are apart.
uint64_t row_bits(const DenseMat &m) {
  return !m.p ? 0 : m.cs != 1 ? ~(uint64_t)0 : (uintptr_t)m.p | (uint64_t)(m.rs * 2);
}

template <bool GATED, int ACT>
cudaError_t launch_act_bwd(const DenseActBwd &a, const DensePack &pack, dim3 grid, int64_t per,
                           cudaStream_t s) {
  const uint64_t bits =
      (uint64_t)a.n * 2 | row_bits(a.dy) | row_bits(a.pre) | row_bits(a.up);
  const int align = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 0;
  auto kernel = a.type == COLL_BF16
                    ? (align == 16  ? act_bwd_kernel<GATED, ACT, COLL_BF16, 16>
                       : align == 4 ? act_bwd_kernel<GATED, ACT, COLL_BF16, 4>
                                    : act_bwd_kernel<GATED, ACT, COLL_BF16, 0>)
                    : (align == 16  ? act_bwd_kernel<GATED, ACT, COLL_F16, 16>
                       : align == 4 ? act_bwd_kernel<GATED, ACT, COLL_F16, 4>
                                    : act_bwd_kernel<GATED, ACT, COLL_F16, 0>);
  const unsigned row_blocks = grid.y;
  if (pack.count) grid.y += (pack.ctas * (unsigned)pack.count + grid.x - 1) / grid.x;
  return dense_launch(kernel, grid, 256, 0, 1, s, a, per, row_blocks, pack);
}

__global__ void __launch_bounds__(256) join_kernel(const DenseJoin j) {
  griddep_launch();
  griddep_wait();
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c < j.n) join_column(j, c);
}

template <bool GATED>
__global__ void __launch_bounds__(256) empty_sum_kernel(const DenseJob j) {
  griddep_launch();
  griddep_wait();
  const int64_t total = j.m * j.n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / j.n, c = i - r * j.n;
    epilogue_one<GATED>(j.e, blockIdx.y, r, c, 0.0f, 0.0f, ask_addends<GATED>(j.e, r, c));
  }
}

unsigned grid_for(int64_t threads) {
  const int64_t b = (threads + 255) / 256;
  return (unsigned)(b < 4864 ? b : 4864);  // four CTAs of eight warps on each of 152 SMs, 8 deep
}

// CTAs for each operand: of the longest, no more than eight an SM.
void cut(DensePack &p) {
  int64_t most = 0;
  for (int i = 0; i < p.count; ++i)
    if (p.rows[i] * (p.ld[i] / 8) > most) most = p.rows[i] * (p.ld[i] / 8);
  const int64_t ctas = (most + 256 * kRuns - 1) / (256 * kRuns);
  p.ctas = (unsigned)(ctas < 1216 ? ctas : 1216);
}

}  // namespace

cudaError_t dense_pack(DensePack &p, cudaStream_t s) {
  cut(p);
  return dense_launch(pack_kernel, dim3(p.ctas, (unsigned)p.count), 256, 0, 1, s, p);
}

cudaError_t dense_empty_sum(const DenseJob &j, cudaStream_t s) {
  const dim3 grid(grid_for(j.m * j.n), (unsigned)j.nbatch);
  return dense_launch(j.gated ? empty_sum_kernel<true> : empty_sum_kernel<false>, grid, 256, 0, 1,
                      s, j);
}

// Row blocks: enough CTAs for two waves of eight a multiprocessor; one turn of the rows at least
// (16), or four where column sums are left for each block.
int64_t dense_act_bwd_row_blocks(int64_t m, int64_t n, bool sums) {
  const int64_t cols = (n + COLS - 1) / COLS, least = sums ? 64 : 16;
  int64_t want = (2432 + cols - 1) / cols;
  const int64_t most = (m + least - 1) / least;
  if (want > most) want = most;
  if (want < 1) want = 1;
  if (want > 65535) want = 65535;
  const int64_t per = (m + want - 1) / want;
  return per ? (m + per - 1) / per : 1;
}

cudaError_t dense_act_bwd(const DenseActBwd &a, DensePack &pack, DenseJoin &join,
                          cudaStream_t s) {
  cut(pack);
  const int64_t blocks = dense_act_bwd_row_blocks(a.m, a.n, a.db != nullptr);
  const int64_t per = (a.m + blocks - 1) / blocks;
  const dim3 grid((unsigned)((a.n + COLS - 1) / COLS), (unsigned)blocks);
  cudaError_t err;
  switch (a.act) {
    case COLL_ACT_NONE: err = launch_act_bwd<false, COLL_ACT_NONE>(a, pack, grid, per, s); break;
#define COLL_ACT_CASE(act)                                             \
  case act:                                                            \
    err = a.gated ? launch_act_bwd<true, act>(a, pack, grid, per, s)   \
                  : launch_act_bwd<false, act>(a, pack, grid, per, s); \
    break;
    COLL_ACT_CASE(COLL_ACT_RELU)
    COLL_ACT_CASE(COLL_ACT_GELU)
    COLL_ACT_CASE(COLL_ACT_GELU_TANH)
    COLL_ACT_CASE(COLL_ACT_SILU)
#undef COLL_ACT_CASE
    default: err = launch_act_bwd<true, COLL_ACT_SIGMOID>(a, pack, grid, per, s);
  }
  join = DenseJoin{a.part, blocks, a.n, !a.gated && blocks > 1 ? a.db : nullptr, a.db_type};
  return err;
}

cudaError_t dense_join(const DenseJoin &join, cudaStream_t s) {
  return dense_launch(join_kernel, dim3((unsigned)((join.n + 255) / 256)), 256, 0, 1, s, join);
}

}  // namespace coll
