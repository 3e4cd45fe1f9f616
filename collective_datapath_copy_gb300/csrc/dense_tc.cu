// The products of the dense operators on the tensor cores (tcgen05).
//
// out = epilogue(A B^T): A [m][k], B [n][k], 16-bit, binary32 accumulators in TMEM. Each operand
// is read by TMA as it lies in memory, rows along k (K-major) or along m or n (MN-major: the
// transposed views of the backward products), into 128-byte-swizzled tiles; the major axis is a
// bit of the instruction descriptor and two offsets of the matrix descriptor, so one kernel takes
// all four combinations.
//
// A pair of CTAs (cta_group::2) computes a tile of 256 rows by up to 256 columns: each CTA holds
// 128 rows of A and half of B's rows, so a k step of 64 brings 32 KiB per SM for 2 x 128 x 256 x
// 64 multiply-adds. Gated: CTA 0 holds rows of the gate's weights and CTA 1 the same rows of the
// up weights, and the accumulator's halves are g and u of the same columns.
//
// Warps: 0 loads (one thread), 1 issues the matrix instructions (the pair's first CTA only), 2
// owns TMEM, 4-7 run the epilogue: TMEM -> registers (a row per lane) -> shared memory -> eight
// consecutive columns per lane, so that global accesses are 16 bytes a lane and 64 contiguous
// bytes a row. Two accumulators of 256 columns let the epilogue of one tile run beside the
// products of the next. The grid is persistent; tiles are walked eight rows of tiles at a time,
// which keeps the operands of the tiles in flight in L2.
//
// Every wait is bounded: a wait that runs out sets an abort flag, the CTA's roles leave their
// loops, in-flight copies and products get time to land, TMEM is freed, and status says so.
#include <cuda.h>
#include <string.h>

#include "dense.h"
#include "dense_epi.cuh"
#include "dense_tc.h"
#include "tcgen05.cuh"

namespace coll {
namespace {

constexpr int kThreads = 256;
constexpr int kTileK = 64;                // elements of k per stage: one 128-byte swizzled row
constexpr uint32_t kABytes = 128 * 128;   // 128 rows
constexpr uint32_t kChunk = 64 * 128;     // MN-major: 64 k rows of 64 elements
constexpr int kMaxStages = 12;
constexpr int kPitch = 36;                // floats per staged row: 32 and a bank shift
constexpr uint32_t kStageOut = 4 * 32 * kPitch * 4;
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 20000000ull;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
  uint32_t abort;
};

// Wait for a phase; on failure raise the abort flag and the caller's status.
__device__ __forceinline__ bool wait_bar(Shared *sh, uint64_t *bar, uint32_t parity,
                                         int32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile uint32_t *flag = &sh->abort;
  if (mbar_wait(bar, parity, kLimitNs, flag)) return true;
  if (!*flag) {
    *flag = 1u;
    if (status) *status = COLL_ETIMEDOUT;
  }
  return false;
}

struct Tile {
  int batch;
  int64_t m0, n0;
};

__device__ __forceinline__ Tile tile_at(const TcParams &p, uint32_t t) {
  Tile r;
  const uint32_t per = p.tiles_m * p.tiles_n;
  r.batch = t / per;
  t -= r.batch * per;
  const uint32_t group = 8u * p.tiles_n, g = t / group, first = g * 8u;
  const uint32_t rows = min(8u, p.tiles_m - first), in = t - g * group;
  r.m0 = (int64_t)(first + in % rows) * p.tile_rows;
  r.n0 = (int64_t)(in / rows) * p.tile_cols;
  return r;
}

template <int CG, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ TcParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  float *const staged = reinterpret_cast<float *>(raw + (ring - smem_u32(raw)) +
                                                  (size_t)p.stages * p.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const bool leader = rank == 0u;
  const uint32_t clusters = gridDim.x / CG, cluster = blockIdx.x / CG;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 4 * CG);
    }
    sh.abort = 0u;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<CG>(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, phase = 0;
      bool ok = true;
      for (uint32_t t = cluster; ok && t < p.tiles; t += clusters) {
        const Tile tl = tile_at(p, t);
        const int32_t m = (int32_t)tl.m0 + (int32_t)rank * 128;
        for (int seg = 0; ok && seg < p.nseg; ++seg) {
          const CUtensorMap *ma = &p.a[p.nbatch == 2 ? tl.batch : seg];
          const CUtensorMap *mb = &p.b[GATED && CG == 2 ? rank : seg];
          const int32_t n = (int32_t)tl.n0 + (GATED ? 0 : (int32_t)rank * p.b_rows);
          const bool amn = p.a_mn[p.nbatch == 2 ? tl.batch : seg];
          const bool bmn = p.b_mn[GATED && CG == 2 ? rank : seg];
          // bytes a stage receives, boxes past the edges counted whole
          const uint32_t kr = p.b_rows * 128, mr = p.b_chunks * kChunk;
          const uint32_t bytes =
              CG * kABytes + (GATED ? (p.b_mn[0] ? mr : kr) + (p.b_mn[1] ? mr : kr)
                                    : CG * (bmn ? mr : kr));
          for (int kb = 0; kb < p.kblocks; ++kb) {
            if (!wait_bar(&sh, &sh.empty[s], phase ^ 1u, p.status)) {
              ok = false;
              break;
            }
            uint32_t bar = smem_u32(&sh.full[s]);
            if (leader) mbar_expect_tx(&sh.full[s], bytes);
            if (CG == 2) bar = map_rank(bar, 0);
            const uint32_t da = ring + s * p.stage_bytes, db = da + kABytes;
            const int32_t k = kb * kTileK;
            auto load = [&](uint32_t d, const CUtensorMap *map, int32_t x, int32_t y) {
              if (CG == 2) tma_box_pair(d, map, x, y, bar);
              else tma_box(d, map, x, y, bar);
            };
            if (amn) {
              load(da, ma, m, k);
              load(da + kChunk, ma, m + 64, k);
            } else {
              load(da, ma, k, m);
            }
            if (bmn) {
              for (int c = 0; c < p.b_chunks; ++c) load(db + c * kChunk, mb, n + 64 * c, k);
            } else {
              load(db, mb, k, n);
            }
            if (GATED && CG == 1) {
              const uint32_t d2 = db + p.b_rows * 128;
              if (p.b_mn[1]) {
                for (int c = 0; c < p.b_chunks; ++c) load(d2 + c * kChunk, &p.b[1], n + 64 * c, k);
              } else {
                load(d2, &p.b[1], k, n);
              }
            }
            if (++s == (uint32_t)p.stages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
      }
      // every slot's last products are done before this CTA may go away
      for (int i = 0; ok && i < p.stages; ++i) {
        ok = wait_bar(&sh, &sh.empty[s], phase ^ 1u, p.status);
        if (++s == (uint32_t)p.stages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      const uint64_t kd = smem_desc(16, 1024), md = smem_desc(kChunk, 1024);
      uint32_t s = 0, phase = 0, it = 0;
      bool ok = true;
      for (uint32_t t = cluster; ok && t < p.tiles; t += clusters, ++it) {
        const uint32_t buf = it & 1u, d = tmem + buf * 256u;
        if (!wait_bar(&sh, &sh.acc_empty[buf], ((it >> 1) & 1u) ^ 1u, p.status)) break;
        tc_fence_after();
        const int batch = p.nbatch == 2 ? tile_at(p, t).batch : 0;
        bool add = false;
        for (int seg = 0; ok && seg < p.nseg; ++seg) {
          const int ia = p.nbatch == 2 ? batch : seg;
          const bool amn = p.a_mn[ia], bmn = p.b_mn[seg];
          const uint64_t ad = amn ? md : kd, bd = bmn ? md : kd;
          const uint32_t as = amn ? 2048u : 32u, bs = bmn ? 2048u : 32u;
          const uint32_t idesc = p.idesc | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16);
          for (int kb = 0; kb < p.kblocks; ++kb) {
            if (!wait_bar(&sh, &sh.full[s], phase, p.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = ring + s * p.stage_bytes, sb = sa + kABytes;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mma_f16<CG>(d, desc_at(ad, sa + q * as), desc_at(bd, sb + q * bs), idesc, add);
              add = true;
            }
            mma_commit<CG>(&sh.empty[s], 3);
            if (++s == (uint32_t)p.stages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
        if (ok) mma_commit<CG>(&sh.acc_full[buf], 3);
      }
    }
  } else if (warp >= 4) {
    const int quad = warp & 3;
    float *const st = staged + quad * 32 * kPitch;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int rr = lane >> 2, cc = (lane & 3) * 8;
    uint32_t it = 0;
    for (uint32_t t = cluster; t < p.tiles; t += clusters, ++it) {
      const Tile tl = tile_at(p, t);
      const uint32_t buf = it & 1u;
      if (!__all_sync(~0u, wait_bar(&sh, &sh.acc_full[buf], (it >> 1) & 1u, p.status))) break;
      tc_fence_after();
      const int64_t row0 = tl.m0 + rank * 128 + quad * 32;
      const int cols = (int)min((int64_t)p.tile_cols, p.n - tl.n0);
      for (int c0 = 0; c0 < cols; c0 += 32) {
        float v[32], g[4][8], u[4][8];
        const uint32_t at = lanes + buf * 256u + c0;
#pragma unroll
        for (int w = 0; w < (GATED ? 2 : 1); ++w) {
          tmem_load32(at + w * p.tile_cols, v);
          if (c0 + 32 >= cols && w == (GATED ? 1 : 0)) {  // the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (CG == 2 && !leader) mbar_arrive_remote(map_rank(smem_u32(&sh.acc_empty[buf]), 0));
              else mbar_arrive(&sh.acc_empty[buf]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4 *>(st + lane * kPitch + 4 * q) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 x = *reinterpret_cast<const float4 *>(st + (q * 8 + rr) * kPitch + cc);
            const float4 y =
                *reinterpret_cast<const float4 *>(st + (q * 8 + rr) * kPitch + cc + 4);
            float *o = w ? u[q] : g[q];
            o[0] = x.x, o[1] = x.y, o[2] = x.z, o[3] = x.w;
            o[4] = y.x, o[5] = y.y, o[6] = y.z, o[7] = y.w;
          }
        }
        const int64_t left = (int64_t)cols - c0 - cc;
        if (left > 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int64_t row = row0 + q * 8 + rr;
            if (row < p.m)
              epilogue_run8<GATED>(p.e, tl.batch, row, tl.n0 + c0 + cc, left, g[q], u[q]);
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (sh.abort) {  // let copies and products in flight land
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < kDrainNs) __nanosleep(1000);
  }
  if (CG == 2) cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<CG>(tmem, 512);
  }
}

template <int CG, bool GATED>
cudaError_t launch(const TcParams &p, uint32_t clusters, uint32_t smem, cudaStream_t s) {
  static const cudaError_t ready = cudaFuncSetAttribute(
      tc_kernel<CG, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
  if (ready != cudaSuccess) return ready;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CG == 2 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, tc_kernel<CG, GATED>, p);
}

int encode(CUtensorMap *map, const TcOperand &o, int64_t type, uint32_t rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return COLL_ECUDA;
  const cuuint64_t inner = (cuuint64_t)(o.mn ? o.rows : o.k);
  const cuuint64_t dims[2] = {inner, (cuuint64_t)(o.mn ? o.k : o.rows)};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
  const cuuint32_t box[2] = {64, o.mn ? 64u : rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map,
            type == COLL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            2, const_cast<void *>(o.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? COLL_OK
             : COLL_EINVAL;
}

uint32_t ceil_div(int64_t a, int64_t b) { return (uint32_t)((a + b - 1) / b); }

}  // namespace

int tc_plan(TcParams &p, const DenseJob &j, const TcOperand *a, const TcOperand *b,
            uint32_t sms) {
  memset(&p, 0, sizeof(p));
  p.e = j.e;
  p.m = j.m;
  p.n = j.n;
  p.status = j.status;
  p.nseg = j.nseg;
  p.nbatch = j.nbatch;
  p.kblocks = (int32_t)ceil_div(j.k, kTileK);
  const uint32_t cg = 2, clusters = sms / cg;
  p.tile_rows = 128 * cg;
  p.tiles_m = ceil_div(j.m, p.tile_rows);
  // Columns of the accumulator: the widest (least operand traffic) unless a narrower tile fills
  // the last wave better. A tile costs its columns plus a fixed part of about 24 (its epilogue's
  // tail and the ring's refill).
  int best = 256;
  int64_t cost = INT64_MAX;
  for (int bn = 256; bn >= 64; bn -= j.gated ? 64 : 32) {
    const int64_t cols = j.gated ? bn / 2 : bn;
    const int64_t tiles = (int64_t)p.tiles_m * ceil_div(j.n, cols) * j.nbatch;
    const int64_t c = (tiles + clusters - 1) / clusters * (bn + 24);
    if (c < cost) {
      cost = c;
      best = bn;
    }
  }
  p.b_rows = best / (int)cg;
  p.tile_cols = j.gated ? best / 2 : best;
  p.b_chunks = (p.b_rows + 63) / 64;
  p.tiles_n = ceil_div(j.n, p.tile_cols);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * j.nbatch;
  if (tiles > 0x7FFFFFFF) return COLL_EINVAL;
  p.tiles = (uint32_t)tiles;
  const int na = j.nbatch == 2 || j.nseg == 2 ? 2 : 1, nb = j.gated || j.nseg == 2 ? 2 : 1;
  bool bmn = false;
  for (int i = 0; i < na; ++i) {
    p.a_mn[i] = a[i].mn;
    const int c = encode(&p.a[i], a[i], j.e.type, 128);
    if (c) return c;
  }
  for (int i = 0; i < nb; ++i) {
    p.b_mn[i] = b[i].mn;
    bmn = bmn || b[i].mn;
    const int c = encode(&p.b[i], b[i], j.e.type, (uint32_t)p.b_rows);
    if (c) return c;
  }
  const uint32_t rows = bmn ? (uint32_t)p.b_chunks * 64u : (uint32_t)p.b_rows;
  p.stage_bytes = kABytes + ((rows * 128u + 1023u) & ~1023u);
  p.stages = (int32_t)((kTcSmem - 1024 - kStageOut) / p.stage_bytes);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.idesc = mma_desc(j.e.type == COLL_BF16, false, false, 128 * cg, (uint32_t)best);
  return COLL_OK;
}

cudaError_t tc_run(const TcParams &p, bool gated, uint32_t sms, cudaStream_t s) {
  const uint32_t most = sms / 2, clusters = p.tiles < most ? p.tiles : most;
  const uint32_t smem = 1024 + (uint32_t)p.stages * p.stage_bytes + kStageOut;
  return gated ? launch<2, true>(p, clusters, smem, s) : launch<2, false>(p, clusters, smem, s);
}

}  // namespace coll
