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
// Warps: 0 loads A, 3 loads B (and adds up column sums that came along), 1 issues the matrix
// instructions (the pair's first CTA only), 2 owns TMEM, 4-11 run the epilogue, two warps for each
// 32 rows, 32 columns at a time: a lane holds 32 columns of its row and accesses whole 32-byte
// sectors. Where an array's rows do not start on 16 bytes, or the row ends inside the 32 columns,
// the block passes through shared memory and neighbouring lanes take neighbouring columns. Two
// accumulators of 256 columns let the epilogue of one tile run beside the products of the next.
// The grid is persistent; tiles are walked eight rows of tiles at a time, which keeps the operands
// of the tiles in flight in L2.
//
// Measured: 4096 x 4096 x 4096 76 us (1820 TFLOP/s); gated 8192 x 14336 x 4096 with everything kept
// 1.02 ms alone (1890 TFLOP/s, tensor pipe 96 % busy) and 1.13 ms back to back, where the card's
// power cap sets the clock. Wide tiles are bound by the tensor pipe, tiles of up to 128 columns by
// issuing (about 27 ns an instruction), sums of a few k blocks by the epilogue's way to HBM
// (8192 x 8192 x 64: 53 us, 2.5 TB/s of writes, where filling the same memory reaches 3.4).
//
// Every wait is bounded: a wait that runs out sets an abort flag, the CTA's roles leave their
// loops, in-flight copies and products get time to land, TMEM is freed, and status says so.
#include <cuda.h>
#include <string.h>

#include <type_traits>

#include "dense.h"
#include "dense_epi.cuh"
#include "dense_tc.h"
#include "tcgen05.cuh"

namespace coll {
namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int CG = 2;                     // CTAs of a tile (cta_group::2)
constexpr float kJoinNs = 2500.0f;        // of joining shares, beside their bytes
constexpr int kMostShares = 16;
constexpr int kTileK = 64;                // elements of k per stage: one 128-byte swizzled row
constexpr uint32_t kABytes = 128 * 128;   // 128 rows
constexpr uint32_t kChunk = 64 * 128;     // MN-major: 64 k rows of 64 elements
constexpr int kMaxStages = 12;
constexpr uint32_t kStageOut = kEpiWarps * 32 * kPitch * 4;  // the epilogue's blocks

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem;
  uint32_t abort;
};

struct Tile {
  int prob, batch, share;
  int64_t m0, n0;
};

// t / d and what remains. Up to 2^22 by a quotient in binary32, off by one at most: a role of one
// warp pays for every instruction of its chain.
__device__ __forceinline__ uint32_t div_rem(uint32_t t, uint32_t d, uint32_t &rest) {
  uint32_t q;
  if (t < (1u << 22)) {
    q = __float2uint_rz(__fdividef((float)t, (float)d));
    int32_t r = (int32_t)(t - q * d);
    if (r < 0) {
      --q;
      r += (int32_t)d;
    } else if (r >= (int32_t)d) {
      ++q;
      r -= (int32_t)d;
    }
    rest = (uint32_t)r;
  } else {
    q = t / d;
    rest = t - q * d;
  }
  return q;
}

// k blocks [x, y) of a share, counted through the segments.
__device__ __forceinline__ int2 share_of(const TcProb &q, int share) {
  const int all = q.nseg * q.kblocks;
  if (q.split == 1) return make_int2(0, all);
  return make_int2((int)((int64_t)share * all / q.split),
                   (int)((int64_t)(share + 1) * all / q.split));
}

// The tiles of one cluster in their order: those of the first product in turn, then the second
// product's. A cluster that got one tile of the first product less takes `even` tiles of the
// second before all others join in, so that the clusters end together.
struct Walk {
  uint32_t cluster, clusters, first, extra;  // its tiles of product 0; clusters with one more
  __device__ __forceinline__ Walk(const TcParams &p) {
    clusters = gridDim.x / CG;
    cluster = blockIdx.x / CG;
    const uint32_t t = p.prob[0].tiles;
    first = t > cluster ? (t - cluster + clusters - 1) / clusters : 0;
    extra = t % clusters;
  }
  // the i-th tile; false past the last
  __device__ __forceinline__ bool at(const TcParams &p, uint32_t i, Tile &r) const {
    uint32_t t;
    r.prob = i >= first;
    if (!r.prob) {
      t = cluster + i * clusters;
    } else {
      i -= first;
      const uint32_t early = p.even * (clusters - extra);
      if (cluster >= extra && i < p.even) t = i * (clusters - extra) + cluster - extra;
      else t = early + (cluster >= extra ? i - p.even : i) * clusters + cluster;
    }
    const TcProb &q = p.prob[r.prob];
    if (t >= q.tiles) return false;
    const uint32_t per = q.tiles_m * q.tiles_n;
    uint32_t row, unit = div_rem(t, per, t);
    r.batch = 0;
    if (q.nbatch == 2) {
      r.batch = unit & 1u;
      unit >>= 1;
    }
    r.share = unit;
    const uint32_t top = div_rem(t, 8u * q.tiles_n, t) * 8u;
    const uint32_t col = div_rem(t, min(8u, q.tiles_m - top), row);
    r.m0 = (int64_t)(top + row) * (128 * CG);
    r.n0 = (int64_t)col * q.tile_cols;
    return true;
  }
};

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ TcParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  uint32_t *const staged = reinterpret_cast<uint32_t *>(raw + (ring - smem_u32(raw)) +
                                                        (size_t)p.stages * p.stage_bytes);
  // the same for all lanes, and known to be
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0u;
  const Walk walk(p);
  Tile tl;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], 2);  // A's and B's loads
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], kEpiWarps * CG);
    }
    sh.abort = 0u;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc<CG>(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  griddep_launch();
  griddep_wait();

  const uint32_t full0 = smem_u32(&sh.full[0]), empty0 = smem_u32(&sh.empty[0]);
  const uint32_t stages = p.stages, stage_bytes = p.stage_bytes;

  if (warp == 0 || warp == 3) {
    const bool first = warp == 0;  // loads A; the other B
    const uint32_t arrive0 = map_rank(full0, 0), offset = first ? 0u : kABytes;
    uint32_t s = 0, phase = 0;
    bool ok = true;
    // k blocks [k, end) of one segment of this warp's operand from row r on, `bytes` of both CTAs
    // a block (boxes past the edges counted whole); `mine`: this CTA has rows of it
    auto segment = [&](auto mn, const CUtensorMap *map, int32_t r, int32_t chunks, uint32_t bytes,
                       bool mine, int32_t k, int32_t end) {
      bool ready = bar_test(empty0 + 8 * s, phase ^ 1u);
      for (; k < end; k += kTileK) {
        if (!ready) ok = ok && wait_bar(&sh.abort, empty0 + 8 * s, phase ^ 1u, p.status);
        const uint32_t bar = arrive0 + 8 * s, full = full0 + 8 * s;
        const uint32_t d = ring + s * stage_bytes + offset;
        if (++s == stages) {
          s = 0;
          phase ^= 1u;
        }
        ready = bar_test(empty0 + 8 * s, phase ^ 1u);  // the next slot, while this one is filled
        if (elect_one() && ok) {
          if (leader) bar_expect(full, bytes);
          if (mine) {
            if (decltype(mn)::value) {
              tma_box_pair(d, map, r, k, bar);
              if (chunks > 1) tma_box_pair(d + kChunk, map, r + 64, k, bar);
            } else {
              tma_box_pair(d, map, k, r, bar);
            }
          }
        }
        __syncwarp();
      }
    };
    using Yes = std::integral_constant<bool, true>;
    using No = std::integral_constant<bool, false>;
    for (uint32_t i = 0; walk.at(p, i, tl); ++i) {
      const TcProb &q = p.prob[tl.prob];
      const int2 range = share_of(q, tl.share);
      const bool second = tl.m0 + 128 < q.m;  // the second CTA's rows of A may all be past the last
      const int32_t r = first ? (int32_t)tl.m0 + (int32_t)rank * 128
                              : (int32_t)tl.n0 + (GATED ? 0 : (int32_t)rank * q.b_rows);
      for (int seg = 0; seg < q.nseg; ++seg) {
        const int k0 = max(range.x - seg * q.kblocks, 0) * kTileK;
        const int k1 = min(range.y - seg * q.kblocks, q.kblocks) * kTileK;
        const CUtensorMap *map = first ? &q.a[q.nbatch == 2 ? tl.batch : seg]
                                       : &q.b[GATED ? (int)rank : seg];
        const bool mn = first ? q.a_mn[seg] : q.b_mn[seg];
        const int32_t chunks = first ? 2 : q.b_chunks;
        const uint32_t one = mn ? chunks * kChunk : (first ? q.a_rows : q.b_box) * 128u;
        const uint32_t bytes = first && !second ? one : CG * one;
        const bool mine = !first || leader || second;
        if (mn) segment(Yes{}, map, r, chunks, bytes, mine, k0, k1);
        else segment(No{}, map, r, chunks, bytes, mine, k0, k1);
      }
    }
    if (!GATED && !first && p.join.db)
      for (int64_t c = (int64_t)blockIdx.x * 32 + lane; c < p.join.n; c += (int64_t)gridDim.x * 32)
        join_column(p.join, c);
    // every slot's last products are done before this CTA may go away
    for (uint32_t i = 0; i < stages; ++i) {
      ok = ok && wait_bar(&sh.abort, empty0 + 8 * s, phase ^ 1u, p.status);
      if (++s == stages) {
        s = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const uint32_t hi = desc_hi(1024), step = stage_bytes >> 4;
      const uint32_t acc_full0 = smem_u32(&sh.acc_full[0]), acc_empty0 = smem_u32(&sh.acc_empty[0]);
      uint32_t s = 0, phase = 0, at = 0;  // at: 16-byte units from the ring's start
      bool ok = true;
      for (uint32_t it = 0; walk.at(p, it, tl); ++it) {
        const TcProb &q = p.prob[tl.prob];
        const uint32_t buf = it & 1u, d = tmem + buf * 256u;
        ok = ok && wait_bar(&sh.abort, acc_empty0 + 8 * buf, ((it >> 1) & 1u) ^ 1u, p.status);
        tc_fence_after();
        uint32_t add = 0;
        const int2 range = share_of(q, tl.share);
        for (int seg = 0; seg < q.nseg; ++seg) {
          const bool amn = q.a_mn[seg], bmn = q.b_mn[seg];  // batches lie alike
          // an MN-major operand's next 16 of k are 16 rows on, a K-major one's 32 bytes
          const uint32_t as = amn ? 2048u >> 4 : 32u >> 4, bs = bmn ? 2048u >> 4 : 32u >> 4;
          const uint32_t a0 = desc_lo(ring, amn ? kChunk : 16u);
          const uint32_t b0 = desc_lo(ring + kABytes, bmn ? kChunk : 16u);
          const uint32_t idesc = q.idesc | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16);
          const int kb0 = max(range.x - seg * q.kblocks, 0);
          const int kb1 = min(range.y - seg * q.kblocks, q.kblocks);
          for (int kb = kb0; kb < kb1; ++kb) {
            ok = ok && wait_bar(&sh.abort, full0 + 8 * s, phase, p.status);
            tc_fence_after();
            if (elect_one() && ok) {
              const uint32_t a = a0 + at, b = b0 + at;
              mma_f16<CG>(d, a, hi, b, hi, idesc, add);
              mma_f16<CG>(d, a + as, hi, b + bs, hi, idesc, 1);
              mma_f16<CG>(d, a + 2 * as, hi, b + 2 * bs, hi, idesc, 1);
              mma_f16<CG>(d, a + 3 * as, hi, b + 3 * bs, hi, idesc, 1);
              mma_commit<CG>(empty0 + 8 * s, 3);
            }
            __syncwarp();
            add = 1;
            at += step;
            if (++s == stages) {
              s = 0;
              at = 0;
              phase ^= 1u;
            }
          }
        }
        if (elect_one() && ok) mma_commit<CG>(acc_full0 + 8 * buf, 3);
        __syncwarp();
      }
    }
  } else if (warp >= 4) {
    const int quad = warp & 3, part = (warp - 4) >> 2;
    uint32_t *const st = staged + (warp - 4) * 32 * kPitch;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    // The residual's lines of a tile into L2 while its products run, a lane for its row, every
    // other line each of the two warps of a row: a block then waits for L2, not for HBM (8192 x
    // 8192 with bias, gelu and residual: 124 -> 109 us).
    auto fetch = [&](const Tile &tl) {
      const TcProb &q = p.prob[tl.prob];
      const int64_t row = tl.m0 + rank * 128 + quad * 32 + lane;
      if (GATED || !q.e.res || q.e.res_cs != 1 || row >= q.m) return;
      const int cols = (int)min((int64_t)q.tile_cols, q.n - tl.n0);
      const int es = q.e.out_type == COLL_F32 ? 4 : 2, line = 128 / es;
      const char *at = static_cast<const char *>(q.e.res) + (row * q.e.res_rs + tl.n0) * es;
      for (int c = part * line; c < cols; c += 2 * line)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c * es));
    };
    for (uint32_t it = 0; walk.at(p, it, tl); ++it) {
      const TcProb &q = p.prob[tl.prob];
      const DenseEpi &e = q.e;
      const bool pre_res = !GATED && e.vec && e.res && e.out_type != COLL_F32;
      const uint32_t buf = it & 1u;
      const int64_t row0 = tl.m0 + rank * 128 + quad * 32, row = row0 + lane;
      const bool live = row < q.m;
      const int cols = (int)min((int64_t)q.tile_cols, q.n - tl.n0);
      // The bias (a lane's column) and the residual of the next 32 columns, asked for ahead: the
      // bias loaded at its use cost 20 to 40 us of 8192 x 8192 outputs.
      uint32_t r[16];
      uint16_t bias = 0;
      auto ask = [&](int c0) {
        if (!GATED && e.bias && c0 + lane < cols)
          bias = static_cast<const uint16_t *>(e.bias)[(tl.n0 + c0 + lane) * e.bias_stride];
        if (pre_res && live && c0 + 32 <= cols) ld_halves(e.res, row * e.res_rs + tl.n0 + c0, r);
      };
      ask(part * 32);
      fetch(tl);
      if (!__all_sync(~0u, wait_bar(&sh.abort, smem_u32(&sh.acc_full[buf]), (it >> 1) & 1u,
                                    p.status)))
        break;
      tc_fence_after();
      for (int c0 = part * 32; c0 < cols; c0 += 64) {
        float g[32], u[GATED ? 32 : 1];
        const uint32_t at = lanes + buf * 256u + c0;
        tmem_load32(at, g);
        if constexpr (GATED) tmem_load32(at + q.tile_cols, u);
        const int64_t col = tl.n0 + c0;
        if (q.split > 1) {  // this share's sums; whole runs, the rows are padded for them
          if (live) {
            const int64_t plane = (tl.share * q.nbatch + tl.batch) * (GATED ? 2 : 1);
            st_run32(q.part, (plane * q.m + row) * q.part_ld + col, COLL_F32, g);
            if constexpr (GATED)
              st_run32(q.part, ((plane + 1) * q.m + row) * q.part_ld + col, COLL_F32, u);
          }
          continue;
        }
        const bool vec = e.vec && c0 + 32 <= cols;
        const int rows = (int)max((int64_t)0, min((int64_t)32, q.m - row0));
        const int left = min(32, cols - c0);
        auto store = [&](void *base, int64_t rs, int type, const float (&v)[32]) {
          if (vec) {
            if (live) st_run32(base, row * rs + col, type, v);
          } else {
            const int64_t at0 = row0 * rs + col;
            staged_store(st, static_cast<char *>(base) + at0 * (type == COLL_F32 ? 4 : 2), rs, type,
                         rows, left, v);
          }
        };
        if constexpr (GATED) {
          if (e.gate) {
            store(e.gate, e.gate_rs, e.type, g);
            store(e.up, e.up_rs, e.type, u);
          }
          act_run(g, e.act);
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] *= u[i];
        } else {
          if (e.bias) add_lanes(st, h2f(bias, e.type), g);
          if (e.pre) store(e.pre, e.pre_rs, e.type, g);
          act_run(g, e.act);
          if (e.res) {
            if (!vec) {
              const int64_t at0 = row0 * e.res_rs + col * e.res_cs;
              staged_add(st,
                         static_cast<const char *>(e.res) + at0 * (e.out_type == COLL_F32 ? 4 : 2),
                         e.res_rs, e.res_cs, e.out_type, rows, left, g);
            } else if (pre_res) {
              add_halves(g, r, e.type);
            } else if (live) {
              const float *rp = static_cast<const float *>(e.res) + row * e.res_rs + col;
              uint32_t x[32];
              ld_row<32>(rp, x);
#pragma unroll
              for (int i = 0; i < 32; ++i) g[i] += __uint_as_float(x[i]);
            }
          }
          ask(c0 + 64);
        }
        store(e.out[tl.batch], e.out_rs[tl.batch], e.out_type, g);
      }
      tc_fence_before();  // this warp has read its part of the accumulator
      __syncwarp();
      if (lane == 0) {
        if (!leader) mbar_arrive_remote(map_rank(smem_u32(&sh.acc_empty[buf]), 0));
        else mbar_arrive(&sh.acc_empty[buf]);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (sh.abort) drain();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<CG>(tmem, 512);
  }
}

// The shares of a split product, added in order of k, and its epilogue: a thread takes one output.
struct ShareJoin {
  DenseJob j[2];
  const float *part[2];
  int64_t part_ld[2];
  int32_t split[2];
};

template <bool GATED>
__global__ void __launch_bounds__(256) share_join_kernel(const __grid_constant__ ShareJoin s) {
  griddep_launch();
  griddep_wait();
  const int w = blockIdx.z;
  const DenseJob &j = s.j[w];
  const int64_t ld = s.part_ld[w], plane = j.m * ld, col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int split = s.split[w];
  if (split < 2 || col >= j.n) return;
  const int64_t rows = j.m * j.nbatch, step = plane * j.nbatch * (GATED ? 2 : 1);
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const int batch = r >= j.m;
    const int64_t row = r - batch * j.m;
    const float *p = s.part[w] + batch * plane + row * ld + col;
    // everything in flight before the first is added
    float a[kMostShares], b[GATED ? kMostShares : 1];
#pragma unroll
    for (int i = 0; i < kMostShares; ++i) {
      a[i] = i < split ? p[i * step] : 0.0f;
      if constexpr (GATED) b[i] = i < split ? p[i * step + plane] : 0.0f;
    }
    const Addends more = ask_addends<GATED>(j.e, row, col);
    float g = a[0], u = GATED ? b[0] : 0.0f;
#pragma unroll
    for (int i = 1; i < kMostShares; ++i) {
      g += a[i];
      if constexpr (GATED) u += b[i];
    }
    epilogue_one<GATED>(j.e, batch, row, col, g, u, more);
  }
}

template <bool GATED>
cudaError_t set_up() {
  static DenseSmemLimit limit;
  return limit((const void *)tc_kernel<GATED>, kTcSmem);
}

template <bool GATED>
cudaError_t launch(const TcParams &p, uint32_t clusters, uint32_t smem, cudaStream_t s) {
  return dense_launch(tc_kernel<GATED>, dim3(clusters * CG), kThreads, smem, CG, s, p);
}

// ns a tile's epilogue takes for each column of its accumulator (256 rows, two CTAs)
float epilogue_ns(const DenseJob &j, int split) {
  if (split > 1) return 14.0f;
  const DenseEpi &e = j.e;
  const float act = j.gated || e.act == COLL_ACT_NONE || e.act == COLL_ACT_RELU ? 0.0f : 6.0f;
  return 7.0f + (e.out_type == COLL_F32 ? 7.0f : 0.0f) + (e.res ? 8.5f : 0.0f) +
         (e.bias ? 2.0f : 0.0f) + (e.pre ? 5.0f : 0.0f) + (e.gate ? 8.0f : 0.0f) + act +
         (e.vec ? 0.0f : 4.0f);
}

int operands_a(const DenseJob &j) { return j.nbatch == 2 || j.nseg == 2 ? 2 : 1; }
int operands_b(const DenseJob &j) { return j.gated || j.nseg == 2 ? 2 : 1; }

uint32_t ceil_div(int64_t a, int64_t b) { return (uint32_t)((a + b - 1) / b); }

}  // namespace

int tc_encode(CUtensorMap *map, const TcOperand &o, int64_t type, uint32_t rows) {
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

int tc_plan(TcParams &p, const TcJob *jobs, int count, uint64_t (&part_bytes)[2]) {
  memset(&p, 0, sizeof(p));
  constexpr uint32_t clusters = kSms / CG;
  // Columns of each product's accumulator and shares of its k: those that end first. A tile takes
  // its k blocks times 62 ns and 1.08 a column (measured at 4096 x 4096 x 8192: 144 ns for 64
  // columns, 186 for 128, 264 for 192, 339 for 256) or the time of its epilogue beside the next
  // tile's products, and every cluster its tiles one after the other; the last epilogue comes on
  // top. An epilogue takes 1.35 us and 7 ns a column, 8.5 more for a residual, 6 for an activation
  // and 2 for a bias (8192 x 8192 x 64: 53 us plain, 84 with a residual, 75 with gelu, 109 with
  // everything); where both take long, not all of the shorter one is hidden (4864 rows, k = 512,
  // 256 columns: 4.05 us a round of 2.7 and 3.2).
  // Joining shares costs a launch and their way through L2. Calls of a few us wait for this, so it
  // tries no more than it has to.
  struct Option {
    int cols, split;
    uint32_t tiles;
    float main, last, join;  // ns: a tile's products, its epilogue; joining shares
    float time() const {
      const float less = main < last ? main : last, more = main < last ? last : main;
      return more + (less < 2700.0f ? 0.3f * less : 800.0f);
    }
  };
  auto option = [&](int i, int bn, int sp) {
    const DenseJob &j = *jobs[i].j;
    Option o = {bn, sp, 0, 0.0f, 0.0f, 0.0f};
    const int64_t tiles =
        (int64_t)ceil_div(j.m, 128 * CG) * ceil_div(j.n, j.gated ? bn / 2 : bn) * j.nbatch * sp;
    o.tiles = tiles > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)tiles;
    o.main = (float)ceil_div((int64_t)ceil_div(j.k, kTileK) * j.nseg, sp) * (62.0f + 1.08f * bn);
    o.last = 1350.0f + bn * epilogue_ns(j, sp);
    if (sp > 1)
      o.join = kJoinNs +
               (float)j.m * (float)j.n * (float)(j.nbatch * (j.gated ? 2 : 1) * sp) / 500.0f;
    return o;
  };
  auto even = [&](const Option &o, const Option &q) {
    return (uint32_t)(o.time() / q.time() + 0.5f);
  };
  // the busiest cluster: of those with one tile of the first product more, or of the others
  auto makespan = [&](const Option &o, const Option *q) {
    const uint32_t whole = o.tiles / clusters, extra = o.tiles % clusters;
    float with = (float)(whole + 1), t = o.time(), end = o.last, join = o.join;
    float without = (float)whole * t;
    with *= t;
    if (q) {
      const uint32_t e = even(o, *q), early = e * (clusters - extra);
      if (q->tiles > early) {
        const float more = (float)((q->tiles - early + clusters - 1) / clusters);
        with += more * q->time();
        without += (more + (float)e) * q->time();
      } else {
        without += (float)((q->tiles + clusters - extra - 1) / (clusters - extra)) * q->time();
      }
      end = q->last;
      join = join > q->join ? join : q->join;
    }
    const float busy = extra && with > without ? with : without;
    // nothing waits for an epilogue before the first tile's products
    return busy - (o.last > o.main ? o.last - o.main : 0.0f) + end + join;
  };
  Option best[2];
  float least = 3.0e38f;
  auto keep = [&](const Option &o, const Option *q) {
    const float t = makespan(o, q);
    if (t >= least) return;
    least = t;
    best[0] = o;
    if (q) best[1] = *q;
  };
  Option second[7];
  if (count == 2)
    for (int x = 0; x < 7; ++x) second[x] = option(1, 256 - 32 * x, 1);
  for (int bn = 256; bn >= 64; bn -= jobs[0].j->gated ? 64 : 32) {
    const Option o = option(0, bn, 1);
    if (count == 1) keep(o, nullptr);
    else
      for (const Option &q : second) keep(o, &q);
  }
  // shares of k, where a tile takes a good part of the whole time
  for (int i = 0; i < count; ++i) {
    if (best[i].main * 2 < least) continue;
    const Option other = best[1 - i < count ? 1 - i : i];
    const int64_t blocks = (int64_t)ceil_div(jobs[i].j->k, kTileK) * jobs[i].j->nseg;
    for (int bn = 256; bn >= 64; bn -= 64)
      for (int sp = 2; sp <= kMostShares && blocks >= 4 * sp; sp += sp < 4 ? 1 : sp < 8 ? 2 : 4) {
        const Option o = option(i, bn, sp);
        if (o.tiles > 4 * clusters) break;
        if (count == 1) keep(o, nullptr);
        else if (i == 0) keep(o, &other);
        else keep(other, &o);
      }
  }
  // with one product's shares settled the other's columns may be better off elsewhere
  if (count == 2 && best[0].split + best[1].split > 2) {
    const Option o = best[0], q = best[1];
    for (int bn = 256; bn >= 64; bn -= 32) {
      const Option a = option(0, bn, o.split), b = option(1, bn, q.split);
      keep(a, &q);
      keep(o, &b);
    }
  }
  p.status = jobs[0].j->status;
  for (int i = 0; i < count; ++i) {
    const DenseJob &j = *jobs[i].j;
    TcProb &q = p.prob[i];
    const int cols = best[i].cols, split = best[i].split;
    if (best[i].tiles == 0x7FFFFFFFu) return COLL_EINVAL;
    q.m = j.m;
    q.n = j.n;
    q.nseg = j.nseg;
    q.nbatch = j.nbatch;
    q.split = split;
    q.kblocks = (int32_t)ceil_div(j.k, kTileK);
    q.tiles_m = ceil_div(j.m, 128 * CG);
    q.a_rows = j.m < 128 ? (int32_t)((j.m + 7) / 8 * 8) : 128;
    q.b_rows = cols / CG;
    q.tile_cols = j.gated ? cols / 2 : cols;
    q.b_box = j.n < q.b_rows ? (int32_t)((j.n + 7) / 8 * 8) : q.b_rows;
    q.b_chunks = (q.b_rows + 63) / 64;
    q.tiles_n = ceil_div(j.n, q.tile_cols);
    q.tiles = best[i].tiles;
    q.idesc = mma_desc(j.e.type == COLL_BF16, false, false, 128 * CG, (uint32_t)cols);
    q.part_ld = (j.n + 31) / 32 * 32;
    part_bytes[i] =
        split > 1 ? (uint64_t)split * j.nbatch * (j.gated ? 2 : 1) * j.m * q.part_ld * 4 : 0;
    bool bmn = false;
    for (int x = 0; x < 2; ++x) {
      q.a_mn[x] = jobs[i].a[x].mn;
      q.b_mn[x] = jobs[i].b[x].mn;
    }
    for (int x = 0; x < operands_b(j); ++x) bmn = bmn || q.b_mn[x];
    const uint32_t rows = bmn ? (uint32_t)q.b_chunks * 64u : (uint32_t)q.b_rows;
    const uint32_t bytes = kABytes + ((rows * 128u + 1023u) & ~1023u);
    if (bytes > p.stage_bytes) p.stage_bytes = bytes;
  }
  for (int i = count; i < 2; ++i) part_bytes[i] = 0;
  p.even = count == 2 && best[0].tiles % clusters ? even(best[0], best[1]) : 0;
  p.stages = (kTcSmem - 1024 - kStageOut) / p.stage_bytes;
  if (p.stages > (uint32_t)kMaxStages) p.stages = kMaxStages;
  return COLL_OK;
}

int tc_prepare(TcParams &p, const TcJob *jobs, int count) {
  for (int i = 0; i < count; ++i) {
    const DenseJob &j = *jobs[i].j;
    TcProb &q = p.prob[i];
    q.e = j.e;
    for (int x = 0; x < operands_a(j); ++x) {
      const int c = tc_encode(&q.a[x], jobs[i].a[x], j.e.type, (uint32_t)q.a_rows);
      if (c) return c;
    }
    for (int x = 0; x < operands_b(j); ++x) {
      const int c = tc_encode(&q.b[x], jobs[i].b[x], j.e.type, (uint32_t)q.b_box);
      if (c) return c;
    }
  }
  return (jobs[0].j->gated ? set_up<true>() : set_up<false>()) == cudaSuccess ? COLL_OK
                                                                              : COLL_ECUDA;
}

cudaError_t tc_run(const TcParams &p, const TcJob *jobs, int count, cudaStream_t s) {
  ShareJoin join = {};
  int64_t cols = 0, rows = 0;
  for (int i = 0; i < count; ++i) {
    const DenseJob &j = *jobs[i].j;
    const TcProb &q = p.prob[i];
    join.split[i] = q.split;
    if (q.split > 1) {
      join.j[i] = j;
      join.part[i] = q.part;
      join.part_ld[i] = q.part_ld;
      if (j.n > cols) cols = j.n;
      if (j.m * j.nbatch > rows) rows = j.m * j.nbatch;
    }
  }
  const bool gated = jobs[0].j->gated != 0;
  const uint64_t most = kSms / CG, tiles = (uint64_t)p.prob[0].tiles + p.prob[1].tiles;
  // with two products every cluster takes part: the tiles are dealt for all of them
  const uint32_t clusters = (uint32_t)(tiles < most && count == 1 ? tiles : most);
  const uint32_t smem = 1024 + p.stages * p.stage_bytes + kStageOut;
  cudaError_t e = gated ? launch<true>(p, clusters, smem, s) : launch<false>(p, clusters, smem, s);
  if (e == cudaSuccess && cols) {
    const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)(rows < 1024 ? rows : 1024),
                    (unsigned)count);
    e = dense_launch(gated ? share_join_kernel<true> : share_join_kernel<false>, grid, 256, 0, 1, s,
                     join);
  }
  return e;
}

}  // namespace coll
