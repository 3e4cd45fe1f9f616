// The products of the dense operators for a small batch of tokens against many output features, on
// the tensor cores with the operands' roles turned: the weights are the 128-row operand, the
// tokens its columns, so no byte that is streamed is padding.
//
// Bound by HBM: every weight is read once (2 n k bytes, gated 4 n k) and each SM has to keep
// about 45 bytes a nanosecond arriving. A CTA takes up to 128 output features (gated: of both
// matrices, two accumulators in the same lanes) over the whole of k; how many is chosen for the
// least time of the busiest SM (skinny_plan), and dense.cu sends only products here whose features
// occupy every SM that way. Against the kernel of CTA pairs, which takes the tokens as rows:
// 14336 x 4096 for 17 to 64 tokens 23 us against 25, gated 41 us (5.7 TB/s) against 45.
//
// Two CTAs fit an SM, so that one's start and end run beside the other's stream. Tensor memory is
// never oversubscribed: the shared memory a CTA asks for keeps a third one off the SM and a CTA
// takes at most 256 of the 512 columns.
#include <cuda.h>
#include <string.h>

#include <type_traits>

#include "dense.h"
#include "dense_epi.cuh"
#include "dense_tc.h"
#include "tcgen05.cuh"

namespace coll {
namespace {

constexpr int kThreads = 192;  // 0 loads, 1 matrix instructions and TMEM, 2-5 epilogue
constexpr int kTileK = 64;
constexpr uint32_t kChunk = 64 * 128;
constexpr int kMaxStages = 12;
constexpr uint32_t kTwoPerSm = 112 * 1024;   // most shared memory that lets two CTAs share an SM
constexpr uint32_t kNoThird = 80 * 1024;     // least that keeps a third one off

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], done;
  uint32_t tmem;
  uint32_t abort;
};

// Up to 32 tokens of one feature (lane): values g (and u) are finished and stored; a warp's lanes
// are neighbouring features, so every access is to neighbouring elements.
template <bool GATED, int TYPE, bool F32>
__device__ __forceinline__ void finish32(const DenseEpi &e, int64_t t0, int64_t f, int tokens,
                                         bool live, float (&g)[32], float (&u)[GATED ? 32 : 1]) {
  auto store = [&](void *base, int64_t rs, const float(&v)[32], auto wide) {
    constexpr bool W = decltype(wide)::value;
    char *o = static_cast<char *>(base) + (t0 * rs + f) * (W ? 4 : 2);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i < tokens && live) {
        if (W) *reinterpret_cast<float *>(o) = v[i];
        else *reinterpret_cast<uint16_t *>(o) = f2h(v[i], TYPE);
      }
      o += rs * (W ? 4 : 2);
    }
  };
  using Wide = std::integral_constant<bool, true>;
  using Half = std::integral_constant<bool, false>;
  if constexpr (GATED) {
    if (e.gate) {
      store(e.gate, e.gate_rs, g, Half{});
      store(e.up, e.up_rs, u, Half{});
    }
    act_run(g, e.act);
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] *= u[i];
  } else {
    if (e.bias) {
      const float b = live ? bias_at(e, f) : 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) g[i] += b;
    }
    if (e.pre) store(e.pre, e.pre_rs, g, Half{});
    act_run(g, e.act);
    if (e.res) {
      const char *q = static_cast<const char *>(e.res) +
                      (t0 * e.res_rs + f * e.res_cs) * (F32 ? 4 : 2);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i < tokens && live)
          g[i] += F32 ? *reinterpret_cast<const float *>(q)
                      : h2f(*reinterpret_cast<const uint16_t *>(q), TYPE);
        q += e.res_rs * (F32 ? 4 : 2);
      }
    }
  }
  if constexpr (F32) store(e.out[0], e.out_rs[0], g, Wide{});
  else store(e.out[0], e.out_rs[0], g, Half{});
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 2)
    skinny_kernel(const __grid_constant__ SkinnyParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t n0 = (int64_t)blockIdx.x * p.rows;
  const uint32_t full0 = smem_u32(&sh.full[0]), empty0 = smem_u32(&sh.empty[0]);
  const uint32_t done = smem_u32(&sh.done);
  const uint32_t stages = p.stages, stage_bytes = p.stage_bytes, w_bytes = p.w_bytes;
  constexpr int W = GATED ? 2 : 1;

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.done, 1);
    sh.abort = 0u;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<1>(&sh.tmem, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  griddep_launch();
  griddep_wait();

  if (warp == 0) {
    uint32_t s = 0, phase = 0;
    bool ok = true;
    const uint32_t bytes = W * (p.w_mn ? p.w_chunks * kChunk : p.rows * 128u) +
                           (p.x_mn ? p.x_chunks * kChunk : p.cols * 128u);
    // Tiles start at different k blocks and wrap around: all reading the same tokens' lines, and
    // the same columns of every weight row, at once would queue on a few slices of L2.
    int kb = (int)(blockIdx.x % (uint32_t)p.kblocks);
    for (int left = p.kblocks; left > 0; --left, kb = kb + 1 < p.kblocks ? kb + 1 : 0) {
      ok = ok && wait_bar(&sh.abort, empty0 + 8 * s, phase ^ 1u, p.status);
      if (elect_one() && ok) {
        const uint32_t bar = full0 + 8 * s, at = ring + s * stage_bytes;
        const int32_t k = kb * kTileK;
        bar_expect(bar, bytes);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          if (p.w_mn) {
            tma_box(at + w * w_bytes, &p.w[w], (int32_t)n0, k, bar);
            if (p.w_chunks > 1)
              tma_box(at + w * w_bytes + kChunk, &p.w[w], (int32_t)n0 + 64, k, bar);
          } else {
            tma_box(at + w * w_bytes, &p.w[w], k, (int32_t)n0, bar);
          }
        }
        if (p.x_mn) {
          for (int c = 0; c < p.x_chunks; ++c)
            tma_box(at + W * w_bytes + c * kChunk, &p.x, 64 * c, k, bar);
        } else {
          tma_box(at + W * w_bytes, &p.x, k, 0, bar);
        }
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    const uint32_t hi = desc_hi(1024), step = stage_bytes >> 4;
    const uint32_t as = p.w_mn ? 2048u >> 4 : 32u >> 4, bs = p.x_mn ? 2048u >> 4 : 32u >> 4;
    uint32_t a = desc_lo(ring, p.w_mn ? kChunk : 16u);
    uint32_t b = desc_lo(ring + W * w_bytes, p.x_mn ? kChunk : 16u);
    const uint32_t second = w_bytes >> 4, d2 = tmem + p.cols;
    uint32_t s = 0, phase = 0, add = 0;
    bool ok = true;
    for (int kb = 0; kb < p.kblocks; ++kb) {
      ok = ok && wait_bar(&sh.abort, full0 + 8 * s, phase, p.status);
      tc_fence_after();
      if (elect_one() && ok) {
        mma_f16<1>(tmem, a, hi, b, hi, p.idesc, add);
        if (GATED) mma_f16<1>(d2, a + second, hi, b, hi, p.idesc, add);
#pragma unroll
        for (uint32_t q = 1; q < 4; ++q) {
          mma_f16<1>(tmem, a + q * as, hi, b + q * bs, hi, p.idesc, 1);
          if (GATED) mma_f16<1>(d2, a + second + q * as, hi, b + q * bs, hi, p.idesc, 1);
        }
        mma_commit<1>(empty0 + 8 * s, 0);
      }
      __syncwarp();
      add = 1;
      a += step;
      b += step;
      if (++s == stages) {
        s = 0;
        phase ^= 1u;
        a -= stages * step;
        b -= stages * step;
      }
    }
    if (elect_one() && ok) mma_commit<1>(done, 0);
    __syncwarp();
  } else {
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const bool live = row < p.rows && n0 + row < p.n;
    if (__all_sync(~0u, wait_bar(&sh.abort, done, 0, p.status))) {
      tc_fence_after();
      const int m = (int)p.m;
      for (int t0 = 0; t0 < m; t0 += 32) {
        float g[32], u[GATED ? 32 : 1];
        tmem_load32(lanes + t0, g);
        if constexpr (GATED) tmem_load32(lanes + p.cols + t0, u);
        const int64_t f = n0 + row;
        if (p.e.type == COLL_BF16) {
          if (p.e.out_type == COLL_F32)
            finish32<GATED, COLL_BF16, !GATED>(p.e, t0, f, m - t0, live, g, u);
          else finish32<GATED, COLL_BF16, false>(p.e, t0, f, m - t0, live, g, u);
        } else {
          if (p.e.out_type == COLL_F32)
            finish32<GATED, COLL_F16, !GATED>(p.e, t0, f, m - t0, live, g, u);
          else finish32<GATED, COLL_F16, false>(p.e, t0, f, m - t0, live, g, u);
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (sh.abort) drain();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<1>(tmem, p.tmem_cols);
  }
}

template <bool GATED>
cudaError_t set_up() {
  static DenseSmemLimit limit;
  return limit((const void *)skinny_kernel<GATED>, kTcSmem);
}

template <bool GATED>
cudaError_t launch(const SkinnyParams &p, cudaStream_t s) {
  return dense_launch(skinny_kernel<GATED>, dim3(p.tiles), kThreads, p.smem, 1, s, p);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int skinny_plan(SkinnyParams &p, const DenseJob &j, const TcOperand *w, const TcOperand &x) {
  memset(&p, 0, sizeof(p));
  p.e = j.e;
  p.m = j.m;
  p.n = j.n;
  p.status = j.status;
  p.kblocks = (int32_t)ceil_div(j.k, kTileK);
  p.cols = (int32_t)ceil_div(j.m, 16) * 16;
  p.w_mn = w[0].mn;
  p.x_mn = x.mn;
  p.x_chunks = (p.cols + 63) / 64;
  const int mats = j.gated ? 2 : 1;
  // accumulators are read 32 columns at a time
  p.tmem_cols = 32;
  while ((int32_t)p.tmem_cols < p.cols * (mats - 1) + (p.cols + 31) / 32 * 32) p.tmem_cols *= 2;
  const uint32_t x_bytes = (p.x_mn ? p.x_chunks * 64u : (uint32_t)p.cols) * 128u;
  // A CTA's ring for so many features: four stages or more within what two CTAs of an SM can have,
  // else one CTA with all of it. A matrix instruction reads 128 rows whatever p.rows is, so the
  // last stage has slack behind it. Returns the CTAs an SM holds.
  auto ring = [&](int rows) {
    p.rows = rows;
    p.w_chunks = (rows + 63) / 64;
    p.w_bytes = (uint32_t)rows * 128u;
    p.stage_bytes = mats * p.w_bytes + ((x_bytes + 1023u) & ~1023u);
    const uint32_t fixed = 1024 + 16384 - p.w_bytes;
    const bool two = p.stage_bytes * 4 <= kTwoPerSm - fixed && p.tmem_cols <= 256;
    p.stages = (int32_t)(((two ? kTwoPerSm : kTcSmem) - fixed) / p.stage_bytes);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.smem = fixed + p.stages * p.stage_bytes;
    if (p.smem < kNoThird) p.smem = kNoThird;
    return two ? 2 : 1;
  };
  // Features per CTA: the least time, in ns. An SM takes 45 bytes a ns; a k block takes 190 ns to
  // issue (gated 300), a wave of CTAs 1.5 us beside its blocks.
  int64_t best = INT64_MAX;
  int best_rows = 128;
  for (int rows = 128; rows >= 32; rows -= p.w_mn ? 64 : 8) {
    const int per_sm = ring(rows);
    const int64_t tiles = ceil_div(j.n, rows), waves = ceil_div(tiles, (int64_t)kSms * per_sm);
    const int64_t beside = tiles > kSms ? per_sm : 1;
    const int64_t arrive = beside * (rows * mats * 128 + x_bytes) / 45;
    const int64_t issue = j.gated ? 300 : 190;
    const int64_t ns = waves * (p.kblocks * (arrive > issue ? arrive : issue) + 1500);
    if (ns < best) {
      best = ns;
      best_rows = rows;
    }
  }
  ring(best_rows);
  p.tiles = (uint32_t)ceil_div(j.n, p.rows);
  p.idesc = mma_desc(j.e.type == COLL_BF16, p.w_mn != 0, p.x_mn != 0, 128, (uint32_t)p.cols);
  for (int i = 0; i < mats; ++i) {
    const int c = tc_encode(&p.w[i], w[i], j.e.type, (uint32_t)p.rows);
    if (c) return c;
  }
  const int c = tc_encode(&p.x, x, j.e.type, (uint32_t)p.cols);
  if (c) return c;
  return (j.gated ? set_up<true>() : set_up<false>()) == cudaSuccess ? COLL_OK : COLL_ECUDA;
}

cudaError_t skinny_run(const SkinnyParams &p, bool gated, cudaStream_t s) {
  return gated ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace coll
