// A token or a few through their chosen experts without staging: every warp loads weights straight into
// the fragments of mma.m16n8k16, as dense_gemv.cu does for one matrix. A chunk of up to eight choices of
// one expert is the columns of a fragment, 16 rows of weights its rows (inner: eight of gate and eight
// of up, so a lane ends up with g and u of the same feature).
//
// Bound by HBM, and for small experts by latency: two launches, the chunks made by a warp of every CTA
// from the ids alone, the sums' first weights asked for while the inner values are still being made, the
// sums' CTAs all on the SMs at once (two waves of them: 24 us where one takes 19, two experts of 4096 x
// 1792). One token, six of 64 experts of 2048 x 176 (13 MB): 8.1 us, where the tensor-core kernels' cut
// tiles and joins take 21; two tokens, four of eight experts of 4096 x 14336: 182 us (6.8 TB/s) against
// 191; 16 tokens of two, eight of 4096 x 1792: 61 against 64; 32 of one, 16 of 1024 x 512 16.7 against
// 22.5. With more choices a CTA's plan takes longer and an expert's choices fill more chunks: 48 choices
// within 3 % either way, 96 of 16 experts of 7168 x 2048 224 against 219 (both before inner values had
// their rests). The warp's number comes by a shuffle, so that the compiler knows it to be the same for all
// lanes (one token: 0.3 us more without).
#include "dense_direct.cuh"
#include "dense_epi.cuh"
#include "dense_tc.h"
#include "experts.h"
#include "tma.cuh"

namespace coll {
namespace {

constexpr int kStep = 64;  // elements of a row that a warp takes at a time
constexpr int kWarps = 8;

template <int ALIGN>
constexpr int kAhead = ALIGN > 2 ? 4 : 2;

// The chunks and, by place, their choices' tokens and weights.
struct Few {
  int4 chunk[kDirectChoices];  // {expert, first place, choices, 0}
  int32_t token[8 * kDirectChoices];
  float weight[8 * kDirectChoices];
  int chunks;
};

// One warp: the chunks of at most 32 choices, by first choice; their places are eight apart.
__device__ __forceinline__ void make_chunks(const DirectParams &p, Few &few) {
  const int s = threadIdx.x & 31, n = p.tokens * p.top;
  int e = -1;
  float w = 0.0f;
  if (s < n) {
    const int i = s / p.top, j = s - i * p.top;
    const int id = static_cast<const int32_t *>(p.ids.p)[i * p.ids.rs + j * p.ids.cs];
    w = static_cast<const float *>(p.weights.p)[i * p.weights.rs + j * p.weights.cs];
    const int64_t d = (int64_t)id - p.first;
    if (id >= 0 && d >= 0 && d < p.experts) e = (int)d;
  }
  const uint32_t same = __match_any_sync(~0u, e);
  const int lead = __ffs(same) - 1, count = __popc(same);
  const int mine = e >= 0 && lead == s ? (count + 7) / 8 : 0;
  int run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, run, o);
    if (s >= o) run += v;
  }
  const int first = __shfl_sync(~0u, run - mine, lead), all = __shfl_sync(~0u, run, 31);
  if (e >= 0) {
    const int place = 8 * first + __popc(same & ((1u << s) - 1u));
    few.token[place] = s / p.top;
    few.weight[place] = w;
  }
  for (int q = 0; q < mine; ++q)
    few.chunk[first + q] = make_int4(e, 8 * (first + q), min(8, count - 8 * q), 0);
  if (s == 0) few.chunks = all;
}

// Tokens off 16 bytes come an element at a time (four tokens of two, eight experts of 4096 x 1792: 49 us,
// 42 on 16 bytes; 16 of them 76, 61; one of six, 64 of 2048 x 176 8.1, 8.1).
__device__ __forceinline__ void load_x(const DirectParams &p, const uint16_t *x, int at, int len,
                                       uint32_t (&r)[8]) {
  if (p.x_align >= 32) load16<32>(x, at, len, r);
  else if (p.x_align >= 16) load16<16>(x, at, len, r);
  else load16<2>(x, at, len, r);
}

// 16 elements of one row of each matrix, AHEAD of them asked for before the first is used.
template <int ALIGN, int AHEAD>
struct Rows {
  uint32_t a[AHEAD][8], b[AHEAD][8];
};

template <int ALIGN, int AHEAD>
__device__ __forceinline__ void load_rows(const uint16_t *const (&pa)[AHEAD],
                                          const uint16_t *const (&pb)[AHEAD],
                                          const int (&at)[AHEAD], const int (&la)[AHEAD],
                                          const int (&lb)[AHEAD], Rows<ALIGN, AHEAD> &r) {
  if constexpr (ALIGN == 2) {
    Around ra[AHEAD], rb[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      ask16(pa[i], at[i], la[i], ra[i]);
      ask16(pb[i], at[i], lb[i], rb[i]);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      take16(pa[i], at[i], la[i], ra[i], r.a[i]);
      take16(pb[i], at[i], lb[i], rb[i], r.b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      load16<ALIGN>(pa[i], at[i], la[i], r.a[i]);
      load16<ALIGN>(pb[i], at[i], lb[i], r.b[i]);
    }
  }
}

// Eight inner features of one chunk's choices at a time: gate's rows are the fragment's first eight,
// up's the others. The warps take the steps of k in turn and join in order.
template <int TYPE, int ALIGN>
__global__ void __launch_bounds__(kWarps * 32, 2)
    direct_inner_kernel(const __grid_constant__ DirectParams p) {
  constexpr int AHEAD = kAhead<ALIGN>;
  __shared__ float part[2][kWarps][8][16];
  __shared__ Few few;
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch();
  if (warp == 0) make_chunks(p, few);
  if (blockIdx.x == 0 && p.splits > 1)
    for (int i = threadIdx.x; i < p.tiles; i += blockDim.x) p.counters[i] = 0u;
  __syncthreads();
  const int tiles = (p.features + kDirectInner - 1) / kDirectInner, items = few.chunks * tiles;
  const int steps = (p.len + kStep - 1) / kStep;
  int turn = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
    const int which = item / tiles, tile = item - which * tiles;
    const int4 c = few.chunk[which];
    const int f0 = tile * kDirectInner, f = f0 + g;
    const int len = f < p.features ? p.len : 0;  // rows that are not there are empty
    const int64_t row = len ? f : 0;
    const uint16_t *wa = p.w[0] + c.x * p.es[0] + row * p.rs[0] + 16 * t;
    const uint16_t *wb = p.w[1] + c.x * p.es[1] + row * p.rs[1] + 16 * t;
    const int x_len = g < c.z ? p.len : 0;
    const uint16_t *x = p.x + (x_len ? few.token[c.y + g] : 0) * p.x_ld + 16 * t;
    float acc[4] = {};
    for (int s = warp; s < steps; s += AHEAD * warps) {
      const uint16_t *pa[AHEAD], *pb[AHEAD];
      int at[AHEAD], la[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = (s + i * warps) * kStep;
        pa[i] = wa + k, pb[i] = wb + k, at[i] = k + 16 * t, la[i] = len;
      }
      Rows<ALIGN, AHEAD> r;
      load_rows<ALIGN, AHEAD>(pa, pb, at, la, la, r);
      uint32_t xs[AHEAD][8];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) load_x(p, x + (s + i * warps) * kStep, at[i], x_len, xs[i]);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma16816<TYPE>(acc, r.a[i][2 * q], r.b[i][2 * q], r.a[i][2 * q + 1], r.b[i][2 * q + 1],
                         xs[i][2 * q], xs[i][2 * q + 1]);
    }
    float(*mine)[16] = part[turn][warp];  // the other half may still be read
    mine[2 * t][g] = acc[0];
    mine[2 * t + 1][g] = acc[1];
    mine[2 * t][g + 8] = acc[2];
    mine[2 * t + 1][g + 8] = acc[3];
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * c.z; i += blockDim.x) {
      const int n = i / 8, j = i % 8;
      if (f0 + j >= p.features) continue;
      float v = 0.0f, u = 0.0f;
      for (int w = 0; w < warps; ++w) {
        v += part[turn][w][n][j];
        u += part[turn][w][n][j + 8];
      }
      uint16_t *h = p.h + (int64_t)(c.y + n) * p.h_ld + f0 + j;
      split_value(act_value(v, p.act) * u, TYPE, h[0], h[p.rest]);
    }
    // the sums read rows in whole runs of 16
    if (tile == tiles - 1)
      for (int i = threadIdx.x; i < 16 * c.z; i += blockDim.x) {
        const int j = p.features + i % 16;
        uint16_t *h = p.h + (int64_t)(c.y + i / 16) * p.h_ld + j;
        if (j < ((p.features + 15) & ~15)) h[0] = h[p.rest] = 0;
      }
  }
}

// 16 outputs of all tokens. The steps of all chunks are one list, the splits' shares of it
// neighbouring, and inside a share the warps take steps in turn; each adds its finished products,
// times their weights, to its own sums in shared memory. The warps join in order, and so do the
// splits, in the last of their CTAs to arrive.
//
// Up to four choices' inner values and their rests are the eight columns of one fragment. More choices
// take a second fragment for the rests; there are registers for two steps of both at a time.
template <int TYPE, int ALIGN>
__global__ void __launch_bounds__(kWarps * 32, 2)
    direct_outer_kernel(const __grid_constant__ DirectParams p) {
  constexpr int AHEAD = kAhead<ALIGN>;
  __shared__ float sums[kWarps][kDirectTokens * 16];
  __shared__ Few few;
  __shared__ uint32_t last;
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, t = lane & 3, size = p.tokens * 16;
  griddep_launch();
  float *mine = sums[warp];
  for (int i = lane; i < size; i += 32) mine[i] = 0.0f;
  // The inner kernel lets this one start after its own wait, so what that waited for (the choices,
  // the weights) is there; its inner values are not before the wait below.
  if (warp == 0) make_chunks(p, few);
  __syncthreads();
  const int n0 = (int)blockIdx.x * kDirectOuter;
  const int la = n0 + g < p.features ? p.len : 0, lb = n0 + g + 8 < p.features ? p.len : 0;
  const uint16_t *wa = p.w[0] + (int64_t)(la ? n0 + g : 0) * p.rs[0] + 16 * t;
  const uint16_t *wb = p.w[0] + (int64_t)(lb ? n0 + g + 8 : 0) * p.rs[0] + 16 * t;
  const uint16_t *h = p.x + 16 * t;
  const int steps = (p.len + kStep - 1) / kStep;
  const int64_t all = (int64_t)few.chunks * steps;
  const int64_t lo = all * blockIdx.y / p.splits, hi = all * (blockIdx.y + 1) / p.splits;
  float acc[4] = {};
  int now = -1;
  // what the accumulators hold of chunk `now` goes to its tokens; of two columns of one token, one
  // after the other
  auto flush = [&]() {
    const int4 c = few.chunk[now];
    if (c.z <= 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor_sync(~0u, acc[j], 2);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (t == q) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (2 * t + j < c.z) {
            float *y = mine + few.token[c.y + 2 * t + j] * 16 + g;
            const float w = few.weight[c.y + 2 * t + j];
            y[0] = fmaf(w, acc[j], y[0]);
            y[8] = fmaf(w, acc[j + 2], y[8]);
          }
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = 0.0f;
  };
  int64_t s = lo + warp;
  int at_chunk = (int)(s / steps), at_step = (int)(s - (int64_t)at_chunk * steps);
  while (s < hi) {
    const uint16_t *pa[AHEAD], *pb[AHEAD], *x[AHEAD];
    int at[AHEAD], ka[AHEAD], kb[AHEAD], which[AHEAD], x_len[AHEAD];
    uint32_t apart = 0;  // steps whose rests are a fragment of their own
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const bool there = s < hi;
      which[i] = there ? at_chunk : -1;
      const int4 c = there ? few.chunk[at_chunk] : make_int4(0, 0, 0, 0);
      const int k = at_step * kStep;
      pa[i] = wa + c.x * p.es[0] + k;
      pb[i] = wb + c.x * p.es[0] + k;
      at[i] = k + 16 * t;
      ka[i] = there ? la : 0;
      kb[i] = there ? lb : 0;
      const int choice = c.z <= 4 ? g & 3 : g;
      x_len[i] = choice < c.z ? p.len : 0;
      x[i] = h + (int64_t)(choice < c.z ? c.y + choice : 0) * p.x_ld + k;
      if (c.z > 4) apart |= 1u << i;
      else if (g >= 4) x[i] += p.rest;
      s += warps;
      at_step += warps;
      while (at_step >= steps) {
        at_step -= steps;
        ++at_chunk;
      }
    }
    Rows<ALIGN, AHEAD> r;
    load_rows<ALIGN, AHEAD>(pa, pb, at, ka, kb, r);
    griddep_wait();
    uint32_t xs[AHEAD][8];
    auto begin = [&](int i) {
      if (which[i] == now) return;
      if (now >= 0) flush();
      now = which[i];
    };
    auto product = [&](int i, const uint32_t (&b)[8]) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mma16816<TYPE>(acc, r.a[i][2 * q], r.b[i][2 * q], r.a[i][2 * q + 1], r.b[i][2 * q + 1],
                       b[2 * q], b[2 * q + 1]);
    };
    if (apart == 0) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) load16<32>(x[i], at[i], x_len[i], xs[i]);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (which[i] < 0) break;
        begin(i);
        product(i, xs[i]);
      }
    } else {
      constexpr int HALF = AHEAD / 2;
#pragma unroll
      for (int i0 = 0; i0 < AHEAD; i0 += HALF) {
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
          const int i = i0 + j;
          load16<32>(x[i], at[i], x_len[i], xs[j]);
          load16<32>(x[i] + p.rest, at[i], apart >> i & 1u ? x_len[i] : 0, xs[HALF + j]);
        }
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
          const int i = i0 + j;
          if (which[i] < 0) break;
          begin(i);
          product(i, xs[j]);
          if (apart >> i & 1u) product(i, xs[HALF + j]);
        }
      }
    }
  }
  if (now >= 0) flush();
  griddep_wait();  // also where nothing was to be done
  __syncthreads();
  auto finish = [&](int i, float v) {
    const int tok = i / 16, f = n0 + i % 16;
    if (f >= p.features) return;
    if (p.res.p) v += ld_elem(p.res.p, tok * p.res.rs + f * p.res.cs, p.out_type);
    st_elem(p.y, tok * p.y_rs + f, v, p.out_type);
  };
  const int64_t share = (int64_t)gridDim.x * size;
  float *part = p.part + (int64_t)blockIdx.x * size;
  for (int i = threadIdx.x; i < size; i += blockDim.x) {
    float v = 0.0f;
    for (int w = 0; w < warps; ++w) v += sums[w][i];
    if (p.splits == 1) finish(i, v);
    else __stcg(part + blockIdx.y * share + i, v);
  }
  if (p.splits == 1) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    last = atomicAdd(&p.counters[blockIdx.x], 1u) == (uint32_t)p.splits - 1u;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int i = threadIdx.x; i < size; i += blockDim.x) {
    float v = 0.0f;
#pragma unroll 8
    for (int w = 0; w < p.splits; ++w) v += __ldcg(part + w * share + i);
    finish(i, v);
  }
}

// Rows on 4 bytes by eight 4-byte loads a fragment, four steps ahead; through the words around them, as rows
// on 2 bytes, two ahead (one token, 6 of 64 experts of 2050 x 178: 10.8 us, 14.1 so; two of eight of 4098 x
// 1790 31.6, 34.3, of 4098 x 14338 173, 185; four tokens of the former 67.7, 71.4, 16 of them 107, 105).
using Kernel = void (*)(const DirectParams);
template <bool INNER, int TYPE>
Kernel pick(int align) {
#define COLL_DIRECT(A) \
  return INNER ? (Kernel)direct_inner_kernel<TYPE, A> : (Kernel)direct_outer_kernel<TYPE, A>
  if (align >= 32) COLL_DIRECT(32);
  if (align >= 16) COLL_DIRECT(16);
  if (align >= 4) COLL_DIRECT(4);
  COLL_DIRECT(2);
#undef COLL_DIRECT
}

}  // namespace

cudaError_t experts_direct_inner(const DirectParams &p, int align, cudaStream_t s) {
  const Kernel k = p.type == COLL_BF16 ? pick<true, COLL_BF16>(align) : pick<true, COLL_F16>(align);
  const int64_t items =
      (int64_t)((p.features + kDirectInner - 1) / kDirectInner) * p.most_chunks;
  const int64_t most = kSms * (16 / p.warps);  // as many as are on the SMs at once
  return dense_launch(k, dim3((unsigned)(items < most ? items : most)), 32 * p.warps, 0, 1, s, p);
}

cudaError_t experts_direct_outer(const DirectParams &p, int align, cudaStream_t s) {
  const Kernel k =
      p.type == COLL_BF16 ? pick<false, COLL_BF16>(align) : pick<false, COLL_F16>(align);
  return dense_launch(k, dim3(p.tiles, p.splits), 32 * p.warps, 0, 1, s, p);
}

}  // namespace coll
