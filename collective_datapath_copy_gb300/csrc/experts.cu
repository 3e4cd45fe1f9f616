// A few tokens through their chosen gated experts: C ABI (include/coll.h) and kernels.
//
//   h_ij = act(gate_e x_i) (up_e x_i),  y_i = residual_i + sum over j of weights_ij down_e h_ij,
//   e = ids_ij - first
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense.h"
#include "dense_check.h"
#include "dense_epi.cuh"
#include "tma.cuh"

namespace coll {
namespace {

constexpr int kMostExperts = 1024;
constexpr int kMostChosen = 32;
constexpr int kWarps = 8;

struct ExpertsParams {
  const uint16_t *gate, *up, *down;
  int64_t gate_es, gate_rs, up_es, up_rs, down_es, down_rs;
  DenseMat x, ids, weights, res;
  void *y;
  int64_t y_rs;
  uint16_t *h;  // [m * top][f]
  int64_t m, n, k, f;
  int32_t experts, first, top, type, out_type, act;
};

__device__ __forceinline__ int local_id(const ExpertsParams &p, int64_t i, int j) {
  const int id = static_cast<const int32_t *>(p.ids.p)[i * p.ids.rs + j * p.ids.cs];
  const int64_t e = (int64_t)id - p.first;
  return id >= 0 && e >= 0 && e < p.experts ? (int)e : -1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// A warp for each inner feature of each (token, choice).
__global__ void __launch_bounds__(kWarps * 32) inner_kernel(const ExpertsParams p) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t all = p.m * p.top * p.f;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); w < all;
       w += (int64_t)gridDim.x * kWarps) {
    const int64_t slot = w / p.f, f = w % p.f, i = slot / p.top;
    const int e = local_id(p, i, (int)(slot % p.top));
    if (e < 0) continue;
    const uint16_t *x = static_cast<const uint16_t *>(p.x.p) + i * p.x.rs;
    const uint16_t *a = p.gate + e * p.gate_es + f * p.gate_rs;
    const uint16_t *b = p.up + e * p.up_es + f * p.up_rs;
    float g = 0.0f, u = 0.0f;
    for (int64_t k = lane; k < p.k; k += 32) {
      const float v = h2f(x[k * p.x.cs], p.type);
      g = fmaf(v, h2f(a[k], p.type), g);
      u = fmaf(v, h2f(b[k], p.type), u);
    }
    g = warp_sum(g);
    u = warp_sum(u);
    if (lane == 0) p.h[slot * p.f + f] = f2h(act_value(g, p.act) * u, p.type);
  }
}

// A warp for each output.
__global__ void __launch_bounds__(kWarps * 32) outer_kernel(const ExpertsParams p) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t all = p.m * p.n;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); w < all;
       w += (int64_t)gridDim.x * kWarps) {
    const int64_t i = w / p.n, n = w % p.n;
    float y = p.res.p ? ld_elem(p.res.p, i * p.res.rs + n * p.res.cs, p.out_type) : 0.0f;
    for (int j = 0; j < p.top; ++j) {
      const int e = local_id(p, i, j);
      if (e < 0) continue;
      const uint16_t *h = p.h + (i * p.top + j) * p.f;
      const uint16_t *a = p.down + e * p.down_es + n * p.down_rs;
      float d = 0.0f;
      for (int64_t f = lane; f < p.f; f += 32)
        d = fmaf(h2f(h[f], p.type), h2f(a[f], p.type), d);
      d = warp_sum(d);
      y = fmaf(static_cast<const float *>(p.weights.p)[i * p.weights.rs + j * p.weights.cs], d, y);
    }
    if (lane == 0) st_elem(p.y, i * p.y_rs + n, y, p.out_type);
  }
}

int check_stack(const coll_stack_t &w, int64_t e, int64_t rows, int64_t cols, View &v) {
  const int64_t lim = (int64_t)kAddressable;
  v = View{w.ptr, 0, 0, 0, 1, 2};
  if (rows == 0 || cols == 0) return COLL_OK;
  if (!w.ptr || w.es < 0 || w.rs < 0) return COLL_EINVAL;
  if ((uintptr_t)w.ptr & 1u) return COLL_EALIGN;
  if ((e > 1 && w.es > lim / (e - 1)) || (rows > 1 && w.rs > lim / (rows - 1))) return COLL_EINVAL;
  // its extent, as e rows
  v.rows = e;
  v.rs = w.es;
  v.cols = (rows - 1) * w.rs + cols;
  return COLL_OK;
}

int check(const coll_experts_t &a) {
  const int64_t most = 0x7FFFFFFF - 4096;
  for (int64_t v : {a.m, a.n, a.k, a.f})
    if (v < 0 || v > most) return COLL_EINVAL;
  if (!is_half(a.dtype) || (a.out_dtype != a.dtype && a.out_dtype != COLL_F32)) return COLL_EINVAL;
  if (a.act < COLL_ACT_RELU || a.act > COLL_ACT_SIGMOID) return COLL_EINVAL;
  if (a.experts < 1 || a.experts > kMostExperts || a.top < 1 || a.top > kMostChosen ||
      a.first < 0 || a.first > most)
    return COLL_EINVAL;
  const int oe = esize(a.out_dtype);
  Check k;
  k.output(view(a.y, a.m, a.n, oe));
  k.input(view(a.x, a.m, a.k, 2));
  k.input(view(a.ids, a.m, a.top, 4));
  k.input(view(a.weights, a.m, a.top, 4));
  const int res = k.input(view(a.residual, a.m, a.n, oe), false);
  if (k.code) return k.code;
  View v;
  int c = check_stack(a.w_gate, a.experts, a.f, a.k, v);
  if (!c) k.in[k.n_in++] = v, c = check_stack(a.w_up, a.experts, a.f, a.k, v);
  if (!c) k.in[k.n_in++] = v, c = check_stack(a.w_down, a.experts, a.n, a.f, v);
  if (c) return c;
  k.in[k.n_in++] = v;
  if ((uintptr_t)a.status % sizeof(int32_t)) return COLL_EALIGN;
  return k.finish(res);
}

int64_t need(const coll_experts_t &a) {
  if (a.m == 0 || a.n == 0) return 0;
  const uint64_t slots = (uint64_t)(a.m * a.top);
  if (a.f && slots > kAddressable / 2 / (uint64_t)a.f) return COLL_EINVAL;
  return (int64_t)(slots * a.f * 2 + 128);
}

int run(const coll_experts_t &a, cudaStream_t s) {
  ExpertsParams p = {};
  p.gate = static_cast<const uint16_t *>(a.w_gate.ptr);
  p.up = static_cast<const uint16_t *>(a.w_up.ptr);
  p.down = static_cast<const uint16_t *>(a.w_down.ptr);
  p.gate_es = a.w_gate.es, p.gate_rs = a.w_gate.rs;
  p.up_es = a.w_up.es, p.up_rs = a.w_up.rs;
  p.down_es = a.w_down.es, p.down_rs = a.w_down.rs;
  p.x = DenseMat{a.x.ptr, a.x.rs, a.x.cs};
  p.ids = DenseMat{a.ids.ptr, a.ids.rs, a.ids.cs};
  p.weights = DenseMat{a.weights.ptr, a.weights.rs, a.weights.cs};
  p.res = DenseMat{a.residual.ptr, a.residual.rs, a.residual.cs};
  p.y = a.y.ptr;
  p.y_rs = a.y.rs;
  p.h = reinterpret_cast<uint16_t *>(((uintptr_t)a.workspace + 127) & ~(uintptr_t)127);
  p.m = a.m, p.n = a.n, p.k = a.k, p.f = a.f;
  p.experts = (int32_t)a.experts;
  p.first = (int32_t)a.first;
  p.top = (int32_t)a.top;
  p.type = (int32_t)a.dtype;
  p.out_type = (int32_t)a.out_dtype;
  p.act = (int32_t)a.act;
  const dim3 grid(152 * 8);
  cudaError_t e = cudaSuccess;
  if (a.f > 0) e = dense_launch(inner_kernel, grid, kWarps * 32, 0, 1, s, p);
  if (e == cudaSuccess) e = dense_launch(outer_kernel, grid, kWarps * 32, 0, 1, s, p);
  return e == cudaSuccess ? COLL_OK : COLL_ECUDA;
}

}  // namespace
}  // namespace coll

extern "C" int64_t coll_gated_experts_workspace(const coll_experts_t *a) {
  if (!a) return COLL_EINVAL;
  const int c = coll::check(*a);
  return c ? c : coll::need(*a);
}

extern "C" int coll_gated_experts(const coll_experts_t *a, void *stream) {
  const int64_t n = coll_gated_experts_workspace(a);
  if (n < 0) return (int)n;
  if (a->m == 0 || a->n == 0) return COLL_OK;
  if (n && (!a->workspace || ((uintptr_t)a->workspace & 15u) ||
            a->workspace_bytes < (uint64_t)n))
    return COLL_EWORKSPACE;
  return coll::run(*a, static_cast<cudaStream_t>(stream));
}
