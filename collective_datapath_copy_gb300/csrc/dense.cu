// C ABI of the dense operators (include/coll.h): argument checks, workspace layout, and which
// kernels a call launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense.h"
#include "dense_check.h"
#include "dense_tc.h"

namespace {

using coll::Check;
using coll::DenseActBwd;
using coll::DenseJob;
using coll::DenseMat;
using coll::TcOperand;
using coll::View;
using coll::esize;
using coll::is_half;
using coll::kAddressable;
using coll::view;

// Bump allocator over the caller's workspace, in steps of 256 bytes from a 128-byte boundary. With
// base == nullptr it only counts.
struct Ws {
  char *base;
  uint64_t used;
  // shapes of the tensor-core launch: the counting pass leaves them for the launching one
  coll::TcParams *plan;
  bool planned;
  uint64_t part[2];
  bool over;  // more was asked for than a device can address; the counting pass ends the call then
  void *take(uint64_t bytes) {
    if (bytes > kAddressable - used) {
      over = true;
      return nullptr;
    }
    const uint64_t at = used;
    used += (bytes + 255) & ~(uint64_t)255;
    return base ? base + at : nullptr;
  }
};

int64_t round8(int64_t v) { return (v + 7) & ~(int64_t)7; }

// Lines of what the workspace holds start on 128 bytes: a tensor copy's 128-byte rows then lie in
// one line each (512 x 1024 x 5462: 23.4 us with lines of 5464 elements, 15.8 with 5504).
int64_t round64(int64_t v) { return (v + 63) & ~(int64_t)63; }

int check_sizes(int64_t m, int64_t n, int64_t k, int64_t dtype) {
  const int64_t most = 0x7FFFFFFF - 4096;
  if (m < 0 || n < 0 || k < 0 || m > most || n > most || k > most) return COLL_EINVAL;
  return is_half(dtype) ? COLL_OK : COLL_EINVAL;
}

bool linear_act(int64_t a) { return a >= COLL_ACT_NONE && a <= COLL_ACT_SILU; }
bool gated_act(int64_t a) { return a >= COLL_ACT_RELU && a <= COLL_ACT_SIGMOID; }

DenseMat mat(const coll_mat_t &m) { return DenseMat{m.ptr, m.rs, m.cs}; }
DenseMat turned(const coll_mat_t &m) { return DenseMat{m.ptr, m.cs, m.rs}; }

// Bits of the addresses of a matrix's rows (all rows start on 16 bytes if no bit below 16 is set).
uint64_t sectors(const void *p, int64_t rs, int es) {
  return p ? (uintptr_t)p | (uint64_t)(rs * es) : 0;
}

// Do rows start on 16 bytes in every array of the epilogue?
void set_vec(DenseJob &j) {
  const coll::DenseEpi &e = j.e;
  const int oe = esize(e.out_type);
  uint64_t v = 0;
  for (int b = 0; b < j.nbatch; ++b) v |= sectors(e.out[b], e.out_rs[b], oe);
  v |= sectors(e.pre, e.pre_rs, 2) | sectors(e.gate, e.gate_rs, 2) | sectors(e.up, e.up_rs, 2) |
       sectors(e.bias, 0, 2) | sectors(e.res, e.res_rs, oe);
  const bool unit = (!e.bias || e.bias_stride == 1) && (!e.res || e.res_cs == 1);
  j.e.vec = unit && v % 16 == 0;
}

DenseJob job(int64_t m, int64_t n, int64_t k, int64_t type, int32_t *status) {
  DenseJob j = {};
  j.m = m;
  j.n = n;
  j.k = k;
  j.nseg = j.nbatch = 1;
  j.e.type = j.e.out_type = (int32_t)type;
  j.status = status;
  return j;
}

void set_out(DenseJob &j, int b, const coll_mat_t &o) {
  j.e.out[b] = o.ptr;
  j.e.out_rs[b] = o.rs;
}

// The operand as a tensor map takes it in place: one unit stride, the other a multiple of 16
// bytes that is no shorter than the line, a 16-byte aligned base. False where it has to be
// laid out first.
bool in_place(const DenseMat &m, int64_t rows, int64_t k, TcOperand &o) {
  const int64_t most = (int64_t)1 << 38;  // the maps' strides are below 2^40 bytes
  if ((uintptr_t)m.p & 15u) return false;
  const bool along_k = m.cs == 1 || k == 1, along_m = m.rs == 1 || rows == 1;
  if (along_k && (rows == 1 || (m.rs % 8 == 0 && m.rs >= k && m.rs < most))) {
    o = TcOperand{m.p, rows, k, rows == 1 ? round8(k) : m.rs, 0};
    return true;
  }
  if (along_m && (k == 1 || (m.cs % 8 == 0 && m.cs >= rows && m.cs < most))) {
    o = TcOperand{m.p, rows, k, k == 1 ? round8(rows) : m.cs, 1};
    return true;
  }
  return false;
}

// Put the operand on the list of those to lay out in the workspace, along `mn` (0: k, 1: rows).
void lay_out(const DenseMat &m, int64_t rows, int64_t k, int mn, Ws &ws, coll::DensePack &todo,
             TcOperand &o) {
  const int i = todo.count++;
  todo.src[i] = mn ? DenseMat{m.p, m.cs, m.rs} : m;
  todo.rows[i] = mn ? k : rows;
  todo.cols[i] = mn ? rows : k;
  todo.ld[i] = round64(todo.cols[i]);
  todo.dst[i] = static_cast<uint16_t *>(ws.take((uint64_t)todo.rows[i] * todo.ld[i] * 2));
  o = TcOperand{todo.dst[i], rows, k, todo.ld[i], mn};
}

void operand(const DenseMat &m, int64_t rows, int64_t k, Ws &ws, coll::DensePack &todo,
             TcOperand &o) {
  if (!in_place(m, rows, k, o)) lay_out(m, rows, k, m.cs != 1 && m.rs == 1, ws, todo, o);
}

// Products that the direct kernel takes: few tokens, everything contiguous along k. It reads the
// tokens again for every 16 outputs, so the more tokens, the sooner that traffic outweighs what it
// saves (no staging, no tensor maps). Up to 16 tokens always (14336 x 4096: 23 us, the next best
// 23). Up to 32 for weights of 32 MiB or less (4096 x 1792 for 32 tokens: 6.7 us against 8.7;
// 6144 x 4096: 20 us against 15) or operands that would have to be laid out first; up to 64 for
// 4 MiB or less (1024 x 1024 for 48: 4.0 us against 4.9; 1792 x 4096: 11.5 against 8.1).
// Whatever the batch, not where the sums are long and the outputs few: a warp's turns through k, at
// the time a turn was measured to take, against the tensor-core launch, its bytes and laying out
// (512 x 12288 for 32 tokens: 13.8 us against 10.0; 76 x 12289: 24 against 11, for one token 16
// against 11).
bool few_tokens(const DenseJob &j) {
  auto along_k = [&](const DenseMat &m) { return m.cs == 1 || j.k == 1; };
  if (!j.forward || j.m > coll::kGemvMost || j.k > (int64_t)1 << 30 || !along_k(j.a[0]) ||
      !along_k(j.b[0]) || (j.gated && !along_k(j.b[1])))
    return false;
  const int64_t bytes = j.n * j.k * (j.gated ? 4 : 2);
  TcOperand o;
  const bool as_it_lies = in_place(j.a[0], j.m, j.k, o) && in_place(j.b[0], j.n, j.k, o) &&
                          (!j.gated || in_place(j.b[1], j.n, j.k, o));
  const int64_t columns = j.m <= 8 ? 1 : j.m <= 16 ? 2 : 4;  // of eight tokens, at most four
  const int64_t turn = as_it_lies ? 100 + 150 * columns : 900 + 300 * columns;  // ns
  const int64_t ns = j.k * turn / (j.m <= 32 ? 1024 : 512);
  if (ns > (as_it_lies ? 4500 + bytes / 5500 : 8000 + bytes / 1850)) return false;
  return j.m <= 16 || (j.m <= 32 && (!as_it_lies || bytes <= (int64_t)32 << 20)) ||
         bytes <= (int64_t)4 << 20;
}

// The same with the weights' rows contiguous: up to 16 tokens and sums short enough that the warps
// of a CTA walk them in a few turns (16 tokens, 1024 x 1024: 3.8 us against 5.8, 4096 x 1792: 7.3
// against 13; 512 x 8192: 19 us against 8).
bool few_tokens_turned(const DenseJob &j) {
  if (!j.forward || j.m > coll::kGemvTMost || j.k * (j.gated ? 2 : 1) > 2048) return false;
  auto along_n = [&](const DenseMat &m) { return m.rs == 1 || j.n == 1; };
  return (j.a[0].cs == 1 || j.k == 1) && along_n(j.b[0]) && (!j.gated || along_n(j.b[1]));
}

// The job through a kernel that takes its operands as they lie.
enum Direct { kNotDirect, kEmptySum, kGemv, kGemvTurned };

cudaError_t run_direct(const DenseJob &j, Direct how, cudaStream_t s) {
  return how == kEmptySum ? coll::dense_empty_sum(j, s)
         : how == kGemv   ? coll::gemv_run(j, s)
                          : coll::gemv_t_run(j, s);
}

// One product, or two independent ones, after the elementwise step `act`, if there is one; only
// counts their workspace where `dry`. Column sums that the step leaves to be added are taken along
// by the launch of the products. Nothing is launched before all that may be refused has been asked
// for: shapes, tensor maps, shared memory.
int products(DenseJob *jobs, int count, Ws &ws, bool dry, cudaStream_t s,
             const DenseActBwd *act = nullptr) {
  coll::TcJob todo[2];
  Direct direct[2] = {};
  coll::DensePack pack = {};
  int n = 0;
  for (int i = 0; i < count; ++i) {
    DenseJob &j = jobs[i];
    if (j.m == 0 || j.n == 0) continue;
    set_vec(j);
    direct[i] = j.k == 0               ? kEmptySum
                : few_tokens(j)        ? kGemv
                : few_tokens_turned(j) ? kGemvTurned
                                       : kNotDirect;
    if (direct[i]) continue;
    coll::TcJob &t = todo[n++];
    t.j = &j;
    const int na = j.nbatch == 2 || j.nseg == 2 ? 2 : 1, nb = j.gated || j.nseg == 2 ? 2 : 1;
    for (int x = 0; x < na; ++x) operand(j.a[x], j.m, j.k, ws, pack, t.a[x]);
    operand(j.b[0], j.n, j.k, ws, pack, t.b[0]);
    // both halves of a gated product's instruction lie the same way, and so do both batches'
    // first operands (they are scratch)
    if (nb == 2 && (!in_place(j.b[1], j.n, j.k, t.b[1]) || (j.gated && t.b[1].mn != t.b[0].mn)))
      lay_out(j.b[1], j.n, j.k, j.gated ? t.b[0].mn : j.b[1].cs != 1 && j.b[1].rs == 1, ws, pack,
              t.b[1]);
  }
  const bool skinny = n == 1 && todo[0].j->forward && todo[0].j->m <= coll::kSkinnyMost &&
                      todo[0].j->n >= coll::kSkinnyLeast;
  coll::TcParams &p = *ws.plan;
  if (n && !skinny) {
    if (!ws.planned) {
      const int c = coll::tc_plan(p, todo, n, ws.part);
      if (c) return c;
      ws.planned = true;
    }
    for (int i = 0; i < n; ++i)
      if (ws.part[i]) p.prob[i].part = static_cast<float *>(ws.take(ws.part[i]));
  }
  if (dry) return COLL_OK;
  coll::SkinnyParams q;
  if (n) {
    const int c = skinny ? coll::skinny_plan(q, *todo[0].j, todo[0].b, todo[0].a[0])
                         : coll::tc_prepare(p, todo, n);
    if (c) return c;
  }
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < count && e == cudaSuccess; ++i)
    if (direct[i]) e = run_direct(jobs[i], direct[i], s);
  coll::DenseJoin join = {};
  if (e == cudaSuccess && act) e = coll::dense_act_bwd(*act, pack, join, s);
  else if (e == cudaSuccess && pack.count) e = coll::dense_pack(pack, s);
  if (e == cudaSuccess) {
    p.join = join;
    if (skinny) e = coll::skinny_run(q, todo[0].j->gated != 0, s);
    else if (n) e = coll::tc_run(p, todo, n, s);
    else if (join.db) e = coll::dense_join(join, s);
  }
  return e == cudaSuccess ? COLL_OK : COLL_ECUDA;
}

// Scratch matrices.
coll_mat_t scratch(Ws &ws, int64_t rows, int64_t cols) {
  const int64_t ld = round64(cols);
  return coll_mat_t{ws.take((uint64_t)rows * ld * 2), ld, 1};
}

// ---- y = act(x w^T + bias) + residual

int check(const coll_linear_t &a) {
  int c = check_sizes(a.m, a.n, a.k, a.dtype);
  if (c) return c;
  if (!linear_act(a.act) || (a.out_dtype != a.dtype && a.out_dtype != COLL_F32))
    return COLL_EINVAL;
  const int oe = esize(a.out_dtype);
  Check k;
  k.output(view(a.y, a.m, a.n, oe));
  k.output(view(a.pre, a.m, a.n, 2), false);
  k.input(view(a.x, a.m, a.k, 2));
  k.input(view(a.w, a.n, a.k, 2));
  const int res = k.input(view(a.residual, a.m, a.n, oe), false);
  k.input(View{a.bias, 1, a.n, 0, a.bias_stride, 2}, false);
  return k.finish(res);
}

int run(const coll_linear_t &a, Ws &ws, bool dry, cudaStream_t s) {
  DenseJob j = job(a.m, a.n, a.k, a.dtype, a.status);
  j.forward = 1;
  j.a[0] = mat(a.x);
  j.b[0] = mat(a.w);
  j.e.out_type = (int32_t)a.out_dtype;
  j.e.act = (int32_t)a.act;
  set_out(j, 0, a.y);
  j.e.pre = a.pre.ptr;
  j.e.pre_rs = a.pre.rs;
  j.e.bias = a.bias;
  j.e.bias_stride = a.bias_stride;
  j.e.res = a.residual.ptr;
  j.e.res_rs = a.residual.rs;
  j.e.res_cs = a.residual.cs;
  return products(&j, 1, ws, dry, s);
}

// ---- its gradients

int check(const coll_linear_bwd_t &a) {
  int c = check_sizes(a.m, a.n, a.k, a.dtype);
  if (c) return c;
  if (!linear_act(a.act) || (a.grad_dtype != a.dtype && a.grad_dtype != COLL_F32))
    return COLL_EINVAL;
  const int ge = esize(a.grad_dtype);
  Check k;
  k.output(view(a.dx, a.m, a.k, 2), false);
  k.output(view(a.dw, a.n, a.k, ge), false);
  k.output(View{a.db, 1, a.n, a.n, 1, ge}, false);
  k.input(view(a.dy, a.m, a.n, 2));
  k.input(view(a.pre, a.m, a.n, 2), a.act != COLL_ACT_NONE);
  k.input(view(a.x, a.m, a.k, 2), a.dw.ptr != nullptr);
  k.input(view(a.w, a.n, a.k, 2), a.dx.ptr != nullptr);
  return k.finish();
}

int run(const coll_linear_bwd_t &a, Ws &ws, bool dry, cudaStream_t s) {
  const bool wanted = a.dx.ptr || a.dw.ptr;
  coll_mat_t dz = a.dy;
  DenseActBwd b = {};
  b.m = a.m;
  b.n = a.n;
  b.dy = mat(a.dy);
  b.type = (int32_t)a.dtype;
  b.db_type = (int32_t)a.grad_dtype;
  b.act = (int32_t)a.act;
  if (a.act != COLL_ACT_NONE) b.pre = mat(a.pre);
  TcOperand o;
  if (wanted && (a.act != COLL_ACT_NONE || !in_place(mat(a.dy), a.m, a.n, o))) {
    dz = scratch(ws, a.m, a.n);  // both products read it
    b.dz = dz.ptr;
    b.ld = dz.rs;
  }
  if (a.db) {
    b.db = a.db;
    const int64_t blocks = coll::dense_act_bwd_row_blocks(a.m, a.n, true);
    if (blocks > 1) b.part = static_cast<float *>(ws.take((uint64_t)blocks * a.n * 4));
  }
  const bool step = (a.db || (b.dz && a.m > 0)) && a.n > 0;
  DenseJob jobs[2];
  int n = 0;
  if (a.dx.ptr) {  // dx(m, k) = sum over n of dz(m, n) w(n, k)
    DenseJob &j = jobs[n++];
    j = job(a.m, a.k, a.n, a.dtype, a.status);
    j.a[0] = mat(dz);
    j.b[0] = turned(a.w);
    set_out(j, 0, a.dx);
  }
  if (a.dw.ptr) {  // dw(n, k) = sum over m of dz(m, n) x(m, k)
    DenseJob &j = jobs[n++];
    j = job(a.n, a.k, a.m, a.dtype, a.status);
    j.a[0] = turned(dz);
    j.b[0] = turned(a.x);
    j.e.out_type = (int32_t)a.grad_dtype;
    set_out(j, 0, a.dw);
  }
  return products(jobs, n, ws, dry, s, step ? &b : nullptr);
}

// ---- h = act(x w_gate^T) (x w_up^T)

int check(const coll_gated_t &a) {
  int c = check_sizes(a.m, a.n, a.k, a.dtype);
  if (c) return c;
  if (!gated_act(a.act) || (a.gate.ptr == nullptr) != (a.up.ptr == nullptr)) return COLL_EINVAL;
  Check k;
  k.output(view(a.h, a.m, a.n, 2));
  k.output(view(a.gate, a.m, a.n, 2), false);
  k.output(view(a.up, a.m, a.n, 2), false);
  k.input(view(a.x, a.m, a.k, 2));
  k.input(view(a.w_gate, a.n, a.k, 2));
  k.input(view(a.w_up, a.n, a.k, 2));
  return k.finish();
}

int run(const coll_gated_t &a, Ws &ws, bool dry, cudaStream_t s) {
  DenseJob j = job(a.m, a.n, a.k, a.dtype, a.status);
  j.forward = j.gated = 1;
  j.a[0] = mat(a.x);
  j.b[0] = mat(a.w_gate);
  j.b[1] = mat(a.w_up);
  j.e.act = (int32_t)a.act;
  set_out(j, 0, a.h);
  j.e.gate = a.gate.ptr;
  j.e.gate_rs = a.gate.rs;
  j.e.up = a.up.ptr;
  j.e.up_rs = a.up.rs;
  return products(&j, 1, ws, dry, s);
}

// ---- its gradients

int check(const coll_gated_bwd_t &a) {
  int c = check_sizes(a.m, a.n, a.k, a.dtype);
  if (c) return c;
  if (!gated_act(a.act) || (a.grad_dtype != a.dtype && a.grad_dtype != COLL_F32) ||
      (a.dw_gate.ptr == nullptr) != (a.dw_up.ptr == nullptr))
    return COLL_EINVAL;
  const int ge = esize(a.grad_dtype);
  Check k;
  k.output(view(a.dx, a.m, a.k, 2), false);
  k.output(view(a.dw_gate, a.n, a.k, ge), false);
  k.output(view(a.dw_up, a.n, a.k, ge), false);
  k.input(view(a.dh, a.m, a.n, 2));
  k.input(view(a.gate, a.m, a.n, 2));
  k.input(view(a.up, a.m, a.n, 2));
  k.input(view(a.x, a.m, a.k, 2), a.dw_gate.ptr != nullptr);
  k.input(view(a.w_gate, a.n, a.k, 2), a.dx.ptr != nullptr);
  k.input(view(a.w_up, a.n, a.k, 2), a.dx.ptr != nullptr);
  return k.finish();
}

int run(const coll_gated_bwd_t &a, Ws &ws, bool dry, cudaStream_t s) {
  if (!a.dx.ptr && !a.dw_gate.ptr) return COLL_OK;
  const coll_mat_t dg = scratch(ws, a.m, a.n), du = scratch(ws, a.m, a.n);
  DenseActBwd b = {};
  b.m = a.m;
  b.n = a.n;
  b.dy = mat(a.dh);
  b.pre = mat(a.gate);
  b.up = mat(a.up);
  b.dz = dg.ptr;
  b.du = du.ptr;
  b.ld = dg.rs;
  b.type = (int32_t)a.dtype;
  b.act = (int32_t)a.act;
  b.gated = 1;
  DenseJob jobs[2];
  int n = 0;
  if (a.dx.ptr) {  // dx = dg w_gate + du w_up: one sum over both
    DenseJob &j = jobs[n++];
    j = job(a.m, a.k, a.n, a.dtype, a.status);
    j.nseg = 2;
    j.a[0] = mat(dg);
    j.a[1] = mat(du);
    j.b[0] = turned(a.w_gate);
    j.b[1] = turned(a.w_up);
    set_out(j, 0, a.dx);
  }
  if (a.dw_gate.ptr) {  // dw_gate = dg^T x, dw_up = du^T x
    DenseJob &j = jobs[n++];
    j = job(a.n, a.k, a.m, a.dtype, a.status);
    j.nbatch = 2;
    j.a[0] = turned(dg);
    j.a[1] = turned(du);
    j.b[0] = turned(a.x);
    j.e.out_type = (int32_t)a.grad_dtype;
    set_out(j, 0, a.dw_gate);
    set_out(j, 1, a.dw_up);
  }
  return products(jobs, n, ws, dry, s, a.m > 0 && a.n > 0 ? &b : nullptr);
}

// Checks, then the counting pass: workspace bytes, or a code.
template <typename T>
int64_t count(const T *a, Ws &ws) {
  if (!a) return COLL_EINVAL;
  const int c = check(*a);
  if (c) return c;
  if ((uintptr_t)a->status % sizeof(int32_t)) return COLL_EALIGN;
  const int r = run(*a, ws, true, nullptr);
  return r ? r : ws.over ? COLL_EINVAL : ws.used ? (int64_t)ws.used + 128 : 0;  // room to start on 128 bytes
}

template <typename T>
int64_t workspace(const T *a) {
  coll::TcParams plan;
  Ws ws = {};
  ws.plan = &plan;
  return count(a, ws);
}

template <typename T>
int call(const T *a, void *stream) {
  coll::TcParams plan;
  Ws ws = {};
  ws.plan = &plan;
  const int64_t need = count(a, ws);
  if (need < 0) return (int)need;
  if (need > 0) {
    if (!a->workspace || ((uintptr_t)a->workspace & 15u) || a->workspace_bytes < (uint64_t)need)
      return COLL_EWORKSPACE;
    ws.base = reinterpret_cast<char *>(((uintptr_t)a->workspace + 127) & ~(uintptr_t)127);
  }
  ws.used = 0;
  return run(*a, ws, false, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" int coll_linear(const coll_linear_t *a, void *stream) { return call(a, stream); }
extern "C" int coll_linear_backward(const coll_linear_bwd_t *a, void *stream) {
  return call(a, stream);
}
extern "C" int coll_gated_ffn(const coll_gated_t *a, void *stream) { return call(a, stream); }
extern "C" int coll_gated_ffn_backward(const coll_gated_bwd_t *a, void *stream) {
  return call(a, stream);
}
extern "C" int64_t coll_linear_workspace(const coll_linear_t *a) { return workspace(a); }
extern "C" int64_t coll_linear_backward_workspace(const coll_linear_bwd_t *a) {
  return workspace(a);
}
extern "C" int64_t coll_gated_ffn_workspace(const coll_gated_t *a) { return workspace(a); }
extern "C" int64_t coll_gated_ffn_backward_workspace(const coll_gated_bwd_t *a) {
  return workspace(a);
}
