// Argument checks of the operators' C entry points (host only): extents, alignment, overlap.
#pragma once

#include <stdint.h>

#include "coll.h"

namespace coll {

constexpr uint64_t kAddressable = (uint64_t)1 << 40;

inline bool is_half(int64_t t) { return t == COLL_BF16 || t == COLL_F16; }
inline int esize(int64_t t) { return t == COLL_F32 ? 4 : 2; }

// A matrix with its extent, for the checks.
struct View {
  const void *p;
  int64_t rows, cols, rs, cs;
  int es;
};

inline View view(const coll_mat_t &m, int64_t rows, int64_t cols, int es) {
  return View{m.ptr, rows, cols, m.rs, m.cs, es};
}

inline bool empty(const View &v) { return !v.p || v.rows <= 0 || v.cols <= 0; }

inline void range(const View &v, uintptr_t &lo, uintptr_t &hi) {
  const int64_t r = (v.rows - 1) * v.rs, c = (v.cols - 1) * v.cs;
  const int64_t a = (r < 0 ? r : 0) + (c < 0 ? c : 0), b = (r > 0 ? r : 0) + (c > 0 ? c : 0);
  lo = (uintptr_t)v.p + (intptr_t)(a * v.es);
  hi = (uintptr_t)v.p + (intptr_t)((b + 1) * v.es);
}

// Do two views share memory? Exact for rows of the same stride (column slices of one buffer);
// otherwise by their address ranges.
inline bool shares(const View &a, const View &b) {
  if (empty(a) || empty(b)) return false;
  uintptr_t a0, a1, b0, b1;
  range(a, a0, a1);
  range(b, b0, b1);
  if (a1 <= b0 || b1 <= a0) return false;
  const int64_t ra = a.rs * a.es, rb = b.rs * b.es;
  const int64_t wa = a.cols * a.es, wb = b.cols * b.es;
  if (a.cs == 1 && b.cs == 1 && ra == rb && ra >= wa && ra >= wb) {
    int64_t d = ((intptr_t)b.p - (intptr_t)a.p) % ra;
    if (d < 0) d += ra;
    return d < wa || d + wb > ra;
  }
  return true;
}

inline bool same(const View &a, const View &b) {
  return a.p == b.p && (a.rs == b.rs || a.rows <= 1) && (a.cs == b.cs || a.cols <= 1) &&
         a.es == b.es;
}

// Codes for one matrix: present where it has to be, its base a multiple of its element, and for
// an output one element per address.
inline int check_mat(const View &v, bool needed, bool output) {
  if (!v.p) return needed && v.rows > 0 && v.cols > 0 ? COLL_EINVAL : COLL_OK;
  if ((uintptr_t)v.p % (unsigned)v.es) return COLL_EALIGN;
  // what a device can address, so that no offset below leaves 64 bits
  const int64_t lim = (int64_t)kAddressable;
  const int64_t rs = v.rows > 1 ? lim / (v.rows - 1) : lim;
  const int64_t cs = v.cols > 1 ? lim / (v.cols - 1) : lim;
  if (v.rs > rs || v.rs < -rs || v.cs > cs || v.cs < -cs) return COLL_EINVAL;
  if (output && v.rows > 0 && v.cols > 0) {
    if (v.cols > 1 && v.cs != 1) return COLL_EINVAL;
    if (v.rows > 1 && v.rs < v.cols) return COLL_EINVAL;
  }
  return COLL_OK;
}

struct Check {
  int code = COLL_OK;
  View in[8], out[4];
  int n_in = 0, n_out = 0;
  int input(const View &v, bool needed = true) {  // returns its place
    if (!code) code = check_mat(v, needed, false);
    in[n_in] = v;
    return n_in++;
  }
  void output(const View &v, bool needed = true) {
    if (!code) code = check_mat(v, needed, true);
    out[n_out++] = v;
  }
  // Overlaps after every check above. `in_place`: the place of the one input that out[0] may
  // equal; another input of the same memory would be read after out[0] was written over it.
  int finish(int in_place = -1) {
    if (code) return code;
    for (int o = 0; o < n_out; ++o) {
      for (int i = 0; i < n_in; ++i) {
        if (!shares(out[o], in[i])) continue;
        if (o == 0 && i == in_place && same(out[o], in[i])) continue;
        return COLL_EOVERLAP;
      }
      for (int q = 0; q < o; ++q)
        if (shares(out[o], out[q])) return COLL_EOVERLAP;
    }
    return COLL_OK;
  }
};

}  // namespace coll
