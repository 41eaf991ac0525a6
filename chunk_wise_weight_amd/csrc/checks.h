// What the entry points check of their arguments: types, workspaces, and arrays that lie over one another.
#pragma once

#include <algorithm>
#include <initializer_list>
#include <vector>

#include "../../include/ttt.h"
#include "errors.h"

constexpr int kMaxWidth = 65536;
constexpr long long kMaxRows = 0x7fffffffLL;

inline bool known(ttt_dtype t) { return t == TTT_F32 || t == TTT_BF16; }
inline size_t size_of(ttt_dtype t) { return t == TTT_BF16 ? 2 : 4; }

// An array of a call: its bytes, and the size of one element.
struct Span {
  const char *name;
  const void *p;
  size_t bytes, elem;
};

inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const char *x = (const char *)a.p, *y = (const char *)b.p;
  return x < y + b.bytes && y < x + a.bytes;
}

// Outputs against inputs and one another. in_place: pairs (output, input) that
// may be the same array.
struct Pair {
  const void *out, *in;
};
inline int check_spans(const char *where, std::initializer_list<Span> in, std::initializer_list<Span> out,
                       std::initializer_list<Pair> in_place) {
  for (const Span &s : in)
    if ((uintptr_t)s.p % s.elem) return ttt_fail(TTT_E_ARG, "%s: %s is not aligned to its elements", where, s.name);
  for (const Span *o = out.begin(); o != out.end(); ++o) {
    if ((uintptr_t)o->p % o->elem) return ttt_fail(TTT_E_ARG, "%s: %s is not aligned to its elements", where, o->name);
    for (const Span &s : in) {
      if (!overlap(*o, s)) continue;
      bool ok = false;
      for (const Pair &p : in_place) ok = ok || (p.out == o->p && p.in == s.p && o->p == s.p && o->bytes == s.bytes);
      if (!ok) return ttt_fail(TTT_E_ARG, "%s: %s overlaps %s", where, o->name, s.name);
    }
    for (const Span *q = out.begin(); q != o; ++q)
      if (overlap(*o, *q)) return ttt_fail(TTT_E_ARG, "%s: %s overlaps %s", where, o->name, q->name);
  }
  return TTT_OK;
}

inline int check_ws(const char *where, const void *ws, size_t have, size_t need) {
  if (!ws) return ttt_fail(TTT_E_NULL, "%s: the workspace is NULL", where);
  if ((uintptr_t)ws % 16) return ttt_fail(TTT_E_ARG, "%s: the workspace must be 16-byte aligned", where);
  if (have < need) return ttt_fail(TTT_E_SHAPE, "%s: needs %zu bytes of workspace, got %zu", where, need, have);
  return TTT_OK;
}

// Where the arrays of a call on many tensors lie: an output overlaps nothing (one written in place counts once).
struct Extent {
  uintptr_t lo, hi;
  bool out;
};
inline int check_extents(const char *where, std::vector<Extent> &e) {
  std::sort(e.begin(), e.end(), [](const Extent &a, const Extent &b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;  // ends of what came before
  for (const Extent &x : e) {
    if (x.lo < outs || (x.out && x.lo < any)) return ttt_fail(TTT_E_ARG, "%s: an output overlaps another array", where);
    any = std::max(any, x.hi);
    if (x.out) outs = std::max(outs, x.hi);
  }
  return TTT_OK;
}
