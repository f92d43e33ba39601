// Argument checks that the entry points on tensors share: operands from layouts, overlaps, pools, tables.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "paged.hpp"

namespace {

using tc::set_last_error;

constexpr int64_t kLim = int64_t(1) << 58;
constexpr float kLog2e = 1.4426950408889634f;

// Thrown inside the entry points and turned into a status at their border.
struct Refusal {
  int code;
  std::string why;
};

[[noreturn]] void refuse(int code, const std::string& why) { throw Refusal{code, why}; }
void need(bool ok, int code, const char* why) {
  if (!ok) refuse(code, why);
}

// The bytes a layout touches: [lo, hi) addresses.
struct Range {
  __int128 lo, hi;
};
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// One operand: a base pointer with its layout's offset folded in, extents, byte strides, byte range.
struct Operand {
  unsigned char* p;
  int64_t e[4], s[4];  // extents, strides in bytes
  Range r;
  bool empty;
};

[[noreturn]] void refuse_operand(int code, const char* name, const char* why) { refuse(code, std::string(name) + why); }

Operand operand(const char* name, const void* p, const tc_layout* l, int rank, int eb) {
  if (!l) refuse_operand(TC_E_NULL, name, ": null layout");
  if (l->rank != rank) refuse(TC_E_RANK, std::string(name) + ": expected " + std::to_string(rank) + " modes");
  Operand o{};
  o.empty = false;
  __int128 hi = 0;
  if (l->offset < -kLim || l->offset > kLim) refuse_operand(TC_E_RANGE, name, ": offset beyond 2^58");
  for (int k = 0; k < rank; ++k) {
    if (l->shape[k] < 0) refuse_operand(TC_E_EXTENT, name, ": negative extent");
    o.e[k] = l->shape[k];
    o.empty = o.empty || o.e[k] == 0;
    if (o.e[k] > 1) {
      if (l->stride[k] < 0) refuse_operand(TC_E_ARG, name, ": negative stride");
      hi += __int128(o.e[k] - 1) * l->stride[k];
      if (l->stride[k] > kLim || hi > kLim) refuse_operand(TC_E_RANGE, name, ": element offsets beyond 2^58");
      o.s[k] = l->stride[k] * eb;
    }
  }
  if (o.empty) return o;
  if (!p) refuse_operand(TC_E_NULL, name, ": null pointer");
  if (reinterpret_cast<uintptr_t>(p) % uintptr_t(eb)) refuse_operand(TC_E_ALIGN, name, ": pointer not aligned to its elements");
  const __int128 base = __int128(reinterpret_cast<uintptr_t>(p)) + __int128(l->offset) * eb;
  o.p = reinterpret_cast<unsigned char*>(uintptr_t(base));
  o.r = Range{base, base + hi * eb + eb};
  return o;
}

// Written operands: no two indices name one element.  Sorted strides have to exceed the span of the
// smaller modes: what views of a tensor look like (anything more interlaced is refused).
void injective(const char* name, const Operand& o, int rank, int eb) {
  int order[4], n = 0;
  for (int k = 0; k < rank; ++k)
    if (o.e[k] > 1) {
      int at = n++;
      while (at > 0 && o.s[order[at - 1]] > o.s[k]) {
        order[at] = order[at - 1];
        --at;
      }
      order[at] = k;
    }
  __int128 span = eb;
  for (int i = 0; i < n; ++i) {
    const int k = order[i];
    if (o.s[k] < span) refuse(TC_E_NONINJECTIVE, std::string(name) + ": two indices name one element");
    span += __int128(o.e[k] - 1) * o.s[k];
  }
}

// Whether two injective operands of one shape share no element: ranges apart, or the same strides
// and a gap that is the stride of one more mode, of two, in an injective layout (halves of one allocation): it lies
// between the spans of two neighbouring modes, and every larger stride exceeds both operands' span.
bool disjoint(const Operand& x, const Operand& y, int rank, int eb) {
  if (!overlap(x.r, y.r)) return true;
  const Operand &a = x.r.lo < y.r.lo ? x : y, &b = x.r.lo < y.r.lo ? y : x;
  int order[4], n = 0;
  for (int k = 0; k < rank; ++k)
    if (a.e[k] > 1) {
      if (a.s[k] != b.s[k]) return false;
      int at = n++;
      while (at > 0 && a.s[order[at - 1]] > a.s[k]) {
        order[at] = order[at - 1];
        --at;
      }
      order[at] = k;
    }
  const __int128 gap = b.r.lo - a.r.lo;
  __int128 span = eb;  // of the modes order[0 .. i-1]
  bool held = false;   // they lie inside the gap, or a smaller mode's do, and those since step over both operands
  for (int i = 0; i <= n; ++i) {
    held = (held || gap >= span) && (i == n || gap + span <= a.s[order[i]]);
    if (i < n) span += __int128(a.e[order[i]] - 1) * a.s[order[i]];
  }
  return held;
}

void unit_inner(const char* name, const Operand& o, int k, int eb) {
  if (o.e[k] > 1 && o.s[k] != eb) refuse(TC_E_ARG, std::string(name) + ": the innermost stride must be 1");
}

int float_bytes(int dtype) {
  if (dtype != TC_F16 && dtype != TC_BF16) refuse(TC_E_DTYPE, "dtype must be TC_F16 or TC_BF16");
  return 2;
}

typedef std::initializer_list<const Operand*> Operands;

struct Pool {
  tc::PagedPool p;
  int64_t heads, dim, pages, page_size;
  int eb, dtype;
  Operand k, v, ks, vs;
  bool empty;  // no pages or no heads: nothing to read or write
};

Pool pool_of(const char* name, const tc_paged_cache* c, bool written) {
  const std::string n(name);  // (short enough to need no allocation)
  if (!c) refuse(TC_E_NULL, n + ": null cache");
  Pool o{};
  o.dtype = c->dtype;
  o.eb = c->dtype == TC_E4M3 ? 1 : (c->dtype == TC_F16 || c->dtype == TC_BF16) ? 2 : 0;
  if (!o.eb) refuse(TC_E_DTYPE, n + ": dtype must be TC_F16, TC_BF16 or TC_E4M3");
  const bool quantised = c->dtype == TC_E4M3;
  o.k = operand("keys", c->k, &c->k_layout, 4, o.eb);
  o.v = operand("values", c->v, &c->v_layout, 4, o.eb);
  for (int i = 0; i < 4; ++i)
    if (o.k.e[i] != o.v.e[i]) refuse(TC_E_EXTENT, n + ": keys and values differ in shape");
  o.pages = o.k.e[0];
  o.page_size = o.k.e[1];
  o.heads = o.k.e[2];
  o.dim = o.k.e[3];
  if (o.dim < 16 || o.dim > tc::kPagedMaxHeadDim || o.dim % 16)
    refuse(TC_E_EXTENT, n + ": head_dim must be a multiple of 16 from 16 to 256");
  if (o.page_size < 1) refuse(TC_E_EXTENT, n + ": page_size must be at least 1");
  if (o.heads < 1) refuse(TC_E_EXTENT, n + ": a cache has at least one head");
  if (o.pages > INT32_MAX || o.page_size > INT32_MAX || o.heads > INT32_MAX)
    refuse(TC_E_RANGE, n + ": pages, page_size and heads must fit 31 bits");
  o.empty = o.k.empty;
  if (quantised) {
    o.ks = operand("k_scale", c->k_scale, &c->k_scale_layout, 3, 4);
    o.vs = operand("v_scale", c->v_scale, &c->v_scale_layout, 3, 4);
    for (int i = 0; i < 3; ++i)
      if (o.ks.e[i] != o.k.e[i] || o.vs.e[i] != o.k.e[i])
        refuse(TC_E_EXTENT, n + ": scales must have shape (pages, page_size, heads)");
  } else if (c->k_scale || c->v_scale) {
    refuse(TC_E_ARG, n + ": only 8-bit caches have scales");
  }
  if (!o.empty) {
    for (const Operand* x : {&o.k, &o.v}) {
      unit_inner(name, *x, 3, o.eb);
      bool ok = reinterpret_cast<uintptr_t>(x->p) % 16 == 0;
      for (int i = 0; i < 3; ++i) ok = ok && x->s[i] % 16 == 0;
      if (!ok) refuse(TC_E_ALIGN, n + ": rows must start on 16-byte boundaries");
      if (written) injective(name, *x, 4, o.eb);
    }
    if (written && !disjoint(o.k, o.v, 4, o.eb)) refuse(TC_E_ALIAS, n + ": keys and values overlap");
    if (written && quantised) {
      injective("k_scale", o.ks, 3, 4);
      injective("v_scale", o.vs, 3, 4);
      if (!disjoint(o.ks, o.vs, 3, 4)) refuse(TC_E_ALIAS, n + ": the scales overlap");
      for (const Operand* x : {&o.k, &o.v})
        if (overlap(x->r, o.ks.r) || overlap(x->r, o.vs.r)) refuse(TC_E_ALIAS, n + ": rows and scales overlap");
    }
  }
  tc::PagedPool& p = o.p;
  p.k = o.k.p;
  p.v = o.v.p;
  p.kp = o.k.s[0], p.kr = o.k.s[1], p.kh = o.k.s[2];
  p.vp = o.v.s[0], p.vr = o.v.s[1], p.vh = o.v.s[2];
  if (quantised) {
    p.ks = reinterpret_cast<float*>(o.ks.p);
    p.vs = reinterpret_cast<float*>(o.vs.p);
    p.ksp = o.ks.s[0] / 4, p.ksr = o.ks.s[1] / 4, p.ksh = o.ks.s[2] / 4;
    p.vsp = o.vs.s[0] / 4, p.vsr = o.vs.s[1] / 4, p.vsh = o.vs.s[2] / 4;
  }
  p.pages = int32_t(o.pages);
  p.page_size = int32_t(o.page_size);
  p.div = tc::make_div32(uint32_t(o.page_size));
  return o;
}

bool touches(const Pool& c, const Operand& x) {
  if (c.empty || x.empty) return false;
  if (overlap(c.k.r, x.r) || overlap(c.v.r, x.r)) return true;
  return c.p.ks && (overlap(c.ks.r, x.r) || overlap(c.vs.r, x.r));
}

tc::PagedTable table_of(const char* name, const int32_t* p, const tc_layout* l, Operand* o) {
  *o = operand(name, p, l, 2, 4);
  if (o->e[0] > INT32_MAX || o->e[1] > INT32_MAX) refuse(TC_E_RANGE, std::string(name) + ": extents beyond 31 bits");
  return tc::PagedTable{reinterpret_cast<const int32_t*>(o->p), o->s[0] / 4, o->s[1] / 4, int32_t(o->e[0]),
                        int32_t(o->e[1])};
}

// A contiguous int32 vector.
Operand vector_of(const char* name, const void* p, int64_t n) {
  tc_layout l{};
  l.rank = 1;
  l.shape[0] = n;
  l.stride[0] = 1;
  return operand(name, p, &l, 1, 4);
}

void apart(const char* what, const Operand& a, const Operand& b) {
  if (!a.empty && !b.empty && overlap(a.r, b.r)) refuse(TC_E_ALIAS, std::string(what) + " overlap");
}

int launched(int rc) {
  if (rc != TC_OK) refuse(rc, "more rows than one launch takes");
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) refuse(TC_E_HIP, std::string("kernel launch failed: ") + hipGetErrorString(e));
  return TC_OK;
}

// Runs an entry point's body; no exception leaves it.
template <class F>
int guarded(F&& f) noexcept {
  try {
    try {
      set_last_error(TC_OK, "");
      return f();
    } catch (const Refusal& r) {
      return set_last_error(r.code, r.why);
    }
  } catch (...) {
    return TC_E_ARG;  // no memory for the check's own text
  }
}

}  // namespace
