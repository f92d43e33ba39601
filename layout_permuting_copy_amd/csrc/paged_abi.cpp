// C ABI of the paged key-value cache operators: argument checks and launches.
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

// (batch, heads, columns >= cols)
tc::PagedRows rows_of(const char* name, const void* p, const tc_layout* l, int64_t batch, int64_t heads, int64_t cols,
                      Operand* o) {
  *o = operand(name, p, l, 3, 4);
  if (o->e[0] != batch || o->e[1] != heads || o->e[2] < cols)
    refuse(TC_E_EXTENT, std::string(name) + ": expected (batch, heads, at least " + std::to_string(cols) + ")");
  return tc::PagedRows{o->s[0] / 4, o->s[1] / 4, o->s[2] / 4, o->e[2]};
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

void attention_sizes(int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_len) {
  need(batch >= 0 && heads >= 1 && q_heads >= 0 && q_heads % heads == 0, TC_E_EXTENT,
       "query heads must be a multiple of the cache's heads");
  need(head_dim >= 16 && head_dim <= tc::kPagedMaxHeadDim && head_dim % 16 == 0, TC_E_EXTENT,
       "head_dim must be a multiple of 16 from 16 to 256");
  need(max_len >= 0 && max_len <= (int64_t(1) << 30), TC_E_RANGE, "max_len beyond 2^30");
  need(batch <= INT32_MAX && q_heads <= 65535 && batch * q_heads <= (int64_t(1) << 30), TC_E_RANGE,
       "q_heads beyond 65535 or batch * q_heads beyond 2^30");
}

// Floats of each part of the workspace.
struct Workspace {
  tc::PagedCut cut;
  int64_t o, ml, parts, final_ml, logits;
  int64_t bytes() const { return 4 * (o + ml + parts + final_ml + logits); }
};
Workspace workspace_of(int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_len, bool weights,
                       bool most) {
  Workspace w{};
  if (batch == 0 || q_heads == 0) return w;
  w.cut = tc::paged_cut(batch, heads, q_heads / heads, head_dim, max_len, most);
  need(w.cut.units < (int64_t(1) << 31) && w.cut.workgroups < (int64_t(1) << 31) && __int128(batch) * q_heads * max_len < kLim, TC_E_RANGE,
       "batch, heads and max_len beyond what the kernels count");
  if (w.cut.cuts) {
    w.o = w.cut.workgroups * 2 * w.cut.tile_heads * head_dim;
    w.ml = w.cut.workgroups * 2 * w.cut.tile_heads * 2;
    w.parts = w.cut.runs * int64_t(sizeof(tc::PagedParts) / 4);
  }
  if (weights) {
    w.final_ml = (batch * q_heads * 2 + 3) / 4 * 4;
    w.logits = batch * q_heads * tc::paged_logit_row(max_len);
  }
  return w;
}

}  // namespace

extern "C" {

int tc_paged_append(const tc_paged_cache* cache, const void* k_new, const tc_layout* k_layout, const void* v_new,
                    const tc_layout* v_layout, int dtype, const int32_t* block_table,
                    const tc_layout* table_layout, const int32_t* seq_lens, const int32_t* token_starts,
                    float* weights, const tc_layout* weights_layout, void* stream) {
  return guarded([&]() -> int {
    const int eb = float_bytes(dtype);
    const Pool c = pool_of("cache", cache, true);
    if (c.dtype != TC_E4M3 && c.dtype != dtype) refuse(TC_E_DTYPE, "new rows and cache differ in type");
    const Operand k = operand("k_new", k_new, k_layout, 3, eb), v = operand("v_new", v_new, v_layout, 3, eb);
    for (int i = 0; i < 3; ++i)
      need(k.e[i] == v.e[i], TC_E_EXTENT, "k_new and v_new differ in shape");
    need(k.e[1] == c.heads && k.e[2] == c.dim, TC_E_EXTENT, "new rows must have shape (tokens, heads, head_dim) of the cache");
    tc::AppendArgs a{};
    Operand t, w{};
    a.table = table_of("block_table", block_table, table_layout, &t);
    const int64_t batch = t.e[0];
    need(token_starts || k.e[0] == batch, TC_E_EXTENT, "without token_starts there is one token a sequence");
    const Operand lens = vector_of("seq_lens", seq_lens, batch);
    const Operand starts = vector_of("token_starts", token_starts, token_starts ? batch + 1 : 0);
    w.empty = true;
    if (weights) a.w = rows_of("weights", weights, weights_layout, batch, c.heads, 0, &w);
    if (!w.empty) injective("weights", w, 3, 4);
    if (k.empty || batch == 0 || c.empty || t.empty) return TC_OK;
    unit_inner("k_new", k, 2, eb);
    unit_inner("v_new", v, 2, eb);
    for (const Operand* x : Operands{&k, &v, &t, &lens, &starts, &w})
      if (touches(c, *x)) refuse(TC_E_ALIAS, "the cache overlaps another argument");
    for (const Operand* x : Operands{&k, &v, &t, &lens, &starts}) apart("weights and an input", w, *x);
    need(k.e[0] <= (int64_t(1) << 31) - 1, TC_E_RANGE, "more than 2^31 tokens");
    a.pool = c.p;
    a.k = k.p;
    a.v = v.p;
    a.kt = k.s[0], a.kh = k.s[1], a.vt = v.s[0], a.vh = v.s[1];
    a.lens = reinterpret_cast<const int32_t*>(lens.p);
    a.starts = token_starts ? reinterpret_cast<const int32_t*>(starts.p) : nullptr;
    a.weights = w.empty ? nullptr : reinterpret_cast<float*>(w.p);
    a.tokens = k.e[0];
    a.heads = int32_t(c.heads);
    a.head_dim = int32_t(c.dim);
    const uintptr_t al = reinterpret_cast<uintptr_t>(k.p) | reinterpret_cast<uintptr_t>(v.p) | uintptr_t(k.s[0]) |
                         uintptr_t(k.s[1]) | uintptr_t(v.s[0]) | uintptr_t(v.s[1]);
    return launched(tc::launch_paged_append(a, dtype, c.dtype, al % 16 == 0, stream));
  });
}

int64_t tc_paged_attention_workspace(int64_t batch, int64_t q_heads, int64_t heads, int64_t head_dim,
                                     int64_t max_len, int with_weights) {
  int64_t bytes = 0;
  const int rc = guarded([&]() -> int {
    attention_sizes(batch, q_heads, heads, head_dim, max_len);
    bytes = workspace_of(batch, q_heads, heads, head_dim, max_len, with_weights != 0, true).bytes();
    return TC_OK;
  });
  return rc == TC_OK ? bytes : rc;
}

int tc_paged_attention(const tc_paged_cache* cache, const void* q, const tc_layout* q_layout, void* out,
                       const tc_layout* out_layout, int dtype, const int32_t* block_table,
                       const tc_layout* table_layout, const int32_t* seq_lens, int64_t max_len, float scale,
                       float* lse, const tc_layout* lse_layout, const float* weights,
                       const tc_layout* weights_layout, float* weights_out, const tc_layout* weights_out_layout,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const int eb = float_bytes(dtype);
    const Pool c = pool_of("cache", cache, false);
    if (c.dtype != TC_E4M3 && c.dtype != dtype) refuse(TC_E_DTYPE, "q and cache differ in type");
    const Operand qo = operand("q", q, q_layout, 3, eb), oo = operand("out", out, out_layout, 3, eb);
    for (int i = 0; i < 3; ++i)
      need(qo.e[i] == oo.e[i], TC_E_EXTENT, "q and out differ in shape");
    const int64_t batch = qo.e[0], q_heads = qo.e[1];
    need(qo.e[2] == c.dim, TC_E_EXTENT, "q and the cache differ in head_dim");
    attention_sizes(batch, q_heads, c.heads, c.dim, max_len);
    need(std::isfinite(scale * kLog2e), TC_E_ARG, "scale (and scale * log2 e) must be finite");
    tc::AttentionArgs a{};
    Operand t, l{}, w{}, wo{};
    a.table = table_of("block_table", block_table, table_layout, &t);
    need(t.e[0] == batch, TC_E_EXTENT, "block_table and q differ in batch");
    const Operand lens = vector_of("seq_lens", seq_lens, batch);
    l.empty = w.empty = wo.empty = true;
    if (lse) {
      l = operand("lse", lse, lse_layout, 2, 4);
      need(l.e[0] == batch && l.e[1] == q_heads, TC_E_EXTENT, "lse must have shape (batch, q_heads)");
      injective("lse", l, 2, 4);
    }
    need((weights != nullptr) == (weights_out != nullptr) || batch == 0 || max_len == 0, TC_E_NULL,
         "weights and weights_out go together");
    if (weights_out) {
      a.w = rows_of("weights", weights, weights_layout, batch, c.heads, max_len, &w);
      a.wo = rows_of("weights_out", weights_out, weights_out_layout, batch, c.heads, max_len, &wo);
      if (!wo.empty) injective("weights_out", wo, 3, 4);
      bool same = w.p == wo.p;
      for (int i = 0; i < 3; ++i) same = same && w.s[i] == wo.s[i];
      if (!same) apart("weights and weights_out", w, wo);
    }
    if (qo.empty) return TC_OK;
    unit_inner("q", qo, 2, eb);
    unit_inner("out", oo, 2, eb);
    injective("out", oo, 3, eb);
    const bool with_weights = weights_out != nullptr && max_len > 0;
    const Workspace ws = workspace_of(batch, q_heads, c.heads, c.dim, max_len, with_weights, false);
    need(workspace_bytes >= ws.bytes(), TC_E_ARG, "workspace too small");
    need(workspace || ws.bytes() == 0, TC_E_NULL, "null workspace");
    need(reinterpret_cast<uintptr_t>(workspace) % 16 == 0, TC_E_ALIGN, "workspace not aligned to 16 bytes");
    Operand work{};
    work.empty = ws.bytes() == 0;
    work.r.lo = reinterpret_cast<uintptr_t>(workspace);
    work.r.hi = work.r.lo + ws.bytes();
    const Operand* outs[] = {&oo, &l, &wo, &work};
    for (const Operand* x : outs) {
      if (touches(c, *x)) refuse(TC_E_ALIAS, "the cache overlaps an output");
      for (const Operand* y : Operands{&qo, &t, &lens}) apart("an output and an input", *x, *y);
      if (x != &wo) apart("weights and another output", *x, w);
      for (const Operand* y : outs)
        if (x != y) apart("two outputs", *x, *y);
    }
    a.pool = c.p;
    a.q = qo.p;
    a.out = oo.p;
    a.qb = qo.s[0], a.qh = qo.s[1], a.ob = oo.s[0], a.oh = oo.s[1];
    a.lens = reinterpret_cast<const int32_t*>(lens.p);
    a.lse = l.empty ? nullptr : reinterpret_cast<float*>(l.p);
    a.lb = l.s[0] / 4, a.lh = l.s[1] / 4;
    a.weights = with_weights ? reinterpret_cast<const float*>(w.p) : nullptr;
    a.weights_out = with_weights ? reinterpret_cast<float*>(wo.p) : nullptr;
    float* f = static_cast<float*>(workspace);
    a.part_o = f;
    a.part_ml = f + ws.o;
    a.parts = ws.cut.cuts ? reinterpret_cast<tc::PagedParts*>(f + ws.o + ws.ml) : nullptr;
    f += ws.o + ws.ml + ws.parts;
    a.final_ml = with_weights ? f : nullptr;
    a.logits = with_weights ? f + ws.final_ml : nullptr;
    a.logit_row = tc::paged_logit_row(max_len);
    a.heads = int32_t(c.heads);
    a.group = int32_t(q_heads / c.heads);
    a.head_dim = int32_t(c.dim);
    // no row past the table's columns, and none of an empty pool
    const int64_t held = t.empty || c.empty ? 0 : std::min<int64_t>(max_len, int64_t(a.table.cols) * c.page_size);
    a.max_len = int32_t(held);
    a.units = ws.cut.units;
    a.runs = int32_t(ws.cut.runs);
    a.least_units = int32_t(ws.cut.least_units);
    a.tile_heads = int32_t(ws.cut.tile_heads);
    a.head_tiles = int32_t(ws.cut.head_tiles);
    a.unit = tc::make_div32(uint32_t(ws.cut.unit_rows));
    a.scale_log2e = scale * kLog2e;
    return launched(tc::launch_paged_attention(a, dtype, c.dtype, stream));
  });
}

int tc_paged_evict(const tc_paged_cache* src, const int32_t* block_table, const tc_layout* table_layout,
                   const int32_t* seq_lens, int64_t max_len, const float* weights, const tc_layout* weights_layout,
                   const tc_paged_cache* dst, const int32_t* dst_table, const tc_layout* dst_table_layout,
                   int64_t budget, int64_t recent, int32_t* lens_out, int32_t* kept, const tc_layout* kept_layout,
                   float* weights_out, const tc_layout* weights_out_layout, void* stream) {
  return guarded([&]() -> int {
    const Pool s = pool_of("src", src, false), d = pool_of("dst", dst, true);
    need(s.dtype == d.dtype, TC_E_DTYPE, "src and dst differ in type");
    need(s.heads == d.heads && s.dim == d.dim, TC_E_EXTENT, "src and dst differ in heads or head_dim");
    need(budget >= 1 && budget <= (int64_t(1) << 30), TC_E_ARG, "budget must be from 1 to 2^30");
    need(recent >= 0 && recent <= budget, TC_E_ARG, "recent must be from 0 to budget");
    need(max_len >= 0 && max_len <= (int64_t(1) << 30), TC_E_RANGE, "max_len beyond 2^30");
    tc::EvictArgs a{};
    Operand t, dt, w, kp, wo{};
    a.table = table_of("block_table", block_table, table_layout, &t);
    a.dst_table = table_of("dst_table", dst_table, dst_table_layout, &dt);
    const int64_t batch = t.e[0];
    need(dt.e[0] == batch, TC_E_EXTENT, "the tables differ in batch");
    // no row past the table's columns
    max_len = std::min<int64_t>(max_len, t.e[1] * s.page_size);
    const int64_t most = std::min<int64_t>(budget, max_len);
    need(dt.e[1] * d.page_size >= most, TC_E_EXTENT, "dst_table holds fewer rows than are kept");
    const Operand lens = vector_of("seq_lens", seq_lens, batch), lo = vector_of("lens_out", lens_out, batch);
    a.w = rows_of("weights", weights, weights_layout, batch, s.heads, max_len, &w);
    a.kr = rows_of("kept", kept, kept_layout, batch, s.heads, most, &kp);
    if (!kp.empty) injective("kept", kp, 3, 4);
    wo.empty = true;
    if (weights_out) {
      a.wo = rows_of("weights_out", weights_out, weights_out_layout, batch, s.heads, most, &wo);
      if (!wo.empty) injective("weights_out", wo, 3, 4);
    }
    need(batch * s.heads <= (int64_t(1) << 30), TC_E_RANGE, "batch * heads beyond 2^30");
    if (batch == 0) return TC_OK;
    const Operand* outs[] = {&lo, &kp, &wo};
    for (const Operand* x : outs) {
      if (touches(s, *x) || touches(d, *x)) refuse(TC_E_ALIAS, "a cache overlaps an output");
      for (const Operand* y : Operands{&t, &dt, &lens, &w}) apart("an output and an input", *x, *y);
      for (const Operand* y : outs)
        if (x != y) apart("two outputs", *x, *y);
    }
    for (const Operand* x : Operands{&t, &dt, &lens, &w})
      if (touches(d, *x)) refuse(TC_E_ALIAS, "dst overlaps an input");
    // the same pool, or another one
    bool same = s.pages == d.pages && s.page_size == d.page_size && s.p.k == d.p.k && s.p.v == d.p.v &&
                s.p.ks == d.p.ks && s.p.vs == d.p.vs;
    for (int i = 0; i < 4; ++i) same = same && s.k.s[i] == d.k.s[i] && s.v.s[i] == d.v.s[i];
    for (int i = 0; i < 3; ++i) same = same && s.ks.s[i] == d.ks.s[i] && s.vs.s[i] == d.vs.s[i];
    if (!same && !d.empty) {
      bool hit = touches(s, d.k) || touches(s, d.v);
      if (d.p.ks) hit = hit || touches(s, d.ks) || touches(s, d.vs);
      if (hit) refuse(TC_E_ALIAS, "src and dst overlap and are not the same pool");
    }
    a.src = s.p;
    a.dst = d.p;
    if (s.empty) a.src.pages = 0;
    if (d.empty) a.dst.pages = 0;
    a.lens = reinterpret_cast<const int32_t*>(lens.p);
    a.lens_out = reinterpret_cast<int32_t*>(lo.p);
    a.weights = reinterpret_cast<const float*>(w.p);
    a.kept = reinterpret_cast<int32_t*>(kp.p);
    a.weights_out = wo.empty ? nullptr : reinterpret_cast<float*>(wo.p);
    a.heads = int32_t(s.heads);
    a.row_bytes = int32_t(s.dim * s.eb);
    a.max_len = int32_t(max_len);
    a.budget = int32_t(budget);
    a.recent = int32_t(recent);
    return launched(tc::launch_paged_evict(a, s.dtype, stream));
  });
}

}  // extern "C"
