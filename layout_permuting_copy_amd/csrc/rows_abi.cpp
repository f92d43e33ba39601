// C ABI of the attention of several query rows a sequence and of the block tables' growth: argument checks and launches.
#include "paged_checks.hpp"

namespace {

constexpr int64_t kMost = int64_t(1) << 30;
constexpr int64_t kTokenStride = int64_t(1) << 24;  // bytes between packed tokens: offsets inside a tile of them are 32-bit

void rows_sizes(int64_t batch, int64_t tokens, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_len) {
  need(batch >= 0 && tokens >= 0 && heads >= 1 && q_heads >= 0 && q_heads % heads == 0, TC_E_EXTENT,
       "query heads must be a multiple of the key heads");
  need(head_dim >= 16 && head_dim <= tc::kPagedMaxHeadDim && head_dim % 16 == 0, TC_E_EXTENT,
       "head_dim must be a multiple of 16 from 16 to 256");
  need(max_len >= 0 && max_len <= kMost, TC_E_RANGE, "max_len beyond 2^30");
  need(batch <= kMost && tokens <= kMost && q_heads <= 65535 && tokens * q_heads <= kMost, TC_E_RANGE,
       "q_heads beyond 65535 or tokens * q_heads beyond 2^30");
}

void aligned(const char* name, const Operand& o, int rank) {
  bool ok = reinterpret_cast<uintptr_t>(o.p) % 16 == 0;
  for (int i = 0; i + 1 < rank; ++i) ok = ok && o.s[i] % 16 == 0;
  if (!ok) refuse_operand(TC_E_ALIGN, name, ": rows must start on 16-byte boundaries");
}

// q, out and lse of a call, and what both operators put into the arguments from them.
struct Queries {
  Operand q, o, l;
};
Queries queries_of(const void* q, const tc_layout* q_layout, void* out, const tc_layout* out_layout, int eb, float scale, float* lse,
                   const tc_layout* lse_layout, tc::RowsArgs* a) {
  Queries c;
  c.q = operand("q", q, q_layout, 3, eb);
  c.o = operand("out", out, out_layout, 3, eb);
  for (int i = 0; i < 3; ++i) need(c.q.e[i] == c.o.e[i], TC_E_EXTENT, "q and out differ in shape");
  const float scale2 = std::fabs(scale) * kLog2e;
  need(std::isfinite(scale2), TC_E_ARG, "scale (and scale * log2 e) must be finite");
  c.l = Operand{};
  c.l.empty = true;
  if (lse) {
    c.l = operand("lse", lse, lse_layout, 2, 4);
    need(c.l.e[0] == c.q.e[0] && c.l.e[1] == c.q.e[1], TC_E_EXTENT, "lse must have shape (tokens, q_heads)");
    injective("lse", c.l, 2, 4);
  }
  if (c.q.empty) return c;
  unit_inner("q", c.q, 2, eb);
  unit_inner("out", c.o, 2, eb);
  aligned("q", c.q, 3);
  aligned("out", c.o, 3);
  injective("out", c.o, 3, eb);
  a->q = c.q.p;
  a->out = c.o.p;
  a->qt = c.q.s[0], a->qh = c.q.s[1], a->ot = c.o.s[0], a->oh = c.o.s[1];
  a->lse = c.l.empty ? nullptr : reinterpret_cast<float*>(c.l.p);
  a->lt = c.l.s[0] / 4, a->lh = c.l.s[1] / 4;
  a->tokens = int32_t(c.q.e[0]);
  a->head_dim = int32_t(c.q.e[2]);
  // the kernels take maxima before the scale, which then must not turn them round: its sign goes to q, and a scale of 0
  // (0 times an infinity is no weight) to a q of zeros
  a->scale = scale == 0.0f ? 1.0f : std::fabs(scale);
  a->scale_log2e = scale == 0.0f ? kLog2e : scale2;
  a->q_and = scale == 0.0f ? 0u : ~0u;
  a->q_xor = scale < 0.0f ? 0x80008000u : 0u;
  return c;
}

void apart_from_inputs(const Operand* const* outs, int n_outs, Operands inputs) {
  for (int i = 0; i < n_outs; ++i)
    for (int j = 0; j < i; ++j) apart("two outputs", *outs[i], *outs[j]);
  for (int i = 0; i < n_outs; ++i)
    for (const Operand* y : inputs) apart("an output and an input", *outs[i], *y);
}

tc::RowsShape prompt_shape(int64_t batch, int64_t tokens, int64_t keys, int64_t q_heads, int64_t heads, int64_t dim) {
  return tc::rows_shape(false, false, batch, tokens, heads, q_heads / heads, dim, keys / batch);
}

// What the call takes of its workspace.
Operand workspace_of(void* workspace, int64_t workspace_bytes, const tc::RowsShape& shape, int64_t dim, tc::RowsArgs* a) {
  need(workspace_bytes >= shape.bytes, TC_E_ARG, "workspace too small");
  need(workspace || shape.bytes == 0, TC_E_NULL, "null workspace");
  need(reinterpret_cast<uintptr_t>(workspace) % 16 == 0, TC_E_ALIGN, "workspace not aligned to 16 bytes");
  Operand work{};
  work.empty = shape.bytes == 0;
  work.r.lo = reinterpret_cast<uintptr_t>(workspace);
  work.r.hi = work.r.lo + shape.bytes;
  a->part_units = static_cast<uint32_t*>(workspace);
  a->part_o = static_cast<float*>(workspace) + tc::kRowsWorkspaceHead / 4;
  a->part_ml = a->part_o + shape.workgroups * shape.tile_rows * dim;
  return work;
}

void dealt(tc::RowsArgs* a, const tc::RowsShape& shape, int64_t heads, int64_t group) {
  need(shape.workgroups < (int64_t(1) << 31), TC_E_RANGE, "more rows than one launch takes");
  a->heads = int32_t(heads);
  a->group = int32_t(group);
  a->group_div = tc::make_div32(uint32_t(group));
  a->heads_div = tc::make_div32(uint32_t(heads));
  a->slots = int32_t(shape.slots);
  a->least = int32_t(shape.least);
  a->tiles = shape.tiles;
  a->workgroups = shape.workgroups;
}

}  // namespace

extern "C" {

int tc_prompt_attention(const void* q, const tc_layout* q_layout, const void* k, const tc_layout* k_layout, const void* v,
                        const tc_layout* v_layout, void* out, const tc_layout* out_layout, int dtype, int64_t batch,
                        const int32_t* token_starts, const int32_t* key_starts, int causal, float scale, float* lse,
                        const tc_layout* lse_layout, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const int eb = float_bytes(dtype);
    tc::RowsArgs a{};
    const Queries c = queries_of(q, q_layout, out, out_layout, eb, scale, lse, lse_layout, &a);
    const Operand ko = operand("k", k, k_layout, 3, eb), vo = operand("v", v, v_layout, 3, eb);
    for (int i = 0; i < 3; ++i) need(ko.e[i] == vo.e[i], TC_E_EXTENT, "k and v differ in shape");
    const int64_t tokens = c.q.e[0], q_heads = c.q.e[1], rows = ko.e[0], heads = ko.e[1], dim = c.q.e[2];
    need(ko.e[2] == dim, TC_E_EXTENT, "q and k differ in head_dim");
    rows_sizes(batch, tokens, q_heads, heads, dim, 0);
    need(rows <= kMost, TC_E_RANGE, "more than 2^30 keys");
    need(key_starts || rows == tokens, TC_E_EXTENT, "without key_starts there is one key a token");
    need(causal == 0 || causal == 1, TC_E_ARG, "causal must be 0 or 1");
    const Operand starts = vector_of("token_starts", token_starts, batch + 1);
    const Operand kstarts = vector_of("key_starts", key_starts ? key_starts : token_starts, batch + 1);
    if (c.q.empty || batch == 0) return TC_OK;
    if (!ko.empty) {
      unit_inner("k", ko, 2, eb);
      unit_inner("v", vo, 2, eb);
      aligned("k", ko, 3);
      aligned("v", vo, 3);
      need(ko.s[0] < kTokenStride && vo.s[0] < kTokenStride, TC_E_RANGE, "keys or values 2^24 bytes apart from token to token");
    }
    const tc::RowsShape shape = prompt_shape(batch, tokens, rows, q_heads, heads, dim);
    const Operand work = workspace_of(workspace, workspace_bytes, shape, dim, &a);
    const Operand* outs[] = {&c.o, &c.l, &work};
    apart_from_inputs(outs, 3, Operands{&c.q, &ko, &vo, &starts, &kstarts});
    a.k = ko.p;
    a.v = vo.p;
    a.kt = ko.s[0], a.kh = ko.s[1], a.vt = vo.s[0], a.vh = vo.s[1];
    a.starts = reinterpret_cast<const int32_t*>(starts.p);
    a.key_starts = reinterpret_cast<const int32_t*>(kstarts.p);
    a.key_rows = int32_t(ko.empty ? 0 : rows);
    a.batch = int32_t(batch);
    a.causal = causal;
    dealt(&a, shape, heads, q_heads / heads);
    return launched(tc::launch_prompt_attention(a, shape, dtype, stream));
  });
}

int64_t tc_prompt_attention_workspace(int64_t batch, int64_t tokens, int64_t keys, int64_t q_heads, int64_t heads, int64_t head_dim) {
  int64_t bytes = 0;
  const int rc = guarded([&]() -> int {
    rows_sizes(batch, tokens, q_heads, heads, head_dim, 0);
    need(keys >= 0 && keys <= kMost, TC_E_RANGE, "more than 2^30 keys");
    if (batch && tokens && q_heads) bytes = prompt_shape(batch, tokens, keys, q_heads, heads, head_dim).bytes;
    return TC_OK;
  });
  return rc == TC_OK ? bytes : rc;
}

int64_t tc_paged_tree_attention_workspace(int64_t batch, int64_t tokens, int64_t q_heads, int64_t heads, int64_t head_dim,
                                          int64_t max_len) {
  int64_t bytes = 0;
  const int rc = guarded([&]() -> int {
    rows_sizes(batch, tokens, q_heads, heads, head_dim, max_len);
    bytes = tc::rows_workspace(batch, tokens, heads, q_heads / heads, head_dim, max_len);
    return TC_OK;
  });
  return rc == TC_OK ? bytes : rc;
}

int tc_paged_tree_attention(const tc_paged_cache* cache, const void* q, const tc_layout* q_layout, void* out,
                            const tc_layout* out_layout, int dtype, const int32_t* block_table, const tc_layout* table_layout,
                            const int32_t* seq_lens, const int32_t* token_starts, const int64_t* masks, int64_t max_len, float scale,
                            float* lse, const tc_layout* lse_layout, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const int eb = float_bytes(dtype);
    const Pool p = pool_of("cache", cache, false);
    if (p.dtype != TC_E4M3 && p.dtype != dtype) refuse(TC_E_DTYPE, "q and cache differ in type");
    tc::RowsArgs a{};
    const Queries c = queries_of(q, q_layout, out, out_layout, eb, scale, lse, lse_layout, &a);
    const int64_t tokens = c.q.e[0], q_heads = c.q.e[1];
    need(c.q.e[2] == p.dim, TC_E_EXTENT, "q and the cache differ in head_dim");
    Operand t;
    a.table = table_of("block_table", block_table, table_layout, &t);
    const int64_t batch = t.e[0], group = q_heads / p.heads;
    rows_sizes(batch, tokens, q_heads, p.heads, p.dim, max_len);
    const Operand lens = vector_of("seq_lens", seq_lens, batch), starts = vector_of("token_starts", token_starts, batch + 1);
    Operand mo{};
    mo.empty = true;
    if (masks) {
      tc_layout l{};
      l.rank = 1, l.shape[0] = tokens, l.stride[0] = 1;
      mo = operand("masks", masks, &l, 1, 8);
    }
    if (c.q.empty || batch == 0) return TC_OK;
    const tc::RowsShape shape = tc::rows_shape(true, p.dtype == TC_E4M3, batch, tokens, p.heads, group, p.dim, max_len);
    const Operand work = workspace_of(workspace, workspace_bytes, shape, p.dim, &a);
    const Operand* outs[] = {&c.o, &c.l, &work};
    for (const Operand* x : outs)
      if (touches(p, *x)) refuse(TC_E_ALIAS, "the cache overlaps an output");
    apart_from_inputs(outs, 3, Operands{&c.q, &t, &lens, &starts, &mo});
    a.pool = p.p;
    a.lens = reinterpret_cast<const int32_t*>(lens.p);
    a.starts = reinterpret_cast<const int32_t*>(starts.p);
    a.masks = masks ? reinterpret_cast<const int64_t*>(mo.p) : nullptr;
    a.batch = int32_t(batch);
    a.causal = 1;
    // no row past the table's columns, and none of an empty pool
    a.max_len = int32_t(t.empty || p.empty ? 0 : std::min<int64_t>(max_len, int64_t(a.table.cols) * p.page_size));
    dealt(&a, shape, p.heads, group);
    return launched(tc::launch_tree_attention(a, shape, dtype, p.dtype, stream));
  });
}

int tc_paged_resize(int32_t* block_table, const tc_layout* table_layout, const int32_t* seq_lens, const int32_t* change,
                    int64_t page_size, int32_t* free_pages, int64_t free_capacity, const int32_t* free_count, int32_t* lens_out,
                    int32_t* count_out, int32_t* missing, int32_t* token_starts, int64_t* slots, int32_t* positions, int64_t tokens,
                    void* stream) {
  return guarded([&]() -> int {
    tc::ResizeArgs a{};
    Operand t;
    a.table = table_of("block_table", block_table, table_layout, &t);
    const int64_t batch = t.e[0];
    need(page_size >= 1 && page_size <= INT32_MAX, TC_E_EXTENT, "page_size must be from 1 to 2^31 - 1");
    need(__int128(batch) * t.e[1] <= INT32_MAX, TC_E_RANGE, "a table of more than 2^31 - 1 entries");
    need(free_capacity >= 0 && free_capacity <= INT32_MAX, TC_E_RANGE, "free_capacity must be from 0 to 2^31 - 1");
    need(tokens >= 0 && tokens <= INT32_MAX, TC_E_RANGE, "tokens must be from 0 to 2^31 - 1");
    if (!t.empty) injective("block_table", t, 2, 4);
    const Operand lens = vector_of("seq_lens", seq_lens, batch), ch = vector_of("change", change, batch);
    const Operand stack = vector_of("free_pages", free_pages, free_capacity), held = vector_of("free_count", free_count, 1);
    const Operand lo = vector_of("lens_out", lens_out, batch), co = vector_of("count_out", count_out, 1);
    Operand mo{}, so{}, po{}, st{};
    mo.empty = so.empty = po.empty = st.empty = true;
    if (missing) mo = vector_of("missing", missing, 1);
    if (token_starts) st = vector_of("token_starts", token_starts, batch + 1);
    need(token_starts || (!slots && !positions), TC_E_NULL, "slots and positions need token_starts");
    if (slots) {
      tc_layout l{};
      l.rank = 1, l.shape[0] = tokens, l.stride[0] = 1;
      so = operand("slots", slots, &l, 1, 8);
    }
    if (positions) po = vector_of("positions", positions, tokens);
    const Operand* written[] = {&t, &stack, &lo, &co, &mo, &st, &so, &po};
    for (const Operand* x : written) {
      apart("an output and change", *x, ch);
      // the lengths and the count may be updated in place
      if (x != &lo || lo.p != lens.p) apart("an output and seq_lens", *x, lens);
      if (x != &co || co.p != held.p) apart("an output and free_count", *x, held);
      for (const Operand* y : written)
        if (x != y) apart("two outputs", *x, *y);
    }
    const auto i32 = [](const Operand& o) { return o.empty ? nullptr : reinterpret_cast<int32_t*>(o.p); };
    if (t.empty) a.table.cols = 0;
    a.table_out = i32(t);
    a.lens = i32(lens);
    a.change = i32(ch);
    a.free_pages = i32(stack);
    a.free_count = i32(held);
    a.lens_out = i32(lo);
    a.count_out = i32(co);
    a.missing = i32(mo);
    a.starts = i32(st);
    a.slots = so.empty ? nullptr : reinterpret_cast<int64_t*>(so.p);
    a.positions = i32(po);
    a.capacity = int32_t(free_capacity);
    a.tokens = slots || positions ? int32_t(tokens) : 0;
    a.page = tc::make_div32(uint32_t(page_size));
    return launched(tc::launch_paged_resize(a, stream));
  });
}

}  // extern "C"
