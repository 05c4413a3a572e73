// Host side of the attention layer's entry points: validation, plan, dispatch.
// Every check runs before the first HIP call.
#include "attn_plan.h"

namespace {

using namespace carve_host;

Entries k_entries(const carve_paged_config* c) {
  return {c->kc_page, c->kc_tok, c->kc_head, c->d, (int64_t)elem_bytes(c->dtype)};
}
Entries v_entries(const carve_paged_config* c) {
  return {c->vc_page, c->vc_tok, c->vc_head, c->d, (int64_t)elem_bytes(c->dtype)};
}

int check_rope(const carve_rope_config* c) {
  if (!c) return CARVE_EINVAL;
  if (c->N < 0 || c->Hq < 0 || c->Hk < 0 || c->rot < 0 || c->table_len < 0) return CARVE_EINVAL;
  if (c->dtype != CARVE_F32 && c->dtype != CARVE_BF16) return CARVE_EINVAL;
  if (c->flags & ~(CARVE_ROPE_INTERLEAVED | CARVE_ROPE_NORM)) return CARVE_EINVAL;
  if ((c->flags & CARVE_ROPE_NORM) && bad_eps(c->eps)) return CARVE_EINVAL;
  if ((c->d != 64 && c->d != 128) || bad_rot(c->rot, c->d)) return CARVE_EUNSUPPORTED;
  if (c->Hq > kMaxInt / c->d || c->Hk > kMaxInt / c->d) return CARVE_EUNSUPPORTED;
  const int64_t H = c->Hq > c->Hk ? c->Hq : c->Hk;
  if (c->N > kMaxTokens || c->N * H > kMaxInt) return CARVE_EUNSUPPORTED;   // rows are numbered in 32 bits
  for (int64_t r : {c->q_row, c->k_row, c->qo_row, c->ko_row, c->dq_row, c->dk_row})
    if (r > kMaxInt) return CARVE_EUNSUPPORTED;
  return CARVE_OK;
}

// Blocks of the gradient: four per CU share the rows of q and k in proportion,
// each tensor at least one where it has rows.
constexpr int kBwdBlocks = 1024;
void bwd_blocks(const carve_rope_config* c, int* nq, int* nk) {
  const int per = carve::kRopeThreads / (c->d * (int)elem_bytes(c->dtype) / 16);
  const int64_t rq = c->N * c->Hq, rk = c->N * c->Hk;
  int64_t bq = up(rq, per), bk = up(rk, per);
  if (bq + bk > kBwdBlocks) {
    const int64_t s = (kBwdBlocks * rq + rq + rk - 1) / (rq + rk);
    bk = bk < kBwdBlocks - s ? bk : kBwdBlocks - s;
    bk = rk > 0 && bk < 1 ? 1 : bk;
    bq = bq < s ? bq : s;
  }
  *nq = (int)bq; *nk = (int)bk;
}

carve::RopeArgs rope_args(const carve_rope_config* c) {
  carve::RopeArgs a{};
  a.N = c->N;
  a.q_row = c->q_row; a.k_row = c->k_row; a.qo_row = c->qo_row; a.ko_row = c->ko_row;
  a.dq_row = c->dq_row; a.dk_row = c->dk_row;
  a.T = c->T; a.Hq = c->Hq; a.Hk = c->Hk; a.rot = c->rot; a.table_len = c->table_len;
  a.interleaved = (c->flags & CARVE_ROPE_INTERLEAVED) != 0;
  a.norm = (c->flags & CARVE_ROPE_NORM) != 0;
  a.eps = c->eps;
  return a;
}

// What the forward and backward passes check alike.
int check_rope_inputs(const carve_rope_config* c, const void* q, const void* k, const void* wq, const void* wk,
                      const float* cos, const float* sin, const int32_t* positions) {
  if (c->N > 0 && ((c->Hq > 0 && !q) || (c->Hk > 0 && !k))) return CARVE_EINVAL;
  if (c->rot > 0 && c->N > 0 && (!cos || !sin)) return CARVE_EINVAL;
  if (!positions && c->N > 0 && c->T <= 0) return CARVE_EINVAL;
  if (!(c->flags & CARVE_ROPE_NORM) && (wq || wk)) return CARVE_EINVAL;
  for (const void* p : {q, k, wq, wk, (const void*)cos, (const void*)sin})
    if (misaligned(p)) return CARVE_EALIGN;
  if (misaligned4(positions)) return CARVE_EALIGN;
  if (c->q_row < 0 || c->k_row < 0) return CARVE_EINVAL;
  if (off16(c->q_row, c->dtype) || off16(c->k_row, c->dtype)) return CARVE_EALIGN;
  return CARVE_OK;
}

int check_paged(const carve_paged_config* c) {
  const int st = check_sequences(c);
  if (st != CARVE_OK) return st;
  // distinct cache entries lie apart
  for (const Entries& e : {k_entries(c), v_entries(c)}) {
    const int bad = check_strides(c, e);
    if (bad != CARVE_OK) return bad;
  }
  for (int64_t s : {c->kc_page, c->kc_tok, c->kc_head, c->vc_page, c->vc_tok, c->vc_head, c->q_row, c->k_row,
                    c->v_row, c->o_row})
    if (off16(s, c->dtype)) return CARVE_EALIGN;
  return CARVE_OK;
}

// Row or tile kernel. Row and tile kernel, all launches, 4 heads: of 128, 16 sequences
// of 4096 keys with 16 rows 35 and 37 us, 24 rows 44 and 37, 32 rows 45 and 41; 64 of
// 2048 with 32 rows 93 and 78; 4 of 1000 with 32 rows 14 and 18; of 64, 16 of 4096 with
// 32 rows 35 and 27, 4 of 1000 with 32 rows 11 and 15.
Plan plan_of(const carve_paged_config* c) {
  const bool f32 = c->dtype == CARVE_F32;
  const int wide = f32 ? carve::RowsLayout<float, 128>::PER_CU : carve::RowsLayout<carve::bf16, 128>::PER_CU;
  const int slim = f32 ? carve::RowsLayout<float, 64>::PER_CU : carve::RowsLayout<carve::bf16, 64>::PER_CU;
  return plan_attention(c, {c->d == 128 ? wide : slim, 0, 0, 32, 16, 2048});
}

template <typename E, int D>
hipError_t dispatch_attention(const carve::PagedArgs& a, const Plan& plan, hipStream_t s) {
  // rows of one load of a wave in one page, their offsets from its first within 32 bits
  using LY = carve::TileLayout<D, 4>;
  const int64_t reach = (LY::WR - 1) * 2 * std::max(a.kc_tok, a.vc_tok) + LY::CPR * 16;
  const bool wide = a.page_shift >= 3 && reach <= 0xffffffffLL;
  if constexpr (sizeof(E) == 2)
    if (plan.tile)
      return wide ? launch_tiles<carve::PlainTiles, D, true>(a, plan, s)
                  : launch_tiles<carve::PlainTiles, D, false>(a, plan, s);
  hipLaunchKernelGGL((carve::paged_rows_kernel<E, D>), dim3(a.shares), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !a.cuts ? e : join_rows<E, D>(a, s);
}

}  // namespace

extern "C" int carve_qk_norm_rope_fwd(const carve_rope_config* cfg, const void* q, const void* k,
                                      const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                                      const int32_t* positions, void* q_out, void* k_out, void* stream) {
  int st = check_rope(cfg);
  if (st == CARVE_OK) st = check_rope_inputs(cfg, q, k, q_weight, k_weight, cos, sin, positions);
  if (st != CARVE_OK) return st;
  const carve_rope_config& c = *cfg;
  if (c.N > 0 && ((c.Hq > 0 && !q_out) || (c.Hk > 0 && !k_out))) return CARVE_EINVAL;
  if (misaligned(q_out) || misaligned(k_out)) return CARVE_EALIGN;
  const int64_t lq = (int64_t)c.Hq * c.d, lk = (int64_t)c.Hk * c.d;
  if (off16(c.qo_row, c.dtype) || off16(c.ko_row, c.dtype)) return CARVE_EALIGN;
  if (bad_rows(c.N, c.qo_row, lq, c.dtype, true) || bad_rows(c.N, c.ko_row, lk, c.dtype, true)) return CARVE_EINVAL;
  const size_t es = elem_bytes(c.dtype);
  const Rows in[2] = {{q, c.N, c.q_row, lq, es}, {k, c.N, c.k_row, lk, es}};
  const Rows out[2] = {{q_out, c.N, c.qo_row, lq, es}, {k_out, c.N, c.ko_row, lk, es}};
  const Rows side[5] = {{q_weight, 1, 0, c.d, es}, {k_weight, 1, 0, c.d, es},
                        {cos, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4},
                        {sin, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4}, {positions, 1, 0, c.N, 4}};
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 2; ++j)
      if (!(i == j && same(out[i], in[j])) && overlaps(out[i], in[j])) return CARVE_EINVAL;
    for (const Rows& s : side)
      if (overlaps(out[i], s)) return CARVE_EINVAL;
  }
  if (overlaps(out[0], out[1])) return CARVE_EINVAL;
  if (c.N * (c.Hq + (int64_t)c.Hk) == 0) return CARVE_OK;
  carve::RopeArgs a = rope_args(cfg);
  a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight;
  a.cos = cos; a.sin = sin; a.positions = positions;
  a.qo = q_out; a.ko = k_out;
  const TokenWaves w = token_waves(c.N, (int64_t)c.Hq + c.Hk, c.d, c.dtype);
  if (w.per_token > 65535) return CARVE_EUNSUPPORTED;
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    return by_pieces(w.per_lane, [&](auto u) {
      hipLaunchKernelGGL((carve::norm_rope_kernel<decltype(t), decltype(d)::value, decltype(u)::value>),
                         dim3((unsigned)up(c.N, carve::kRopeThreads / 64), w.per_token), dim3(carve::kRopeThreads), 0,
                         reinterpret_cast<hipStream_t>(stream), a);
      return hipGetLastError();
    });
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}

extern "C" int carve_qk_norm_rope_workspace(const carve_rope_config* cfg, int32_t weights, int64_t* bytes) {
  const int st = check_rope(cfg);
  if (st != CARVE_OK) return st;
  if (!bytes) return CARVE_EINVAL;
  int nq, nk;
  bwd_blocks(cfg, &nq, &nk);
  *bytes = weights ? (int64_t)(nq + nk) * cfg->d * 4 : 0;
  return CARVE_OK;
}

extern "C" int carve_qk_norm_rope_bwd(const carve_rope_config* cfg, const void* q, const void* k,
                                      const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                                      const int32_t* positions, const void* d_q_out, const void* d_k_out, void* dq,
                                      void* dk, float* dq_weight, float* dk_weight, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  int st = check_rope(cfg);
  if (st == CARVE_OK) st = check_rope_inputs(cfg, q, k, q_weight, k_weight, cos, sin, positions);
  if (st != CARVE_OK) return st;
  const carve_rope_config& c = *cfg;
  if (c.N > 0 && ((c.Hq > 0 && (!d_q_out || !dq)) || (c.Hk > 0 && (!d_k_out || !dk)))) return CARVE_EINVAL;
  if ((q_weight && !dq_weight) || (k_weight && !dk_weight)) return CARVE_EINVAL;
  if (!q_weight) dq_weight = nullptr;
  if (!k_weight) dk_weight = nullptr;
  for (const void* p : {d_q_out, d_k_out, (const void*)dq, (const void*)dk, (const void*)workspace})
    if (misaligned(p)) return CARVE_EALIGN;
  if (misaligned4(dq_weight) || misaligned4(dk_weight)) return CARVE_EALIGN;
  const int64_t lq = (int64_t)c.Hq * c.d, lk = (int64_t)c.Hk * c.d;
  for (int64_t r : {c.qo_row, c.ko_row, c.dq_row, c.dk_row})
    if (off16(r, c.dtype)) return CARVE_EALIGN;
  if (bad_rows(c.N, c.qo_row, lq, c.dtype, false) || bad_rows(c.N, c.ko_row, lk, c.dtype, false) ||
      bad_rows(c.N, c.dq_row, lq, c.dtype, true) || bad_rows(c.N, c.dk_row, lk, c.dtype, true))
    return CARVE_EINVAL;
  int64_t need = 0;
  carve_qk_norm_rope_workspace(cfg, q_weight || k_weight, &need);
  if (workspace_bytes < (size_t)need) return CARVE_EWORKSPACE;
  if (need > 0 && !workspace) return CARVE_EINVAL;
  const size_t es = elem_bytes(c.dtype);
  // each gradient may be written over its own output gradient or its own input
  const Rows in[2][2] = {{{q, c.N, c.q_row, lq, es}, {d_q_out, c.N, c.qo_row, lq, es}},
                         {{k, c.N, c.k_row, lk, es}, {d_k_out, c.N, c.ko_row, lk, es}}};
  const Rows out[5] = {{dq, c.N, c.dq_row, lq, es}, {dk, c.N, c.dk_row, lk, es}, {dq_weight, 1, 0, c.d, 4},
                       {dk_weight, 1, 0, c.d, 4}, {need ? workspace : nullptr, 1, 0, need, 1}};
  const Rows side[5] = {{q_weight, 1, 0, c.d, es}, {k_weight, 1, 0, c.d, es},
                        {cos, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4},
                        {sin, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4}, {positions, 1, 0, c.N, 4}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 2; ++j)
      for (const Rows& r : in[j])
        if (!(i == j && same(out[i], r)) && overlaps(out[i], r)) return CARVE_EINVAL;
    for (const Rows& s : side)
      if (overlaps(out[i], s)) return CARVE_EINVAL;
    for (int j = i + 1; j < 5; ++j)
      if (overlaps(out[i], out[j])) return CARVE_EINVAL;
  }
  carve::RopeArgs a = rope_args(cfg);
  a.q = q; a.k = k; a.wq = q_weight; a.wk = k_weight;
  a.cos = cos; a.sin = sin; a.positions = positions;
  a.qo = const_cast<void*>(d_q_out); a.ko = const_cast<void*>(d_k_out);
  a.dq = dq; a.dk = dk;
  a.part = need ? static_cast<float*>(workspace) : nullptr;
  int nq, nk;
  bwd_blocks(cfg, &nq, &nk);
  a.blocks_q = nq; a.blocks = nq + nk;
  const bool weights = q_weight || k_weight;
  if (a.blocks == 0 && !weights) return CARVE_OK;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    constexpr int D = decltype(d)::value;
    if (a.blocks > 0) {
      hipLaunchKernelGGL((carve::norm_rope_bwd_kernel<decltype(t), D>), dim3(a.blocks), dim3(carve::kRopeThreads), 0,
                         s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || !weights) return e;
    }
    // without tokens the sums are empty and come out as zeros
    hipLaunchKernelGGL((carve::norm_rope_dw_kernel<D>), dim3(D / carve::kDwCols, 2), dim3(carve::kDwThreads), 0, s,
                       a.part, a.blocks_q, a.blocks, dq_weight, dk_weight);
    return hipGetLastError();
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}

extern "C" int carve_paged_append(const carve_paged_config* cfg, const void* k, const void* v, const void* q,
                                  const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                                  const int32_t* cu, const int32_t* kv_lens, const int32_t* table, void* k_cache,
                                  void* v_cache, void* q_out, void* stream) {
  const int st = check_paged(cfg);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = *cfg;
  const bool step = (c.flags & CARVE_PAGED_STEP) != 0, norm = (c.flags & CARVE_ROPE_NORM) != 0;
  if (bad_rot(c.rot, c.d)) return CARVE_EUNSUPPORTED;
  if (norm && bad_eps(c.eps)) return CARVE_EINVAL;
  if (c.N > kMaxTokens) return CARVE_EUNSUPPORTED;
  if (entries_overlap(cfg, k_entries(cfg)) || entries_overlap(cfg, v_entries(cfg))) return CARVE_EINVAL;
  if (!norm && (q_weight || k_weight)) return CARVE_EINVAL;
  const bool work = c.N > 0 && c.S > 0 && c.Hq + c.Hk > 0;
  if (work) {
    if (c.Hk > 0 && (!k || !v)) return CARVE_EINVAL;
    if (c.Hk > 0 && c.pages > 0 && (!k_cache || !v_cache)) return CARVE_EINVAL;
    if (c.Hq > 0 && (!q || !q_out)) return CARVE_EINVAL;
    if (!kv_lens || (c.width > 0 && !table) || (!step && !cu)) return CARVE_EINVAL;
    if (c.rot > 0 && (!cos || !sin)) return CARVE_EINVAL;
  }
  for (const void* p : {k, v, q, q_weight, k_weight, (const void*)cos, (const void*)sin, (const void*)k_cache,
                        (const void*)v_cache, (const void*)q_out})
    if (misaligned(p)) return CARVE_EALIGN;
  if (misaligned4(cu) || misaligned4(kv_lens) || misaligned4(table)) return CARVE_EALIGN;
  const int64_t lq = (int64_t)c.Hq * c.d, lk = (int64_t)c.Hk * c.d;
  if (bad_rows(c.N, c.o_row, lq, c.dtype, true)) return CARVE_EINVAL;
  const size_t es = elem_bytes(c.dtype);
  const Rows rq{q, c.N, c.q_row, lq, es}, rk{k, c.N, c.k_row, lk, es}, rv{v, c.N, c.v_row, lk, es},
      ro{q_out, c.N, c.o_row, lq, es};
  const size_t ks = cache_span(cfg, k_entries(cfg)), vs = cache_span(cfg, v_entries(cfg));
  const Rows side[] = {{q_weight, 1, 0, c.d, es}, {k_weight, 1, 0, c.d, es},
                       {cos, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4},
                       {sin, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4},
                       {cu, 1, 0, step ? 0 : (int64_t)c.S + 1, 4}, {kv_lens, 1, 0, c.S, 4},
                       {table, c.S, c.table_row, c.width, 4}};
  if (overlaps(ro, rk) || overlaps(ro, rv) || (!same(ro, rq) && overlaps(ro, rq))) return CARVE_EINVAL;
  for (const Rows& r : side)
    if (overlaps(ro, r)) return CARVE_EINVAL;
  // the two caches may interleave in one tensor; nothing else lies in them
  for (const Rows& r : {rq, rk, rv, ro, side[0], side[1], side[2], side[3], side[4], side[5], side[6]})
    if (carve_host::overlaps(k_cache, ks, r.p, r.span()) || carve_host::overlaps(v_cache, vs, r.p, r.span()))
      return CARVE_EINVAL;
  if (k_cache && v_cache && entries_meet(cfg, k_cache, k_entries(cfg), v_cache, v_entries(cfg))) return CARVE_EINVAL;
  if (!work) return CARVE_OK;
  carve::AppendArgs a{};
  a.k = k; a.v = v; a.q = q; a.wq = q_weight; a.wk = k_weight;
  a.cos = cos; a.sin = sin;
  a.cu = step ? nullptr : cu; a.kv_lens = kv_lens; a.table = table;
  a.kc = k_cache; a.vc = v_cache; a.qo = q_out;
  a.k_row = c.k_row; a.v_row = c.v_row; a.q_row = c.q_row; a.qo_row = c.o_row; a.table_row = c.table_row;
  a.kc_page = c.kc_page; a.kc_tok = c.kc_tok; a.kc_head = c.kc_head;
  a.vc_page = c.vc_page; a.vc_tok = c.vc_tok; a.vc_head = c.vc_head;
  a.N = c.N; a.S = c.S; a.Hq = c.Hq; a.Hk = c.Hk; a.rot = c.rot; a.table_len = c.table_len;
  a.width = c.width; a.pages = c.pages; a.page_shift = shift_of(c.page_size);
  a.interleaved = (c.flags & CARVE_ROPE_INTERLEAVED) != 0;
  a.norm = norm;
  a.eps = c.eps;
  const TokenWaves w = token_waves(c.N, (int64_t)c.Hq + 2 * (int64_t)c.Hk, c.d, c.dtype);
  if (w.per_token > 65535) return CARVE_EUNSUPPORTED;
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    return by_pieces(w.per_lane, [&](auto u) {
      hipLaunchKernelGGL((carve::paged_append_kernel<decltype(t), decltype(d)::value, decltype(u)::value>),
                         dim3((unsigned)up(c.N, 4), w.per_token), dim3(256), 0, reinterpret_cast<hipStream_t>(stream),
                         a);
      return hipGetLastError();
    });
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}

namespace {
int check_attention(const carve_paged_config* c) {
  const int st = check_paged(c);
  if (st != CARVE_OK) return st;
  if (!(c->scale > 0.f)) return CARVE_EINVAL;
  if (!(c->scale <= 16.f)) return CARVE_EUNSUPPORTED;
  if (c->Hq > 0 && (c->Hk == 0 || c->Hq % c->Hk)) return CARVE_EINVAL;
  return check_plan(c, plan_of(c));
}
}  // namespace

extern "C" int carve_paged_workspace(const carve_paged_config* cfg, int64_t* bytes) {
  const int st = check_attention(cfg);
  if (st != CARVE_OK) return st;
  if (!bytes) return CARVE_EINVAL;
  *bytes = plan_of(cfg).bytes;
  return CARVE_OK;
}

extern "C" int carve_paged_attention(const carve_paged_config* cfg, const void* q, const void* k_cache,
                                     const void* v_cache, const int32_t* cu, const int32_t* kv_lens,
                                     const int32_t* table, void* o, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const int st = check_attention(cfg);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = *cfg;
  const bool step = (c.flags & CARVE_PAGED_STEP) != 0;
  const bool work = c.N > 0 && c.S > 0 && c.Hq > 0;
  if (work) {
    if (!q || !o || !kv_lens || (!step && !cu) || (c.width > 0 && !table)) return CARVE_EINVAL;
    // keys that do not exist are loaded from page 0 and dropped
    if (c.pages < 1 || !k_cache || !v_cache) return CARVE_EINVAL;
  }
  for (const void* p : {q, k_cache, v_cache, (const void*)o, (const void*)workspace})
    if (misaligned(p)) return CARVE_EALIGN;
  if (misaligned4(cu) || misaligned4(kv_lens) || misaligned4(table) || misaligned4(lse)) return CARVE_EALIGN;
  const int64_t lq = (int64_t)c.Hq * c.d;
  if (bad_rows(c.N, c.o_row, lq, c.dtype, true)) return CARVE_EINVAL;
  const Plan plan = plan_of(cfg);
  if (workspace_bytes < (size_t)plan.bytes) return CARVE_EWORKSPACE;
  if (plan.bytes > 0 && !workspace) return CARVE_EINVAL;
  const size_t es = elem_bytes(c.dtype);
  const Rows in[] = {{q, c.N, c.q_row, lq, es},
                     {cu, 1, 0, step ? 0 : (int64_t)c.S + 1, 4},
                     {kv_lens, 1, 0, c.S, 4},
                     {table, c.S, c.table_row, c.width, 4},
                     {k_cache, 1, 0, (int64_t)cache_span(cfg, k_entries(cfg)), 1},
                     {v_cache, 1, 0, (int64_t)cache_span(cfg, v_entries(cfg)), 1}};
  const Rows out[] = {{o, c.N, c.o_row, lq, es}, {lse, 1, 0, (int64_t)c.N * c.Hq, 4},
                      {plan.bytes ? workspace : nullptr, 1, 0, plan.bytes, 1}};
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (overlaps(out[i], r)) return CARVE_EINVAL;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(out[i], out[j])) return CARVE_EINVAL;
  }
  if (!work) return CARVE_OK;
  carve::PagedArgs a{};
  a.q = q; a.kc = k_cache; a.vc = v_cache;
  a.cu = step ? nullptr : cu; a.kv_lens = kv_lens; a.table = table;
  a.o = o; a.lse = lse;
  a.po = static_cast<float*>(workspace);
  a.pml = plan.bytes ? a.po + plan.rows * c.d : nullptr;
  a.cuts = plan.bytes ? reinterpret_cast<int*>(a.pml + plan.rows * 2) : nullptr;
  a.q_row = c.q_row; a.o_row = c.o_row; a.table_row = c.table_row;
  a.kc_page = c.kc_page; a.kc_tok = c.kc_tok; a.kc_head = c.kc_head;
  a.vc_page = c.vc_page; a.vc_tok = c.vc_tok; a.vc_head = c.vc_head;
  a.N = c.N; a.S = c.S; a.Hq = c.Hq; a.Hk = c.Hk; a.G = c.Hq / c.Hk;
  a.width = c.width; a.pages = c.pages; a.page_shift = shift_of(c.page_size);
  a.window = c.window;
  a.splits = plan.splits; a.tiles = (int)plan.tiles; a.shares = plan.shares;
  a.by_g = carve::Divisor(a.G); a.by_hk = carve::Divisor(a.Hk); a.by_hq = carve::Divisor(a.Hq);
  a.by_shares = carve::Divisor(a.shares);
  a.scale = c.scale; a.c = c.scale * carve::kLog2e;
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    return dispatch_attention<decltype(t), decltype(d)::value>(a, plan, reinterpret_cast<hipStream_t>(stream));
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}
