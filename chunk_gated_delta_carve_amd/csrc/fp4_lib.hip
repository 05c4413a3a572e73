// Host side of the 4-bit paged cache's entry points and of the room in a paged
// cache: validation, plan, dispatch. Every check runs before the first HIP call.
#include "attn_plan.h"
#include "kernels/assign.h"
#include "kernels/fp4.h"
#include "kernels/paged_fp4.h"

namespace {

using namespace carve_host;

// The four parts of the cache: codes and scales of keys and of values.
struct Parts { Entries kc, ks, vc, vs; };
Parts parts_of(const carve_fp4_config* f) {
  const carve_paged_config& c = f->paged;
  return {{c.kc_page, c.kc_tok, c.kc_head, c.d / 2, 1},
          {f->ks_page, f->ks_tok, f->ks_head, c.d / carve::kFp4Block, 1},
          {c.vc_page, c.vc_tok, c.vc_head, c.d / 2, 1},
          {f->vs_page, f->vs_tok, f->vs_head, c.d / carve::kFp4Block, 1}};
}

int check_fp4(const carve_fp4_config* f) {
  const int st = check_sequences(f ? &f->paged : nullptr);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = f->paged;
  const Parts p = parts_of(f);
  for (const Entries& e : {p.kc, p.ks, p.vc, p.vs}) {
    const int bad = check_strides(&c, e);
    if (bad != CARVE_OK) return bad;
  }
  for (const Entries& e : {p.kc, p.vc})
    if ((e.page | e.tok | e.head) & 15) return CARVE_EALIGN;
  for (const Entries& e : {p.ks, p.vs})
    if ((e.page | e.tok | e.head) & (e.len - 1)) return CARVE_EALIGN;
  for (int64_t r : {c.q_row, c.k_row, c.v_row, c.o_row})
    if (off16(r, c.dtype)) return CARVE_EALIGN;
  return CARVE_OK;
}

carve::Fp4Strides strides(const Entries& e) { return {e.page, e.tok, e.head}; }

}  // namespace

extern "C" int carve_paged_append_fp4(const carve_fp4_config* cfg, const void* k, const void* v, const void* q,
                                      const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                                      const int32_t* cu, const int32_t* kv_lens, const int32_t* table,
                                      uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                                      void* q_out, void* stream) {
  const int st = check_fp4(cfg);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = cfg->paged;
  const bool step = (c.flags & CARVE_PAGED_STEP) != 0, norm = (c.flags & CARVE_ROPE_NORM) != 0;
  if (bad_rot(c.rot, c.d)) return CARVE_EUNSUPPORTED;
  if (norm && bad_eps(c.eps)) return CARVE_EINVAL;
  if (c.N > kMaxTokens) return CARVE_EUNSUPPORTED;
  const Parts parts = parts_of(cfg);
  const Entries kinds[4] = {parts.kc, parts.ks, parts.vc, parts.vs};
  for (const Entries& e : kinds)
    if (entries_overlap(&c, e)) return CARVE_EINVAL;
  if (!norm && (q_weight || k_weight)) return CARVE_EINVAL;
  const void* const caches[4] = {k_codes, k_scales, v_codes, v_scales};
  const bool work = c.N > 0 && c.S > 0 && c.Hq + c.Hk > 0;
  if (work) {
    if (c.Hk > 0 && (!k || !v)) return CARVE_EINVAL;
    if (c.Hk > 0 && c.pages > 0)
      for (const void* p : caches)
        if (!p) return CARVE_EINVAL;
    if (c.Hq > 0 && (!q || !q_out)) return CARVE_EINVAL;
    if (!kv_lens || (c.width > 0 && !table) || (!step && !cu)) return CARVE_EINVAL;
    if (c.rot > 0 && (!cos || !sin)) return CARVE_EINVAL;
  }
  for (const void* p : {k, v, q, q_weight, k_weight, (const void*)cos, (const void*)sin, (const void*)k_codes,
                        (const void*)v_codes, (const void*)q_out})
    if (misaligned(p)) return CARVE_EALIGN;
  for (const void* p : {(const void*)cu, (const void*)kv_lens, (const void*)table, (const void*)k_scales,
                        (const void*)v_scales})
    if (misaligned4(p)) return CARVE_EALIGN;
  const int64_t lq = (int64_t)c.Hq * c.d, lk = (int64_t)c.Hk * c.d;
  if (bad_rows(c.N, c.o_row, lq, c.dtype, true)) return CARVE_EINVAL;
  const size_t es = elem_bytes(c.dtype);
  const Rows rq{q, c.N, c.q_row, lq, es}, ro{q_out, c.N, c.o_row, lq, es};
  const Rows in[] = {{k, c.N, c.k_row, lk, es}, {v, c.N, c.v_row, lk, es},
                     {q_weight, 1, 0, c.d, es}, {k_weight, 1, 0, c.d, es},
                     {cos, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4},
                     {sin, 1, 0, (int64_t)c.table_len * (c.rot / 2), 4},
                     {cu, 1, 0, step ? 0 : (int64_t)c.S + 1, 4}, {kv_lens, 1, 0, c.S, 4},
                     {table, c.S, c.table_row, c.width, 4}};
  if (!same(ro, rq) && overlaps(ro, rq)) return CARVE_EINVAL;
  for (const Rows& r : in)
    if (overlaps(ro, r)) return CARVE_EINVAL;
  // the cache's parts may interleave in one tensor; nothing else lies in them
  for (int i = 0; i < 4; ++i) {
    const size_t span = cache_span(&c, kinds[i]);
    for (const Rows& r : in)
      if (carve_host::overlaps(caches[i], span, r.p, r.span())) return CARVE_EINVAL;
    for (const Rows& r : {rq, ro})
      if (carve_host::overlaps(caches[i], span, r.p, r.span())) return CARVE_EINVAL;
    for (int j = i + 1; j < 4; ++j)
      if (caches[i] && caches[j] && entries_meet(&c, caches[i], kinds[i], caches[j], kinds[j])) return CARVE_EINVAL;
  }
  if (!work) return CARVE_OK;
  carve::Fp4AppendArgs f{};
  carve::AppendArgs& a = f.a;
  a.k = k; a.v = v; a.q = q; a.wq = q_weight; a.wk = k_weight;
  a.cos = cos; a.sin = sin;
  a.cu = step ? nullptr : cu; a.kv_lens = kv_lens; a.table = table;
  a.kc = k_codes; a.vc = v_codes; a.qo = q_out;
  a.k_row = c.k_row; a.v_row = c.v_row; a.q_row = c.q_row; a.qo_row = c.o_row; a.table_row = c.table_row;
  a.kc_page = c.kc_page; a.kc_tok = c.kc_tok; a.kc_head = c.kc_head;
  a.vc_page = c.vc_page; a.vc_tok = c.vc_tok; a.vc_head = c.vc_head;
  a.N = c.N; a.S = c.S; a.Hq = c.Hq; a.Hk = c.Hk; a.rot = c.rot; a.table_len = c.table_len;
  a.width = c.width; a.pages = c.pages; a.page_shift = shift_of(c.page_size);
  a.interleaved = (c.flags & CARVE_ROPE_INTERLEAVED) != 0;
  a.norm = norm;
  a.eps = c.eps;
  f.ks = k_scales; f.vs = v_scales;
  f.k = strides(parts.ks); f.v = strides(parts.vs);
  const TokenWaves w = token_waves(c.N, (int64_t)c.Hq + 2 * (int64_t)c.Hk, c.d, c.dtype);
  if (w.per_token > 65535) return CARVE_EUNSUPPORTED;
  // several tokens to a wave where there are more waves than the GPU holds at once, eight pieces to a lane at most
  const bool run = (int64_t)c.N * w.per_token > kFewWaves;
  const bool turn = c.rot > 0 || norm;
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    return by_pieces(w.per_lane, [&](auto u) {
      constexpr int U = decltype(u)::value, D = decltype(d)::value;
      auto launch = [&](auto tok, auto turned) {
        constexpr int TOK = decltype(tok)::value;
        hipLaunchKernelGGL((carve::paged_append_fp4_kernel<decltype(t), D, U, TOK, decltype(turned)::value>),
                           dim3((unsigned)up(c.N, 4 * TOK), w.per_token), dim3(256), 0,
                           reinterpret_cast<hipStream_t>(stream), f);
        return hipGetLastError();
      };
      auto tokens = [&](auto turned) {
        return run ? launch(std::integral_constant<int, U <= 2 ? 4 : 2>{}, turned)
                   : launch(std::integral_constant<int, 1>{}, turned);
      };
      return turn ? tokens(std::true_type{}) : tokens(std::false_type{});
    });
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}

extern "C" int carve_paged_read_fp4(const carve_fp4_config* cfg, const uint8_t* k_codes, const uint8_t* k_scales,
                                    const uint8_t* v_codes, const uint8_t* v_scales, const int64_t* slots, void* k,
                                    void* v, void* stream) {
  const int st = check_fp4(cfg);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = cfg->paged;
  if (c.N > kMaxTokens) return CARVE_EUNSUPPORTED;
  const int64_t heads = (int64_t)c.Hk * ((k != nullptr) + (v != nullptr));
  const bool work = c.N > 0 && heads > 0;
  if (work && !slots) return CARVE_EINVAL;
  if (work && c.pages > 0 && ((k && (!k_codes || !k_scales)) || (v && (!v_codes || !v_scales)))) return CARVE_EINVAL;
  for (const void* p : {(const void*)k_codes, (const void*)v_codes, (const void*)k, (const void*)v})
    if (misaligned(p)) return CARVE_EALIGN;
  if (misaligned4(k_scales) || misaligned4(v_scales) || (reinterpret_cast<uintptr_t>(slots) & 7u)) return CARVE_EALIGN;
  const int64_t lk = (int64_t)c.Hk * c.d;
  if ((k && bad_rows(c.N, c.k_row, lk, c.dtype, true)) || (v && bad_rows(c.N, c.v_row, lk, c.dtype, true)))
    return CARVE_EINVAL;
  const Parts parts = parts_of(cfg);
  const size_t es = elem_bytes(c.dtype);
  const Rows out[2] = {{k, c.N, c.k_row, lk, es}, {v, c.N, c.v_row, lk, es}};
  const Rows in[5] = {{slots, 1, 0, c.N, 8},
                      {k_codes, 1, 0, (int64_t)cache_span(&c, parts.kc), 1},
                      {k_scales, 1, 0, (int64_t)cache_span(&c, parts.ks), 1},
                      {v_codes, 1, 0, (int64_t)cache_span(&c, parts.vc), 1},
                      {v_scales, 1, 0, (int64_t)cache_span(&c, parts.vs), 1}};
  for (const Rows& o : out)
    for (const Rows& r : in)
      if (overlaps(o, r)) return CARVE_EINVAL;
  if (overlaps(out[0], out[1])) return CARVE_EINVAL;
  if (!work) return CARVE_OK;
  carve::Fp4ReadArgs a{};
  a.kc = k_codes; a.ks = k_scales; a.vc = v_codes; a.vs = v_scales;
  a.slots = slots; a.k = k; a.v = v;
  a.kcs = strides(parts.kc); a.kss = strides(parts.ks); a.vcs = strides(parts.vc); a.vss = strides(parts.vs);
  a.k_row = c.k_row; a.v_row = c.v_row;
  a.entries = (int64_t)c.pages * c.page_size;
  a.N = c.N; a.Hk = c.Hk; a.heads = (int)heads; a.page_shift = shift_of(c.page_size);
  const int64_t blocks = up(c.N * heads * (c.d * (int64_t)es / 16), carve::kReadThreads * carve::kReadPieces);
  if (blocks > kMaxThreads / carve::kReadThreads) return CARVE_EUNSUPPORTED;
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    hipLaunchKernelGGL((carve::paged_read_fp4_kernel<decltype(t), decltype(d)::value>), dim3((unsigned)blocks),
                       dim3(carve::kReadThreads), 0, reinterpret_cast<hipStream_t>(stream), a);
    return hipGetLastError();
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}

namespace {
// Blocks of 128 keys up to which an item is left to one workgroup (twice as many where
// there are items for every CU): splitting it needs a second launch to join the parts.
// Undivided and divided, kernel time of all launches, bf16: 4 heads of 128, 16 sequences
// of 1000 keys 13.6 and 12.5 us (and 3 us of the host's for a launch, which a captured graph
// does not pay: there the second is better), 2000 keys 21.6 and 15.0; 64 of 500 10.6 and
// 15.9, of 2000 23.2 and 24.6, of 4000 42 and 36; 12 heads of 64, 64 of 1000 18.1 and 24.5, of
// 2000 29 and 36, of 200 to 8192 87 and 61.
// The keys are those that the table holds: under a wide one short contexts are divided too.
constexpr int kWhole = 8;

// Rows (tokens x grouped heads) per sequence on average up to which the row kernel is taken:
// a 16-row tile of it opens every block anew, but deals single tokens and chunks evenly
// and leaves no tile half empty. Row and tile kernels a call, heads of 128, 16 on 16, 8 times
// 40 tokens over 3000 to 6000 keys 52 and 171 us, 100 times 80 over 200 to 400 keys 103 and 133,
// 160 tokens 186 and 136; 16 on 4, 2 times 40 over 6000 to 12000 keys 31 and 33, 80 tokens 47
// and 40, 63 single tokens and a chunk of 256 over 200 to 8192 keys 76 and 353, of 2048 324 and
// 362. Heads of 64, 12 on 12, 28 times 40 tokens over 750 to 1500 keys 26 and 45, 100 times 40
// over 200 to 400 keys 34 and 33, 80 tokens 57 and 35; 8 times 80 over 3000 to 6000 keys 47 and
// 48, 160 tokens 79 and 71.
struct Rows16 { int few_keys, many_keys; };
constexpr Rows16 kRows128{128, 128}, kRows64{48, 80};

Plan plan_of(const carve_paged_config* c) {
  const int per_cu = c->d == 128 ? carve::RowsFp4<float, 128>::PER_CU : carve::RowsFp4<float, 64>::PER_CU;   // of bf16 too
  const Rows16 rows = c->d == 128 ? kRows128 : kRows64;
  const Plan p = plan_attention(c, {per_cu, carve::kStart, kWhole, rows.few_keys, rows.many_keys, 2048});
  if (p.most <= kMaxInt) return p;
  // more blocks than the row kernel counts: in bf16 the tile kernels take any number
  return plan_attention(c, {per_cu, carve::kStart, kWhole, 0, 0, 2048});
}

template <typename E, int D>
hipError_t dispatch_attention(const carve::Fp4Args& a, const Plan& plan, hipStream_t s) {
  // rows of one load of a wave in one page, their offsets from its first within 32 bits
  constexpr int WR = carve::Fp4Tiles<D, 4, true>::WR;
  const bool wide = (1 << a.page_shift) >= WR && (WR - 1) * std::max(a.kc_tok, a.vc_tok) + D / 2 <= 0xffffffffLL &&
                    (WR - 1) * std::max(a.k.tok, a.v.tok) + D / carve::kFp4Block <= 0xffffffffLL;
  if constexpr (sizeof(E) == 2)
    if (plan.tile)
      return wide ? launch_tiles<carve::Fp4Tiles, D, true>(a, plan, s) : launch_tiles<carve::Fp4Tiles, D, false>(a, plan, s);
  const bool runs = a.page_shift >= 4 && 15 * std::max(a.kc_tok, a.vc_tok) + D / 2 <= 0xffffffffLL &&
                    15 * std::max(a.k.tok, a.v.tok) + D / carve::kFp4Block <= 0xffffffffLL;
  if (runs)
    hipLaunchKernelGGL((carve::paged_rows_fp4_kernel<E, D, true>), dim3(a.shares), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((carve::paged_rows_fp4_kernel<E, D, false>), dim3(a.shares), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !a.po ? e : join_rows<E, D>(a, s);
}

int check_attention(const carve_fp4_config* f) {
  const int st = check_fp4(f);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = f->paged;
  if (!(c.scale > 0.f)) return CARVE_EINVAL;
  if (!(c.scale <= 16.f)) return CARVE_EUNSUPPORTED;
  if (c.Hq > 0 && (c.Hk == 0 || c.Hq % c.Hk)) return CARVE_EINVAL;
  return check_plan(&c, plan_of(&c));
}
}  // namespace

extern "C" int carve_paged_workspace_fp4(const carve_fp4_config* cfg, int64_t* bytes) {
  const int st = check_attention(cfg);
  if (st != CARVE_OK) return st;
  if (!bytes) return CARVE_EINVAL;
  *bytes = plan_of(&cfg->paged).bytes;
  return CARVE_OK;
}

extern "C" int carve_paged_attention_fp4(const carve_fp4_config* cfg, const void* q, const uint8_t* k_codes,
                                         const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                                         const int32_t* cu, const int32_t* kv_lens, const int32_t* table, void* o,
                                         float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_attention(cfg);
  if (st != CARVE_OK) return st;
  const carve_paged_config& c = cfg->paged;
  const bool step = (c.flags & CARVE_PAGED_STEP) != 0;
  const bool work = c.N > 0 && c.S > 0 && c.Hq > 0;
  if (work) {
    if (!q || !o || !kv_lens || (!step && !cu) || (c.width > 0 && !table)) return CARVE_EINVAL;
    // keys that do not exist are loaded from page 0 and dropped
    if (c.pages < 1 || !k_codes || !k_scales || !v_codes || !v_scales) return CARVE_EINVAL;
  }
  for (const void* p : {q, (const void*)k_codes, (const void*)v_codes, (const void*)o, (const void*)workspace})
    if (misaligned(p)) return CARVE_EALIGN;
  for (const void* p : {(const void*)cu, (const void*)kv_lens, (const void*)table, (const void*)lse,
                        (const void*)k_scales, (const void*)v_scales})
    if (misaligned4(p)) return CARVE_EALIGN;
  const int64_t lq = (int64_t)c.Hq * c.d;
  if (bad_rows(c.N, c.o_row, lq, c.dtype, true)) return CARVE_EINVAL;
  const Plan plan = plan_of(&c);
  const int64_t need = plan.bytes;
  if (workspace_bytes < (size_t)need) return CARVE_EWORKSPACE;
  if (need > 0 && !workspace) return CARVE_EINVAL;
  const Parts parts = parts_of(cfg);
  const size_t es = elem_bytes(c.dtype);
  const Rows in[] = {{q, c.N, c.q_row, lq, es},
                     {cu, 1, 0, step ? 0 : (int64_t)c.S + 1, 4},
                     {kv_lens, 1, 0, c.S, 4},
                     {table, c.S, c.table_row, c.width, 4},
                     {k_codes, 1, 0, (int64_t)cache_span(&c, parts.kc), 1},
                     {k_scales, 1, 0, (int64_t)cache_span(&c, parts.ks), 1},
                     {v_codes, 1, 0, (int64_t)cache_span(&c, parts.vc), 1},
                     {v_scales, 1, 0, (int64_t)cache_span(&c, parts.vs), 1}};
  const Rows out[] = {{o, c.N, c.o_row, lq, es}, {lse, 1, 0, (int64_t)c.N * c.Hq, 4},
                      {need ? workspace : nullptr, 1, 0, need, 1}};
  for (int i = 0; i < 3; ++i) {
    for (const Rows& r : in)
      if (overlaps(out[i], r)) return CARVE_EINVAL;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(out[i], out[j])) return CARVE_EINVAL;
  }
  if (!work) return CARVE_OK;
  carve::Fp4Args a{};
  a.q = q; a.kc = k_codes; a.vc = v_codes; a.ks = k_scales; a.vs = v_scales;
  a.cu = step ? nullptr : cu; a.kv_lens = kv_lens; a.table = table;
  a.o = o; a.lse = lse;
  a.q_row = c.q_row; a.o_row = c.o_row; a.table_row = c.table_row;
  a.kc_page = c.kc_page; a.kc_tok = c.kc_tok; a.kc_head = c.kc_head;
  a.vc_page = c.vc_page; a.vc_tok = c.vc_tok; a.vc_head = c.vc_head;
  a.k = strides(parts.ks); a.v = strides(parts.vs);
  a.N = c.N; a.S = c.S; a.Hq = c.Hq; a.Hk = c.Hk; a.G = c.Hq / c.Hk;
  a.width = c.width; a.pages = c.pages; a.page_shift = shift_of(c.page_size);
  a.window = c.window;
  a.scale = c.scale; a.c = c.scale * carve::kLog2e;
  a.po = need ? static_cast<float*>(workspace) : nullptr;
  a.pml = need ? a.po + plan.rows * c.d : nullptr;
  a.cuts = need ? reinterpret_cast<int*>(a.pml + plan.rows * 2) : nullptr;
  a.splits = plan.splits; a.tiles = (int)plan.tiles; a.shares = plan.shares; a.whole = plan.whole;
  a.by_g = carve::Divisor(a.G); a.by_hk = carve::Divisor(a.Hk); a.by_hq = carve::Divisor(a.Hq);
  a.by_shares = carve::Divisor(a.shares);
  const hipError_t e = by_type(c.dtype, c.d, [&](auto t, auto d) {
    return dispatch_attention<decltype(t), decltype(d)::value>(a, plan, reinterpret_cast<hipStream_t>(stream));
  });
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}

extern "C" int carve_paged_assign(const carve_assign_config* cfg, const int32_t* kv_lens, const int32_t* new_lens,
                                  const int32_t* done, int32_t* table, int32_t* free_pages, const int32_t* free_count,
                                  int32_t* kv_lens_out, int32_t* cu, int32_t* positions, int64_t* slots,
                                  int32_t* free_count_out, void* stream) {
  if (!cfg) return CARVE_EINVAL;
  const carve_assign_config& c = *cfg;
  if (c.S < 0 || c.N < 0 || c.page_size < 1 || c.width < 0 || c.table_row < 0 || c.capacity < 0 ||
      (c.S > 1 && c.table_row < c.width))
    return CARVE_EINVAL;
  if ((c.page_size & (c.page_size - 1)) || (int64_t)c.width * c.page_size > (1 << 30)) return CARVE_EUNSUPPORTED;
  if (c.table_row > kMaxInt || c.capacity > kMaxInt || (int64_t)c.S * c.width > kMaxInt) return CARVE_EUNSUPPORTED;
  if (!free_count || !cu || !free_count_out) return CARVE_EINVAL;
  if (c.S > 0 && (!kv_lens || !new_lens || !kv_lens_out || (c.width > 0 && !table))) return CARVE_EINVAL;
  if (c.capacity > 0 && !free_pages) return CARVE_EINVAL;
  for (const void* p : {(const void*)kv_lens, (const void*)new_lens, (const void*)done, (const void*)table,
                        (const void*)free_pages, (const void*)free_count, (const void*)kv_lens_out, (const void*)cu,
                        (const void*)positions, (const void*)free_count_out})
    if (misaligned4(p)) return CARVE_EALIGN;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return CARVE_EALIGN;
  const Rows in[] = {{kv_lens, 1, 0, c.S, 4}, {new_lens, 1, 0, c.S, 4}, {done, 1, 0, c.S, 4}, {free_count, 1, 0, 2, 4}};
  const Rows out[] = {{kv_lens_out, 1, 0, c.S, 4}, {free_count_out, 1, 0, 2, 4}, {table, c.S, c.table_row, c.width, 4},
                      {free_pages, 1, 0, c.capacity, 4}, {cu, 1, 0, (int64_t)c.S + 1, 4}, {positions, 1, 0, c.N, 4},
                      {slots, 1, 0, c.N, 8}};
  for (int i = 0; i < 7; ++i) {
    for (const Rows& r : in)
      if (overlaps(out[i], r) && !((i == 0 && kv_lens_out == kv_lens && r.p == kv_lens) ||
                                   (i == 1 && free_count_out == free_count && r.p == free_count)))
        return CARVE_EINVAL;
    for (int j = i + 1; j < 7; ++j)
      if (overlaps(out[i], out[j])) return CARVE_EINVAL;
  }
  carve::AssignArgs a{};
  a.kv_lens = kv_lens; a.new_lens = new_lens; a.done = done; a.free_count = free_count;
  a.table = table; a.free_pages = free_pages; a.kv_out = kv_lens_out; a.cu = cu;
  a.positions = positions; a.count_out = free_count_out; a.slots = slots;
  a.table_row = c.table_row; a.capacity = c.capacity;
  a.S = c.S; a.N = c.N; a.width = c.width; a.page_shift = shift_of(c.page_size);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(carve::paged_assign_kernel, dim3(1), dim3(carve::kAssignThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && (c.N > carve::kAssignTokens || c.S > carve::kAssignThreads) && c.N > 0 && (positions || slots)) {
    hipLaunchKernelGGL(carve::paged_assign_tokens_kernel, dim3((unsigned)up(c.N, 1024)), dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  return e == hipSuccess ? CARVE_OK : hip_failed(e);
}
