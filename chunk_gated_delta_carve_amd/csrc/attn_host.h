// What the host sides of the attention layer's entry points share: rows and cache
// entries that may overlap, the checks of sequences and strides, launch sizes.
#pragma once
#include <algorithm>
#include <cfloat>

#include "host.h"
#include "kernels/rope.h"

namespace carve_host {

constexpr int64_t kMaxInt = 0x7fffffffLL;
constexpr int64_t kMaxThreads = 0xffffffffLL;                // of a launch, in x
constexpr int64_t kMaxTokens = kMaxThreads / 256 * 4;        // a wave each, in workgroups of 256

inline bool off16(int64_t stride, int dtype) { return (stride * (int64_t)elem_bytes(dtype)) & 15; }

// Rows of `len` elements, `row` apart.
struct Rows {
  const void* p;
  int64_t n, row, len;
  size_t es;
  size_t span() const { return p && n > 0 ? (size_t)((n - 1) * row + len) * es : 0; }
};

inline bool same(const Rows& a, const Rows& b) {
  return a.p == b.p && a.n == b.n && a.len == b.len && (a.row == b.row || a.n == 1);
}

// Whether two sets of rows share an element. Rows of one stride may interleave
// (the parts of one projection's output).
inline bool overlaps(const Rows& a, const Rows& b) {
  if (!carve_host::overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.row != b.row || a.es != b.es || a.row <= 0) return true;
  const int64_t R = a.row * (int64_t)a.es, la = a.len * (int64_t)a.es, lb = b.len * (int64_t)b.es;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % R;
  if (d < 0) d += R;
  return d < la || d + lb > R;
}

// eps carries a row of zeros through the inverse root, which takes denormals as 0.
inline bool bad_eps(float eps) { return !(eps >= FLT_MIN); }

inline bool bad_rot(int rot, int d) { return rot < 0 || rot > d || rot % 16; }

inline bool bad_rows(int64_t n, int64_t row, int64_t len, int dtype, bool written) {
  return row < 0 || (written && n > 1 && row < len) || off16(row, dtype);
}

inline int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename F>
hipError_t by_type(int dtype, int d, F&& f) {
  if (dtype == CARVE_BF16)
    return d == 64 ? f(carve::bf16{}, std::integral_constant<int, 64>{})
                   : f(carve::bf16{}, std::integral_constant<int, 128>{});
  return d == 64 ? f(float{}, std::integral_constant<int, 64>{}) : f(float{}, std::integral_constant<int, 128>{});
}

constexpr int64_t kFewWaves = 4096;   // four waves per SIMD

// Pieces per lane of the kernels that take a token's rows by waves. Few waves: one
// piece each, for the shortest chain (64 tokens of 18 heads of 128: 3.6 us against 5.3). Many:
// up to four, which shares the token's angles and keeps four loads in flight, in
// the fewest waves per token.
struct TokenWaves { int per_lane; unsigned per_token; };
inline TokenWaves token_waves(int64_t tokens, int64_t heads, int d, int dtype) {
  const int64_t passes = up(heads * (d * (int64_t)elem_bytes(dtype) / 16), 64);
  if (passes * tokens <= kFewWaves) return {1, (unsigned)passes};
  const int64_t waves = up(passes, carve::kRopePieces);
  return {(int)up(passes, waves), (unsigned)waves};
}
template <typename F>
hipError_t by_pieces(int n, F&& f) {
  switch (n) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

inline int shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

// What every call over paged sequences has to have, whatever its caches hold.
inline int check_sequences(const carve_paged_config* c) {
  if (!c) return CARVE_EINVAL;
  if (c->N < 0 || c->S < 0 || c->Hq < 0 || c->Hk < 0 || c->page_size < 1 || c->pages < 0 || c->width < 0 ||
      c->rot < 0 || c->table_len < 0 || c->window < 0)
    return CARVE_EINVAL;
  if (c->dtype != CARVE_F32 && c->dtype != CARVE_BF16) return CARVE_EINVAL;
  if (c->flags & ~(CARVE_ROPE_INTERLEAVED | CARVE_ROPE_NORM | CARVE_PAGED_STEP)) return CARVE_EINVAL;
  if ((c->flags & CARVE_PAGED_STEP) && c->N != c->S) return CARVE_EINVAL;
  if (c->d != 64 && c->d != 128) return CARVE_EUNSUPPORTED;
  if (c->page_size & (c->page_size - 1)) return CARVE_EUNSUPPORTED;
  if ((int64_t)c->width * c->page_size > (1 << 30)) return CARVE_EUNSUPPORTED;
  const int64_t heads = (int64_t)c->Hq + 2 * (int64_t)c->Hk;
  if (heads * c->d > kMaxInt || (int64_t)c->N * heads > kMaxInt) return CARVE_EUNSUPPORTED;
  for (int64_t r : {c->q_row, c->k_row, c->v_row, c->o_row, c->table_row})
    if (r > kMaxInt) return CARVE_EUNSUPPORTED;
  if (c->q_row < 0 || c->k_row < 0 || c->v_row < 0 || c->o_row < 0 || c->table_row < 0 ||
      (c->S > 1 && c->table_row < c->width))
    return CARVE_EINVAL;
  return CARVE_OK;
}

// A cache's entries: strides and length in elements of `es` bytes.
struct Entries { int64_t page, tok, head, len, es; };

inline int check_strides(const carve_paged_config* c, const Entries& e) {
  if (e.page < 0 || e.tok < 0 || e.head < 0) return CARVE_EINVAL;
  for (int64_t n : {e.page, e.tok, e.head})
    if (n > kMaxInt) return CARVE_EUNSUPPORTED;   // a stride's bytes are counted in 32 bits (bf16)
  if ((c->pages > 1 && e.page < e.len) || (c->page_size > 1 && e.tok < e.len) || (c->Hk > 1 && e.head < e.len))
    return CARVE_EINVAL;
  return CARVE_OK;
}

// Whether two entries of a cache may share channels: ordered by stride, every
// dimension has to step past all that the ones before it reach.
inline bool entries_overlap(const carve_paged_config* c, const Entries& e) {
  struct Dim { int64_t n, stride; } dims[3] = {{c->pages, e.page}, {c->page_size, e.tok}, {c->Hk, e.head}};
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  int64_t reach = e.len;
  for (const Dim& x : dims) {
    if (x.n < 2) continue;
    if (x.stride < reach) return true;
    reach += (x.n - 1) * x.stride;
  }
  return false;
}

// Whether an entry of cache a and one of cache b (elements of the same size) share
// channels, where both have the same strides (each past what the smaller ones reach,
// as entries_overlap saw to): the distance of the two starts is then looked for among
// the distances of entries, from the largest stride down. Caches that interleave with
// different strides are the caller's to keep apart.
inline bool entries_meet(const carve_paged_config* c, const void* a, const Entries& ea, const void* b,
                         const Entries& eb) {
  struct Dim { int64_t n, a, b; } dims[3] = {{c->pages, ea.page, eb.page}, {c->page_size, ea.tok, eb.tok},
                                             {c->Hk, ea.head, eb.head}};
  const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / ea.es;
  auto same_place = [&](int64_t n) { return n < ea.len && n > -eb.len; };
  for (const Dim& x : dims)
    if (x.n < 1) return false;
  if (same_place(apart)) return true;               // the first entries
  for (const Dim& x : dims)
    if (x.n > 1 && x.a != x.b) return false;
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return (x.n > 1 ? x.a : 0) > (y.n > 1 ? y.a : 0); });
  auto meets = [&](auto&& self, int i, int64_t left) -> bool {
    if (i == 3 || dims[i].n < 2) return same_place(left);
    const int64_t s = dims[i].a, q = left / s;
    for (int64_t m = q - 1; m <= q + 1; ++m)
      if (m < dims[i].n && m > -dims[i].n && self(self, i + 1, left - m * s)) return true;
    return false;
  };
  return meets(meets, 0, apart);
}

inline size_t cache_span(const carve_paged_config* c, const Entries& e) {
  if (c->pages == 0 || c->Hk == 0) return 0;
  return (size_t)((c->pages - 1) * e.page + (c->page_size - 1) * e.tok + (c->Hk - 1) * e.head + e.len) * e.es;
}

}  // namespace carve_host
