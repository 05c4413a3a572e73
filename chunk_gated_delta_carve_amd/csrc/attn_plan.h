// Kernel and split of an attention call, from sizes alone, and the launches that a
// cache of either kind shares.
#pragma once
#include "attn_host.h"
#include "kernels/paged_attn.h"

namespace carve_host {

// The row kernel takes fp32 and, in bf16, batches whose sequences average at most
// `rows_long` rows (tokens x grouped heads; one tile of it has 16), or `rows_short`
// where their tables or the window hold fewer than `long_keys` keys, which is too short
// to pay for the tile kernels' start.
// Tiles have 128 rows (four waves) at d = 64. At d = 128 they have 256 (eight) where
// those occupy more than half of the CUs, and 128 otherwise, two workgroups to a CU:
// twice as many parts to spread, fewer rows wasted in a sequence's last tile, a
// shorter start. With 256 and 128 rows, all launches, heads of 128 in bf16: 64 tokens of
// 16 on 2 heads over 4096 keys 27 and 23 us, 8 times 128 tokens of 16 on 4 over 4096 keys
// 93 and 85, 256 tokens over 32768 keys 123 and 118; 22 times 100 tokens of 16 on 2 over
// 3600 keys, 180 tiles of 256 rows, 134 and 144.
constexpr int kTileSplits = 128;
constexpr int kCUs = 256;
constexpr int64_t kManyRows = 16384;   // rows to join: eight to a wave are two waves per SIMD
constexpr int kWideJoin = 32;          // shares per item from which a workgroup joins a row, not a wave
struct Choice {
  int per_cu;                // row kernel: workgroups that a CU holds
  int more;                  // and blocks that an item counts for beside its own
  int whole;                 // and blocks up to which items are dealt undivided, twice that where they fill the CUs; 0: never
  int rows_short, rows_long, long_keys;
};
struct Plan {
  bool tile, whole;
  int waves;                 // tile kernels: of a workgroup
  int64_t tiles, most;       // row kernel: blocks of keys at most, over all items
  int splits, shares;
  int64_t rows;              // partial results
  int64_t bytes;
};

inline Plan plan_attention(const carve_paged_config* c, const Choice& ch) {
  Plan p{};
  if (c->N == 0 || c->S == 0 || c->Hk == 0 || c->Hq == 0) return p;
  const int64_t G = c->Hq / c->Hk;
  const bool step = (c->flags & CARVE_PAGED_STEP) != 0;
  int64_t keys = (int64_t)c->width * c->page_size;
  const int64_t seen = c->window > 0 && c->window < keys ? c->window : keys;
  p.tile = c->dtype == CARVE_BF16 && (int64_t)c->N * G > (int64_t)(seen < ch.long_keys ? ch.rows_short : ch.rows_long) * c->S;
  auto tiles = [&](int BM) { return step ? c->S * up(G, BM) : up((int64_t)c->N * G, BM) + c->S - 1; };
  p.waves = c->d == 128 && 2 * tiles(256) * c->Hk > kCUs ? 8 : 4;
  const int BM = p.tile ? 32 * p.waves : 16, BN = p.tile ? 64 : 128;
  p.tiles = tiles(BM);
  if (c->window > 0 && keys > (int64_t)c->window + BM + BN) keys = (int64_t)c->window + BM + BN;
  if (p.tile) {
    // four waves: as many workgroups as the CUs hold at once; eight fill them with a tile each
    const int64_t most = up(keys, (int64_t)BN * 4);
    int64_t s = p.waves == 8 ? 1 : kCUs * (c->d == 64 ? 4 : 2) / (p.tiles * c->Hk);
    s = s < most ? s : most;
    s = s < kTileSplits ? s : kTileSplits;
    p.splits = s < 1 ? 1 : (int)s;
    p.rows = p.splits > 1 ? (int64_t)p.splits * c->N * c->Hq : 0;
  } else {
    // a workgroup per block of keys at most; no item has more blocks than this counts
    const int64_t items = p.tiles * c->Hk, nb = up(keys, BN) + 1;
    const int64_t want = std::min(kCUs * ch.per_cu, carve::kMostNotes);
    p.whole = ch.whole > 0 && nb - 1 <= (items >= kCUs ? 2 : 1) * ch.whole;     // (a table without pages has no blocks)
    p.most = items * (p.whole ? 1 : nb + ch.more);
    p.shares = (int)(p.most < want ? p.most : want);
    p.rows = p.shares > 1 && !p.whole ? 2 * (int64_t)p.shares * BM : 0;
  }
  const int64_t cuts = p.rows == 0 ? 0 : p.tile ? p.tiles * c->Hk : p.shares;
  p.bytes = (p.rows * (c->d + 2) + cuts * carve::kCutInts) * 4;
  return p;
}

// Calls larger than the launches take.
inline int check_plan(const carve_paged_config* c, const Plan& p) {
  if (p.tile && p.tiles * p.splits * c->Hk > kMaxThreads / (64 * p.waves)) return CARVE_EUNSUPPORTED;
  if (p.most > kMaxInt) return CARVE_EUNSUPPORTED;
  return CARVE_OK;
}

template <typename W, int WAVES>
constexpr auto tile_kernel() {
  if constexpr (WAVES == 8) return carve::paged_step_kernel<W>;
  else return carve::paged_tile_kernel<W>;
}

template <typename W, int WAVES>
hipError_t launch_tile_kernel(const typename W::Args& a, hipStream_t s) {
  using LY = typename W::LY;
  constexpr int D = W::D;
  constexpr auto kern = tile_kernel<W, WAVES>();
  hipError_t e = set_lds<kern>(LY::bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)a.tiles * a.splits * a.Hk)), dim3(LY::NT), LY::bytes, s, a);
  e = hipGetLastError();
  if constexpr (WAVES == 4) {
    if (e != hipSuccess || a.splits == 1) return e;
    const unsigned tiles = a.tiles * a.Hk;
    const carve::PagedArgs& rows = a;
    if (a.splits > carve::kFewShares || (int64_t)a.N * a.Hq < kManyRows)
      hipLaunchKernelGGL((carve::paged_tile_combine_kernel<D, 1>), dim3(tiles, LY::BM / 4), dim3(256), 0, s, rows);
    else
      hipLaunchKernelGGL((carve::paged_tile_combine_kernel<D, 8>), dim3(tiles, LY::BM / 32), dim3(256), 0, s, rows);
    e = hipGetLastError();
  }
  return e;
}

// The tile kernels over blocks that Tiles<D, waves, WIDE> loads.
template <template <int, int, bool> class Tiles, int D, bool WIDE, typename Args>
hipError_t launch_tiles(const Args& a, const Plan& plan, hipStream_t s) {
  if constexpr (D == 128)
    if (plan.waves == 8) return launch_tile_kernel<Tiles<D, 8, WIDE>, 8>(a, s);
  return launch_tile_kernel<Tiles<D, 4, WIDE>, 4>(a, s);
}

// Joins the row kernel's partial results.
template <typename E, int D>
hipError_t join_rows(const carve::PagedArgs& a, hipStream_t s) {
  constexpr int BM = carve::RowsLayout<E, D>::BM;
  const int64_t most = (a.cu ? a.N : 1) * (int64_t)a.G;      // rows of an item
  const int rows = (int)(most < BM ? most : BM);
  const int64_t items = a.Hk * (up((int64_t)a.N * a.G, BM) > a.S ? up((int64_t)a.N * a.G, BM) : a.S);
  if (a.shares >= kWideJoin * items)
    hipLaunchKernelGGL((carve::paged_rows_combine_kernel<E, D, 4>), dim3(a.tiles * a.Hk, rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((carve::paged_rows_combine_kernel<E, D, 1>), dim3(a.shares, up(rows, 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace carve_host
