// Attention of new tokens over a paged cache.
//
// Sequence s has kv tokens, the last n of them new. New token i stands at
// p = kv - n + i and sees the keys j in (p - window, p] (all j <= p without a
// window). Query head h reads key/value head h / G, G = Hq / Hk, so the rows of
// one key/value head are the (token, head in group) pairs r = i G + g, and a
// tile of rows shares every key and value it loads.
//
//   o_r = sum_j e^{c (x_rj - m)} v_j / l,  l = sum_j e^{c (x_rj - m)},  x_rj = q_r . k_j
//
// in one pass over the keys: m is a running reference near the row maximum (in
// fp32, as l and o are), and the exponentials are powers of two with
// c = scale log2 e. Products run transposed, X^T = K Q^T and O^T = V^T P^T: a
// lane then owns one row (a column of the C tile), its maximum needs one or two
// cross-lane steps, rescaling is lane-local, and P^T leaves the first product
// in the very registers the second one wants as its B operand. In bf16 P has to be
// rounded for that: with few rows it goes in as two parts of 8 bits each (free
// beside the loads), with many as one, off by at most 2^-8 of each weight (a
// second product would cost a third of the matrix time); l sums it unrounded.
//
// Masked keys never reach a row: their scores are replaced before use, pages
// outside the cache and keys no row of the tile may see are loaded as zeros,
// and a row whose result is not finite is computed again over its visible keys
// alone (careful_row), since 0 x inf inside a product that other rows need
// would have put a NaN there. So is a row whose scores are too large for one pass.
//
// Where rows are few, long contexts are split over workgroups, each leaving
// (o, m, l) in fp32; a second kernel joins them in a fixed order. How many a tile
// needs is worked out from its own key range on the device, so no length is read
// on the host and a captured graph follows the lengths there.
#pragma once
#include "common.h"
#include "rope.h"

namespace carve {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct PagedArgs {
  const void *q, *kc, *vc;
  const int *cu, *kv_lens, *table;
  void* o;
  float* lse;                                       // [N][Hq] or NULL
  float *po, *pml;                                  // partial results (o, and m with l)
  int* cuts;                                        // notes on items with partial results
  int64_t q_row, o_row, table_row;
  int64_t kc_page, kc_tok, kc_head, vc_page, vc_tok, vc_head;
  int N, S, Hq, Hk, G, width, pages, page_shift, window;
  int tiles, splits;                                // tile kernel: tiles, workgroups per tile at most
  int shares;                                       // row kernel: workgroups that the work is dealt to
  float scale, c;                                   // c = scale log2 e
};

// The reference m of a row follows its maximum only when that has grown by more
// than 2^kSlack: the weights then stay below 2^kSlack (harmless in fp32 and in
// bf16, whose relative step is the same everywhere) and most blocks spare the
// rescaling of o.
constexpr float kSlack = 8.f;
constexpr float kNoMax = -1e37f;                    // where m starts: c kNoMax stays finite (c < 24)
constexpr float kLeast = -3.4028234663852886e38f;   // m of a row without weights: no finite score lies below

// The weights of a row that sees keys sum to about 1 or more (its maximum's own) and
// to less than keys 2^kSlack. Outside of these bounds the sum tells nothing: scores
// below kNoMax leave no weights, and from scores of about 2^24 / c on, the exponent
// c x - c m holds the rounding of c m, which may be any number. Such a row is computed
// again by careful_row, which forms c (x - m).
constexpr float kLeastSum = 0x1p-20f, kMostSum = 0x1p60f;
__device__ __forceinline__ bool odd_sum(float l) {   // 0, which rows that see nothing have, apart
  return !(l >= kLeastSum && l <= kMostSum) && l != 0.f;
}

// The tile `t` of BM rows: its sequence, its rows and the keys they see.
struct AttnTile {
  int n0;                                           // the sequence's first token
  int row0, rows;                                   // first row in the sequence, rows in the tile (0: nothing to do)
  int s, pos0;                                      // sequence, position of its first new token
  int lo, hi;                                       // keys some row may see
};

__device__ __forceinline__ int first_position(const PagedArgs& a, int s, int cnt) {
  const int kv = a.kv_lens[s];
  return (kv > 0 ? kv : 0) - cnt;
}

__device__ __forceinline__ AttnTile tile_of_rows(const PagedArgs& a, int s, int n0, int cnt, int pos0, int row0,
                                                 int BM) {
  AttnTile x;
  x.s = s; x.n0 = n0; x.row0 = row0; x.pos0 = pos0;
  const int all = cnt * a.G;
  x.rows = all - row0 < BM ? all - row0 : BM;
  const int64_t cap = (int64_t)a.width << a.page_shift;
  const int64_t first = (int64_t)x.pos0 + row0 / a.G, last = (int64_t)x.pos0 + (row0 + x.rows - 1) / a.G;
  const int64_t hi = last + 1 < cap ? last + 1 : cap;
  const int64_t lo = a.window > 0 && first - a.window + 1 > 0 ? first - a.window + 1 : 0;
  x.hi = hi > 0 ? (int)hi : 0;
  x.lo = lo < x.hi ? (int)lo : x.hi;
  return x;
}

// Tiles are numbered without knowing the lengths: sequence s starts at tile
// floor(cu[s] G / BM) + s, which leaves room for its ceil(n G / BM) tiles.
__device__ __forceinline__ AttnTile find_tile(const PagedArgs& a, int t, int BM) {
  AttnTile none;
  none.rows = 0;
  if (!a.cu) {
    const int per = (a.G + BM - 1) / BM, s = t / per;
    if (s >= a.S || s >= a.N) return none;
    return tile_of_rows(a, s, s, 1, first_position(a, s, 1), (t - s * per) * BM, BM);
  }
  int lo = 0, n0, n1, pos0;
  if (a.S <= 64) {                                  // a lane per sequence: everything about it in one trip to memory
    const int s = lane_id() < a.S ? lane_id() : a.S - 1;
    const int c0 = a.cu[s], c1 = a.cu[s + 1], kv = a.kv_lens[s];
    const bool past = lane_id() < a.S && (int64_t)c1 * a.G / BM + lane_id() + 1 <= t;
    lo = __popcll(__ballot(past));
    if (lo >= a.S) return none;
    n0 = __builtin_amdgcn_readlane(c0, lo);
    n1 = __builtin_amdgcn_readlane(c1, lo);
    pos0 = __builtin_amdgcn_readlane(kv, lo);
    n1 = n1 < a.N ? n1 : a.N;
    pos0 = (pos0 > 0 ? pos0 : 0) - (n1 - n0);
  } else {                                          // as find_sequence, over the tiles' starts
    int len = a.S;
    while (len > 0) {
      const int step = (len + 63) >> 6, at = (lane_id() + 1) * step;
      const bool past = at <= len && (int64_t)a.cu[lo + at] * a.G / BM + lo + at <= t;
      const int k = __popcll(__ballot(past));
      lo += k * step;
      len = step - 1 < len - k * step ? step - 1 : len - k * step;
    }
    if (lo >= a.S) return none;
    n0 = a.cu[lo];
    n1 = a.cu[lo + 1];
    n1 = n1 < a.N ? n1 : a.N;
    pos0 = first_position(a, lo, n1 - n0);
  }
  if (n0 < 0 || n1 <= n0) return none;
  const int64_t row0 = (t - ((int64_t)n0 * a.G / BM + lo)) * BM;
  if (row0 < 0 || row0 >= (int64_t)(n1 - n0) * a.G) return none;
  return tile_of_rows(a, lo, n0, n1 - n0, pos0, (int)row0, BM);
}

// Blocks of BN keys per workgroup when a tile's keys are dealt to several: the
// longest sequence of the call fills all `splits` of them, at least `least`
// blocks each, and shorter ones need fewer, so that every workgroup has about
// the same to do. The whole wave takes part.
__device__ __forceinline__ int share_blocks(const PagedArgs& a, int BM, int BN, int least) {
  if (a.splits == 1) return 0x40000000;
  int top = 0;
  for (int s = lane_id(); s < a.S; s += 64) top = top > a.kv_lens[s] ? top : a.kv_lens[s];
#pragma unroll
  for (int w = 1; w < 64; w <<= 1) { const int y = __shfl_xor(top, w); top = top > y ? top : y; }
  const int64_t cap = (int64_t)a.width << a.page_shift;
  int64_t keys = top < cap ? top : cap;
  // a window's tile starts inside a block
  if (a.window > 0 && keys > (int64_t)a.window + BM + BN) keys = (int64_t)a.window + BM + BN;
  const int64_t nb = (keys + BN - 1) / BN;
  const int per = (int)((nb + a.splits - 1) / a.splits);
  return __builtin_amdgcn_readfirstlane(per > least ? per : least);
}

// The keys [lo, hi) in blocks of BN (aligned), `per` of them to a workgroup.
struct Share { int b0, per, count; };
__device__ __forceinline__ Share share_of(int lo, int hi, int BN, int per) {
  Share x;
  x.b0 = lo / BN;
  x.per = per;
  const int nb = hi > lo ? (hi + BN - 1) / BN - x.b0 : 0;
  x.count = (nb + per - 1) / per;
  return x;
}

__device__ __forceinline__ int page_of(const PagedArgs& a, int s, int j) {   // page number or -1
  const int slot = j >> a.page_shift;
  if (j < 0 || slot >= a.width) return -1;
  const int id = a.table[s * a.table_row + slot];
  return id >= 0 && id < a.pages ? id : -1;
}

// What is noted down about an item (rows of one key/value head) whose keys several
// workgroups share: first token of the sequence, first row, rows (0: no such item),
// head, and the number of workgroups that hold parts of it. The row kernel's
// workgroups note the item that starts in their stretch and goes on behind it, the
// tile kernels' first share of every tile notes that.
constexpr int kCutInts = 8;                         // of workspace
__device__ __forceinline__ void note_cut(int* cut, const AttnTile& x, int h, int count) {
  cut[0] = x.n0; cut[1] = x.row0; cut[2] = x.rows; cut[3] = h; cut[4] = count;
}

__device__ __forceinline__ float log_sum(const PagedArgs& a, float m, float l) {
  return l == 0.f ? -__builtin_inff() : m * a.scale + fast_log2(l) * 0.6931471805599453f;
}

// First key at or behind k0 that a token at position p sees.
__device__ __forceinline__ int first_seen(const PagedArgs& a, int p, int k0) {
  const int k = a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
  return k > k0 ? k : k0;
}
// Whether it sees a key of [k0, k1), holes aside.
__device__ __forceinline__ bool sees_any(const PagedArgs& a, int p, int k0, int k1) {
  return first_seen(a, p, k0) < (p + 1 < k1 ? p + 1 : k1);
}

// Where a row's results go: the output itself when one workgroup sees all of
// the row's keys, otherwise its place among the partial results.
template <typename E, int D>
struct RowOut {
  const PagedArgs& a;
  int h;
  bool whole;
  int64_t part0, part_row;                          // partial index of row r: part0 + (part_row ? r : index(r))
  __device__ __forceinline__ int64_t index(const AttnTile& x, int r) const {     // n Hq + query head
    const int row = x.row0 + r;
    return (int64_t)(x.n0 + row / a.G) * a.Hq + h * a.G + row % a.G;
  }
  __device__ __forceinline__ int64_t slot(int64_t at, int r) const { return part0 + (part_row ? r : at); }
  __device__ __forceinline__ E* out(int64_t at) const {
    return static_cast<E*>(a.o) + at / a.Hq * a.o_row + at % a.Hq * D;
  }
  __device__ __forceinline__ float* part(int64_t at, int r) const { return a.po + slot(at, r) * D; }
  __device__ __forceinline__ void stats(int64_t at, int r, float m, float l) const {    // one lane per row
    if (whole) {
      if (a.lse) a.lse[at] = log_sum(a, m, l);
    } else {
      float* p = a.pml + slot(at, r) * 2;
      p[0] = l == 0.f ? kLeast : m;
      p[1] = l;
    }
  }
};

// One row over keys [k0, k1) by a whole wave, key by key and without products
// that other rows share: lanes score 64 keys at once, then add their values.
template <typename E, int D>
__device__ __forceinline__ void careful_row(const RowOut<E, D>& ro, const AttnTile& x, int r, int k0, int k1) {
  constexpr int V = Piece<E>::V, PER = D / 64;
  const PagedArgs& a = ro.a;
  const int h = ro.h;
  const int64_t at = ro.index(x, r);
  const int p = x.pos0 + (x.row0 + r) / a.G, lane = lane_id();
  const E* q = static_cast<const E*>(a.q) + at / a.Hq * a.q_row + at % a.Hq * D;
  const E* kc = static_cast<const E*>(a.kc) + h * a.kc_head;
  const E* vc = static_cast<const E*>(a.vc) + h * a.vc_head;
  const int first = first_seen(a, p, k0), end = p + 1 < k1 ? p + 1 : k1;
  float m = kLeast, l = 0.f, o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) o[i] = 0.f;
  for (int j0 = first; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    int id = j < end ? page_of(a, x.s, j) : -1;
    const int64_t off = j & ((1 << a.page_shift) - 1);
    float s = -__builtin_inff();
    if (id >= 0) {
      const E* k = kc + id * a.kc_page + off * a.kc_tok;
      s = 0.f;
      for (int i = 0; i < D; i += V) {
        float kx[V], qx[V];
        Piece<E>::open(*reinterpret_cast<const u32x4*>(k + i), kx);
        Piece<E>::open(*reinterpret_cast<const u32x4*>(q + i), qx);
#pragma unroll
        for (int u = 0; u < V; ++u) s += kx[u] * qx[u];
      }
    }
    if (__ballot(s != s)) {                         // a visible score is NaN: so is the row
      l = __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = l;
      break;
    }
    if (s == -__builtin_inff()) id = -1;            // not seen: its value stays out
    float top = s;
#pragma unroll
    for (int w = 1; w < 64; w <<= 1) top = fmaxf(top, __shfl_xor(top, w));
    if (top == -__builtin_inff()) continue;
    const float mn = fmaxf(m, top), al = fast_exp2((m - mn) * a.c);
    const float e = fast_exp2((s - mn) * a.c);      // +inf - +inf: NaN, as the formula has it
    m = mn;
    l = l * al + wave_sum(e);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] *= al;
    for (int u = 0; u < 64; ++u) {
      const int uid = __shfl(id, u);
      if (uid < 0) continue;
      const float w = __shfl(e, u);
      const E* v = vc + uid * a.vc_page + ((j0 + u) & ((1 << a.page_shift) - 1)) * a.vc_tok + lane * PER;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] += w * to_f32(v[i]);
    }
  }
  if (ro.whole) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < PER; ++i) ro.out(at)[lane * PER + i] = from_f32<E>(o[i] * inv);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) ro.part(at, r)[lane * PER + i] = o[i];
  }
  if (lane == 0) ro.stats(at, r, m, l);
}

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// ---------------------------------------------------------------------------
// Few rows: 16 rows at a time, four waves taking alternate blocks of 32 keys and
// joined at the end. Keys go from memory straight into operand registers (a
// 16-byte piece of a key's row is one operand), values through a wave's own LDS
// to be transposed (ds_read_b64_tr_b16 hands a lane four keys of one channel),
// so there is no barrier in the loop. Bound by reading the cache: per 32 keys of
// 256 bytes a wave spends 16 + 16 matrix instructions of 16 cycles, a tenth of
// the time its share of HBM needs to deliver them.
//
// Lengths differ, so the work is dealt evenly: the items (sequence, tile of 16
// rows, key/value head), each as many blocks of BN keys as its sequence's rows
// see (with a window, as 16 rows can see at most, from the item's own first key),
// are laid end to end, and every workgroup takes an equal stretch of blocks.
// An item that ends up in several workgroups leaves partial results: a workgroup
// has at most two, the item its stretch starts inside of and the one it ends in.
// 64 sequences of 200 to 8192 keys, 4 heads of 128 (551 MB): 110 to 113 us, 5.0 TB/s,
// the rate of a large copy; with a fixed number of shares per sequence 132 us.
template <typename E, int D>
struct RowsLayout {
  static constexpr int BM = 16, KT = 32, BN = 128;                               // BN: keys per round of four waves
  // Workgroups per CU that registers allow without spills in the loop; so many
  // are launched, one stretch of the work each.
  static constexpr int PER_CU = D == 128 ? 2 : 3;
  static constexpr int NP = D * (int)sizeof(E) / 64;                             // pieces per lane and key
  static constexpr int VLD = D * (int)sizeof(E) + (sizeof(E) == 2 ? 32 : 16);    // bytes per value row: spread banks
  static constexpr int OLD = D + 4;                                              // floats per row of a wave's result
  static constexpr int v_bytes = 4 * KT * VLD, o_bytes = 4 * BM * OLD * 4;
  static constexpr int bytes = v_bytes > o_bytes ? v_bytes : o_bytes;
};

template <typename E>
__device__ __forceinline__ f32x4 mma_piece(u32x4 k, u32x4 q, f32x4 acc) {
  if constexpr (sizeof(E) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q), acc, 0,
                                                   0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[i]), __uint_as_float(q[i]), acc, 0, 0, 0);
    return acc;
  }
}

typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
__device__ __forceinline__ s16x4 read_tr(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p));
}

// A sequence's part of the work: `items` times `nb` blocks, each item's from the
// block of its first key on.
struct RowsWork {
  int n0, cnt, pos0, items, nb;
  __device__ __forceinline__ int blocks() const { return items * nb; }
};
__device__ __forceinline__ RowsWork rows_work(const PagedArgs& a, int s, int BM, int BN) {
  RowsWork w;
  w.n0 = s; w.cnt = 1;
  if (a.cu) {
    w.n0 = a.cu[s];
    const int n1 = a.cu[s + 1];
    w.cnt = w.n0 < 0 ? 0 : (n1 < a.N ? n1 : a.N) - w.n0;
  }
  if (w.cnt <= 0) { w.pos0 = w.items = w.nb = w.cnt = 0; return w; }
  w.pos0 = first_position(a, s, w.cnt);
  const AttnTile x = tile_of_rows(a, s, w.n0, w.cnt, w.pos0, 0, 0x7fffffff);
  w.items = (w.cnt * a.G + BM - 1) / BM * a.Hk;
  w.nb = x.hi > x.lo ? (x.hi + BN - 1) / BN - x.lo / BN : 1;    // rows without keys are an item too
  if (a.window > 0) {                               // BM rows see window + BM - 1 keys at most, starting inside a block
    const int most = (int)(((unsigned)a.window + BM + BN - 3) / BN) + 1;
    w.nb = w.nb < most ? w.nb : most;
  }
  return w;
}

// Prefix sums of the sequences' blocks, a lane per run of sequences; with one
// sequence a lane, `own` keeps what the lane worked out. Counts stay below 2^31
// (checked on the host for the most keys that the table and the window let an item see).
struct RowsPlan {
  int run, before;                                  // sequences per lane, blocks before this lane's run
  RowsWork own;
  int total, shares;                                // blocks, workgroups in use
  int base, more;                                   // blocks per workgroup, one more for the first `more`
  __device__ __forceinline__ int start(int w) const { return w * base + (w < more ? w : more); }
  __device__ __forceinline__ int share(int b) const {      // the workgroup that holds block b
    const int big = more * (base + 1);
    return b < big ? b / (base + 1) : more + (b - big) / base;
  }
  __device__ __forceinline__ RowsWork work(const PagedArgs& a, int s, int BM, int BN) const {
    if (run > 1) return rows_work(a, s, BM, BN);
    auto at = [&](int v) { return __builtin_amdgcn_readlane(v, s); };
    return RowsWork{at(own.n0), at(own.cnt), at(own.pos0), at(own.items), at(own.nb)};
  }
};
__device__ __forceinline__ RowsPlan rows_plan(const PagedArgs& a, int BM, int BN) {
  RowsPlan p;
  p.run = (a.S + 63) >> 6;
  p.own = RowsWork{};
  int sum = 0;
#pragma unroll 4
  for (int i = 0; i < p.run; ++i) {
    const int s = lane_id() * p.run + i;
    const RowsWork w = rows_work(a, s < a.S ? s : a.S - 1, BM, BN);
    if (s < a.S) { p.own = w; sum += w.blocks(); }
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane_id() >= d) incl += y;
  }
  p.before = incl - sum;
  p.total = __builtin_amdgcn_readlane(incl, 63);
  p.shares = p.total < a.shares ? p.total : a.shares;
  p.base = p.total / (p.shares > 0 ? p.shares : 1);
  p.more = p.total - p.base * p.shares;
  return p;
}

template <typename E, int D>
__global__ __launch_bounds__(256, (RowsLayout<E, D>::PER_CU)) void paged_rows_kernel(PagedArgs a) {
  using LY = RowsLayout<E, D>;
  constexpr int NP = LY::NP, KT = LY::KT;
  __shared__ __align__(16) char lds[LY::bytes];
  __shared__ float ms[4][16], ls[4][16];
  __shared__ int bad[16];
  const int lane = lane_id(), wave = wave_id(), c = lane & 15, g = lane >> 4;
  const RowsPlan plan = rows_plan(a, LY::BM, LY::BN);
  int* cut = a.cuts + blockIdx.x * kCutInts;
  if (threadIdx.x == 0 && a.shares > 1) cut[2] = 0;
  if ((int)blockIdx.x >= plan.shares) return;
  int at_block = plan.start(blockIdx.x);
  const int end_block = plan.start(blockIdx.x + 1);
  // the sequence that holds at_block
  const int in = 63 - __clzll(__ballot(plan.before <= at_block));
  int s = in * plan.run;
  int seq_block = __builtin_amdgcn_readlane(plan.before, in);
  RowsWork w = plan.work(a, s, LY::BM, LY::BN);
  while (at_block < end_block) {
  while (at_block >= seq_block + w.blocks()) {
    seq_block += w.blocks();
    w = plan.work(a, ++s, LY::BM, LY::BN);
  }
  const int item = (at_block - seq_block) / w.nb, blk = at_block - seq_block - item * w.nb;
  const int take = w.nb - blk < end_block - at_block ? w.nb - blk : end_block - at_block;
  const int last_block = at_block - blk + w.nb - 1;  // of the item
  at_block += take;
  const int h = item % a.Hk;
  const AttnTile x = tile_of_rows(a, s, w.n0, w.cnt, w.pos0, item / a.Hk * LY::BM, LY::BM);
  const int64_t k0_ = (int64_t)(x.lo / LY::BN + blk) * LY::BN, k1_ = k0_ + (int64_t)take * LY::BN;
  const int k0 = k0_ > x.lo ? (int)k0_ : x.lo, k1 = k1_ < x.hi ? (int)k1_ : x.hi;
  const RowOut<E, D> ro{a, h, take == w.nb, (int64_t)(2 * blockIdx.x + (blk > 0 ? 0 : 1)) * LY::BM, 1};
  if (threadIdx.x == 0 && blk == 0 && take < w.nb) note_cut(cut, x, h, plan.share(last_block) - blockIdx.x + 1);

  // this lane's row and its queries, in the pieces the keys come in
  const int row = x.row0 + (c < x.rows ? c : x.rows - 1);
  const int p = x.pos0 + row / a.G;
  const int p_min = x.pos0 + x.row0 / a.G, p_max = x.pos0 + (x.row0 + x.rows - 1) / a.G;
  const int lo = first_seen(a, p, 0), lo_max = first_seen(a, p_max, 0);
  const E* qp = static_cast<const E*>(a.q) + (int64_t)(x.n0 + row / a.G) * a.q_row + (h * a.G + row % a.G) * D;
  u32x4 q[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) q[i] = reinterpret_cast<const u32x4*>(qp)[4 * i + g];

  const char* kb = reinterpret_cast<const char*>(static_cast<const E*>(a.kc) + h * a.kc_head) + 16 * g;
  const char* vb = reinterpret_cast<const char*>(static_cast<const E*>(a.vc) + h * a.vc_head) + 16 * g;
  const int pmask = (1 << a.page_shift) - 1;
  char* vl = lds + wave * KT * LY::VLD;

  f32x4 o[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i] = zero4();
  float m = kNoMax, l = 0.f;

  // A lane looks up the pages of its two keys (c and 16 + c of the block). The
  // entries are used a block later: loads return in order, so looking at them any
  // sooner would wait for the keys and values under way.
  const int* trow = a.table + s * a.table_row;
  auto lookup = [&](int j0, int (&id)[2]) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = j0 + 16 * b + c;
      id[b] = trow[(j < k1 ? j : k1 - 1) >> a.page_shift];
    }
  };
  u32x4 kr[2][NP], vr[2][NP];
  unsigned long long okn = 0;                       // which of the 32 keys exist (bit = key)
  auto fetch = [&](int j0, const int (&id)[2]) {
    bool ok[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j = j0 + 16 * b + c;
      ok[b] = j >= k0 && j < k1 && (unsigned)id[b] < (unsigned)a.pages;
      const int64_t pg = ok[b] ? id[b] : 0, off = j & pmask;
      const char* kp = kb + (pg * a.kc_page + off * a.kc_tok) * (int64_t)sizeof(E);
      const char* vp = vb + (pg * a.vc_page + off * a.vc_tok) * (int64_t)sizeof(E);
#pragma unroll
      for (int i = 0; i < NP; ++i) kr[b][i] = *reinterpret_cast<const u32x4*>(kp + 64 * i);
#pragma unroll
      for (int i = 0; i < NP; ++i) vr[b][i] = *reinterpret_cast<const u32x4*>(vp + 64 * i);
    }
    okn = (__ballot(ok[0]) & 0xffffu) | ((__ballot(ok[1]) & 0xffffu) << 16);
  };
  constexpr int STEP = 4 * KT;
  int j0 = (k0 / LY::BN) * LY::BN + wave * KT;
  int id[2];
  if (j0 < k1) {
    int id0[2];
    lookup(j0, id0);
    lookup(j0 + STEP, id);
    fetch(j0, id0);
  }
  for (; j0 < k1; j0 += STEP) {
    const unsigned ok = (unsigned)okn;
    f32x4 s[2] = {zero4(), zero4()};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < NP; ++i) s[b] = mma_piece<E>(kr[b][i], q[i], s[b]);
    // values to LDS; rows that do not exist as zeros
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const bool z = ok != 0xffffffffu && !((ok >> (16 * b + c)) & 1u);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (z) vr[b][i] = u32x4{0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(vl + (16 * b + c) * LY::VLD + 64 * i + 16 * g) = vr[b][i];
      }
    }
    if (j0 + STEP < k1) {
      int id2[2];
      lookup(j0 + 2 * STEP, id2);
      fetch(j0 + STEP, id);
      id[0] = id2[0]; id[1] = id2[1];
    }
    // lane: row c, keys 16 b + 4 g + i
    if (ok != 0xffffffffu || j0 + KT - 1 > p_min || j0 < lo_max) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kk = 16 * b + 4 * g + i, j = j0 + kk;
          const bool see = ((ok >> kk) & 1u) && j <= p && j >= lo;
          s[b][i] = see ? s[b][i] : -__builtin_inff();
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[b][i]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__ballot((top - m) * a.c > kSlack)) {
      const float mn = fmaxf(m, top), al = fast_exp2((m - mn) * a.c);
      m = mn;
      l *= al;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i] *= al;
    }
    const float mc = m * a.c;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[b][i] = fast_exp2(s[b][i] * a.c - mc);
        l += s[b][i];
      }
    if constexpr (sizeof(E) == 2) {
      // The weights go in as two bf16 parts, which leaves them 16 bits: the second
      // product costs nothing beside the loads, and the output's own rounding is
      // then the only one that counts.
      const bf16x8 pb = Mma<bf16>::pack(s);
      f32x4 rest[2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) rest[b][i] = s[b][i] - (float)pb[4 * b + i];
      const bf16x8 pr = Mma<bf16>::pack(rest);
      const char* src = vl + (4 * g + (lane & 15) / 4) * LY::VLD + (lane & 3) * 8;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const s16x4 v0 = read_tr(src + 32 * d), v1 = read_tr(src + 32 * d + 16 * LY::VLD);
        const bf16x4 b0 = __builtin_bit_cast(bf16x4, v0), b1 = __builtin_bit_cast(bf16x4, v1);
        const bf16x8 v = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
        o[d] = Mma<bf16>::mma(v, pr, Mma<bf16>::mma(v, pb, o[d]));
      }
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const float v = *reinterpret_cast<const float*>(vl + (16 * b + 4 * g + i) * LY::VLD + (16 * d + c) * 4);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, s[b][i], o[d], 0, 0, 0);
          }
    }
  }

  // join the four waves (the last item's readers are past the barrier that ended it)
  l = sum_groups(l);
  if (threadIdx.x < 16) bad[threadIdx.x] = 0;
  if (g == 0) { ms[wave][c] = m; ls[wave][c] = l; }
  __syncthreads();
  float* ol = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
    *reinterpret_cast<f32x4*>(ol + (wave * 16 + c) * LY::OLD + 16 * d + 4 * g) = o[d];
  __syncthreads();
  const int r = threadIdx.x >> 4, t = threadIdx.x & 15;
  if (r < x.rows) {
    float M = ms[0][r], L = 0.f, acc[D / 16];
#pragma unroll
    for (int w = 1; w < 4; ++w) M = fmaxf(M, ms[w][r]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = fast_exp2((ms[w][r] - M) * a.c);
      L += ls[w][r] * f;
#pragma unroll
      for (int i = 0; i < D / 16; i += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(ol + (w * 16 + r) * LY::OLD + t * (D / 16) + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[i + u] += v[u] * f;
      }
    }
    const int64_t at = ro.index(x, r);
    bool nf = odd_sum(L) || (L == 0.f && sees_any(a, x.pos0 + (x.row0 + r) / a.G, k0, k1));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) nf = nf || not_finite(acc[i]);
    if (nf) bad[r] = 1;
    if (ro.whole) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      E* out = ro.out(at) + t * (D / 16);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) out[i] = from_f32<E>(acc[i] * inv);
    } else {
      f32x4* out = reinterpret_cast<f32x4*>(ro.part(at, r) + t * (D / 16));
#pragma unroll
      for (int i = 0; i < D / 16; i += 4) out[i / 4] = f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
    }
    if (t == 0) ro.stats(at, r, M, L);
  }
  __syncthreads();
  for (int i = wave; i < x.rows; i += 4)
    if (bad[i]) careful_row<E, D>(ro, x, i, k0, k1);
  __syncthreads();                                  // the next item writes the same LDS
  }
}

// ---------------------------------------------------------------------------
// Many rows (bf16): 32 rows per wave, over blocks of 64 keys that the workgroup
// shares through LDS. What the two kernels for it have in common: a workgroup's
// tile and blocks, a wave's rows and queries, the way of a block from the cache to
// LDS, and the end.
template <int D, int NW_>
struct TileLayout {
  static constexpr int NW = NW_, BM = 32 * NW, BN = 64, NT = 64 * NW, LEAST = 4;
  static constexpr int KLD = 2 * D + 16, VLD = 2 * D + 32;   // bytes per row: row starts walk over the banks
  static constexpr int k_bytes = BN * KLD, v_bytes = BN * VLD, bytes = 2 * (k_bytes + v_bytes);
  static constexpr int CPR = D / 8;                          // 16-byte chunks per row
  static constexpr int ST = BN * CPR / NT;                   // chunks per thread and tensor
  static constexpr int RS = NT / CPR;                        // rows between a thread's chunks
  static constexpr int WR = 64 / CPR;                        // rows of one load of a wave
};

template <int D, int NW, bool WIDE>
struct TileWork {
  using LY = TileLayout<D, NW>;
  using E = bf16;
  static constexpr bool SPLIT = NW == 4;            // eight waves run where tiles fill the CUs: one workgroup each
  const PagedArgs& a;
  AttnTile x;
  int h, sp, first_b, T;                            // key/value head, share, first block, blocks
  bool whole;
  int lane, wave, c, hf;                            // the wave's column and half of the lane
  int p, p_min, p_max;                              // position of the lane's row, of the wave's first and last
  int lo_min, lo_max;                               // first keys that the wave's first and last rows see
  bf16x8 q[D / 16];
  const char *kb, *vb;
  const int* trow;
  int pmask, sr, sc;
  unsigned k_page, k_tok, v_page, v_tok, k_off, v_off;   // strides in bytes, below 2^32

  __device__ __forceinline__ TileWork(const PagedArgs& a_) : a(a_) {
    h = blockIdx.x % a.Hk;
    const int rest = blockIdx.x / a.Hk;
    sp = SPLIT ? rest / a.tiles : 0;
    // the last tiles of a sequence see the most keys: start with them
    x = find_tile(a, a.tiles - 1 - (SPLIT ? rest % a.tiles : rest), LY::BM);
    T = 0;
    if constexpr (SPLIT) {
      int* cut = a.splits > 1 && sp == 0 && threadIdx.x == 0 ? a.cuts + (int64_t)blockIdx.x * kCutInts : nullptr;
      if (cut) cut[2] = 0;
      if (x.rows <= 0) return;
      const Share sh = share_of(x.lo, x.hi, LY::BN, share_blocks(a, LY::BM, LY::BN, LY::LEAST));
      if (cut && sh.count > 1) note_cut(cut, x, h, sh.count);
      if (sp > 0 && sp >= sh.count) { x.rows = 0; return; }
      whole = sh.count <= 1;
      first_b = sh.b0 + sp * sh.per;
      const int all = x.hi > x.lo ? (x.hi + LY::BN - 1) / LY::BN : sh.b0;
      const int last_b = sh.per < all - first_b ? first_b + sh.per : all;
      T = last_b > first_b ? last_b - first_b : 0;
    } else {
      if (x.rows <= 0) return;
      whole = true;
      first_b = x.lo / LY::BN;
      T = x.hi > x.lo ? (x.hi + LY::BN - 1) / LY::BN - first_b : 0;
    }
    lane = lane_id(); wave = wave_id(); c = lane & 31; hf = lane >> 5;
    // rows past the tile's end repeat the last one and are not stored
    const int wr0 = wave * 32 < x.rows ? wave * 32 : x.rows - 1;
    const int wr1 = wave * 32 + 31 < x.rows ? wave * 32 + 31 : x.rows - 1;
    const int row = x.row0 + (wave * 32 + c < x.rows ? wave * 32 + c : x.rows - 1);
    p = x.pos0 + row / a.G;
    p_min = x.pos0 + (x.row0 + wr0) / a.G;
    p_max = x.pos0 + (x.row0 + wr1) / a.G;
    lo_min = first_seen(a, p_min, 0);
    lo_max = first_seen(a, p_max, 0);
    const E* qp = static_cast<const E*>(a.q) + (int64_t)(x.n0 + row / a.G) * a.q_row + (h * a.G + row % a.G) * D;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = *reinterpret_cast<const bf16x8*>(qp + 16 * i + 8 * hf);
    kb = reinterpret_cast<const char*>(static_cast<const E*>(a.kc) + h * a.kc_head);
    vb = reinterpret_cast<const char*>(static_cast<const E*>(a.vc) + h * a.vc_head);
    trow = a.table + x.s * a.table_row;
    pmask = (1 << a.page_shift) - 1;
    sr = threadIdx.x / LY::CPR;
    sc = threadIdx.x % LY::CPR;
    k_page = (unsigned)a.kc_page * 2u; k_tok = (unsigned)a.kc_tok * 2u;
    v_page = (unsigned)a.vc_page * 2u; v_tok = (unsigned)a.vc_tok * 2u;
    k_off = (lane / LY::CPR) * k_tok + sc * 16;
    v_off = (lane / LY::CPR) * v_tok + sc * 16;
  }
  // The queries are here before the loop: without this the waits for them stand in it.
  __device__ __forceinline__ void have_queries() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(q[i]));
  }
  // Lane l of every wave looks up key l of block first_b + t (a block past the end
  // falls on the last key's page). The entry is not looked at before the next
  // block's turn: loads return in order, so that would wait for the keys and values
  // under way.
  __device__ __forceinline__ int lookup(int t) const {
    const int j = (first_b + t) * LY::BN + lane;
    return trow[(j < x.hi ? j : x.hi - 1) >> a.page_shift];
  }
  __device__ __forceinline__ unsigned long long valid(int t, int id) const {   // the block's keys that exist, a bit each
    const int j = (first_b + t) * LY::BN + lane;
    return __ballot((j >= x.lo) & (j < x.hi) & ((unsigned)id < (unsigned)a.pages));
  }
  // Byte offset of the lane's key of block t, on page `id` (page 0 where there is none).
  __device__ __forceinline__ uint64_t place(int t, int id, unsigned page_bytes, unsigned tok_bytes) const {
    const unsigned pg = (unsigned)id < (unsigned)a.pages ? id : 0;
    const unsigned off = ((first_b + t) * LY::BN + lane) & pmask;
    return (uint64_t)pg * page_bytes + (uint64_t)off * tok_bytes;
  }
  // The thread's chunk i of a block. The rows that one load of a wave covers (4, or
  // 8 at d = 64) lie in one page of at least 8 tokens (WIDE): their first row's
  // address is a scalar then, and a lane adds a constant of 32 bits. Token strides
  // that would pass those take the other form.
  __device__ __forceinline__ u32x4 load(const char* base, uint64_t at, unsigned lane_off, int i) const {
    if constexpr (WIDE) {
      const int r0 = wave * LY::WR + LY::RS * i;
      const unsigned lo = __builtin_amdgcn_readlane((int)at, r0), hi = __builtin_amdgcn_readlane((int)(at >> 32), r0);
      return *reinterpret_cast<const u32x4*>(base + ((uint64_t)hi << 32 | lo) + lane_off);
    } else {
      const int rr = sr + LY::RS * i;
      const unsigned lo = __shfl((int)at, rr), hi = __shfl((int)(at >> 32), rr);
      return *reinterpret_cast<const u32x4*>(base + ((uint64_t)hi << 32 | lo) + sc * 16);
    }
  }
  __device__ __forceinline__ u32x4 load_k(uint64_t at, int i) const { return load(kb, at, k_off, i); }
  __device__ __forceinline__ u32x4 load_v(uint64_t at, int i) const { return load(vb, at, v_off, i); }
  // Zeros in the place of values whose key does not exist: a weight of 0 would not
  // drop what an unused cache entry holds if that is not finite.
  __device__ __forceinline__ void clear(unsigned long long ok, u32x4 (&vr)[LY::ST]) const {
    if (ok != ~0ull) {
#pragma unroll
      for (int i = 0; i < LY::ST; ++i) {
        const unsigned keep = (ok >> (sr + LY::RS * i)) & 1ull ? ~0u : 0u;
        vr[i] &= u32x4{keep, keep, keep, keep};
      }
    }
  }
  // Scores of block t that a row does not see. Lane: row c, keys 32 kb2 + 8 (u / 4) + 4 hf + u % 4.
  __device__ __forceinline__ void mask(int t, unsigned long long ok, f32x16 (&s)[2]) const {
    const int j0 = (first_b + t) * LY::BN;
    if (ok != ~0ull) {                              // keys that do not exist
      const unsigned long long mine = ok >> (4 * hf);
#pragma unroll
      for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
        for (int u = 0; u < 16; ++u)
          s[kb2][u] = (mine >> (32 * kb2 + 8 * (u / 4) + u % 4)) & 1ull ? s[kb2][u] : -__builtin_inff();
    }
    if (j0 + LY::BN - 1 > p_min || j0 < lo_max) {
      const int far = p - j0 - 4 * hf;              // visible: far - window < key <= far
      const unsigned wide = a.window > 0 ? a.window : 0x7fffffff;
#pragma unroll
      for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
        for (int u = 0; u < 16; ++u)
          s[kb2][u] = (unsigned)(far - (32 * kb2 + 8 * (u / 4) + u % 4)) < wide ? s[kb2][u] : -__builtin_inff();
    }
  }
  // Moves the row's reference up to `top` where that has grown far enough.
  __device__ __forceinline__ void rescale(float top, float& m, float& l, f32x16 (&o)[D / 32]) const {
    if (__ballot((top - m) * a.c > kSlack)) {
      const float mn = fmaxf(m, top), al = fast_exp2((m - mn) * a.c);
      m = mn;
      l *= al;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int u = 0; u < 16; ++u) o[i][u] *= al;
    }
  }
  __device__ __forceinline__ void finish(const f32x16 (&o)[D / 32], float m, float l) const {
    l += __shfl_xor(l, 32);
    const RowOut<E, D> ro{a, h, !SPLIT || whole, (int64_t)sp * a.N * a.Hq, 0};
    const int r = wave * 32 + c;
    bool nf = false, none = false;
    if (r < x.rows) {
      const int64_t at = ro.index(x, r);
      nf = odd_sum(l);
      none = l == 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int u = 0; u < 16; ++u) nf = nf || not_finite(o[i][u]);
      if (!SPLIT || whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        E* out = ro.out(at) + 4 * hf;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            *reinterpret_cast<bf16x4*>(out + 32 * i + 2 * u) =
                bf16x4{(bf16)(o[i][u] * inv), (bf16)(o[i][u + 1] * inv), (bf16)(o[i][u + 2] * inv),
                       (bf16)(o[i][u + 3] * inv)};
      } else {
        float* out = ro.part(at, r) + 4 * hf;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int u = 0; u < 16; u += 4)
            *reinterpret_cast<f32x4*>(out + 32 * i + 2 * u) = f32x4{o[i][u], o[i][u + 1], o[i][u + 2], o[i][u + 3]};
      }
      if (hf == 0) ro.stats(at, r, m, l);
    }
    const int k0 = first_b * LY::BN > x.lo ? first_b * LY::BN : x.lo;
    const int64_t k1_ = (int64_t)(first_b + T) * LY::BN;
    const int k1 = k1_ < x.hi ? (int)k1_ : x.hi;
    unsigned long long again = __ballot(nf);
    if (__ballot(none)) again |= __ballot(none && sees_any(a, x.pos0 + (x.row0 + r) / a.G, k0, k1));
    again = (again | again >> 32) & 0xffffffffull;
    while (again) {
      const int i = __ffsll((unsigned long long)again) - 1;
      again &= again - 1;
      careful_row<E, D>(ro, x, wave * 32 + i, k0, k1);
    }
  }
};

// d = 64: four waves, each block in turn (products, softmax, products), four
// workgroups per CU that fill each other's waits. Vector work outweighs the
// products here (130 vector instructions of a softmax block against 16 products),
// and four waves per SIMD issue it faster than two that interleave: on ragged
// windowed prompts (51 GFLOP) the kernel below took 133 us when this one, then
// with three workgroups per CU, took 107 us; with four a call takes 90 to 92 us (560
// TFLOP/s). In the loop the matrix units are busy 57% of the time; a workgroup of 18
// blocks spends an eighth of its time on finding its tile and its first loads.
// d = 128: two workgroups per CU, for calls of few tiles.
template <int D, bool WIDE>
__global__ __launch_bounds__(256, D == 64 ? 4 : 2) void paged_tile_kernel(PagedArgs a) {
  using W = TileWork<D, 4, WIDE>;
  using LY = typename W::LY;
  extern __shared__ __align__(16) char lds[];
  W w(a);
  if (w.x.rows <= 0) return;
  const int T = w.T;
  f32x16 o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int u = 0; u < 16; ++u) o[i][u] = 0.f;
  float m = kNoMax, l = 0.f;
  constexpr int buf_bytes = LY::k_bytes + LY::v_bytes;
  u32x4 kr[LY::ST], vr[LY::ST];
  auto fetch = [&](int t, int id) {
    const uint64_t k_at = w.place(t, id, w.k_page, w.k_tok), v_at = w.place(t, id, w.v_page, w.v_tok);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) {
      kr[i] = w.load_k(k_at, i);
      vr[i] = w.load_v(v_at, i);
    }
  };
  auto store = [&](int buf, unsigned long long ok) {
    char* kl = lds + buf * buf_bytes + w.sr * LY::KLD + w.sc * 16;
    char* vl = lds + buf * buf_bytes + LY::k_bytes + w.sr * LY::VLD + w.sc * 16;
    w.clear(ok, vr);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) {
      *reinterpret_cast<u32x4*>(kl + LY::RS * i * LY::KLD) = kr[i];
      *reinterpret_cast<u32x4*>(vl + LY::RS * i * LY::VLD) = vr[i];
    }
  };
  unsigned long long ok = 0;
  int idn = 0;                                      // table entry of the block after the one in registers
  if (T > 0) {
    const int id0 = w.lookup(0);
    idn = w.lookup(1);
    ok = w.valid(0, id0);
    fetch(0, id0);
    store(0, ok);
  }
  w.have_queries();
  for (int t = 0; t < T; ++t) {
    const int buf = t & 1;
    __syncthreads();                                // block t is in LDS; nobody reads the other buffer any more
    const unsigned long long okn = w.valid(t + 1, idn);
    const int id2 = w.lookup(t + 2);
    fetch(t + 1, idn);
    idn = id2;
    const int j0 = (w.first_b + t) * LY::BN;
    if (j0 <= w.p_max && j0 + LY::BN > w.lo_min) {
      const char* kl = lds + buf * buf_bytes;
      const char* vl = kl + LY::k_bytes;
      f32x16 s[2];
#pragma unroll
      for (int kb2 = 0; kb2 < 2; ++kb2) {
#pragma unroll
        for (int u = 0; u < 16; ++u) s[kb2][u] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const bf16x8 k = *reinterpret_cast<const bf16x8*>(kl + (32 * kb2 + w.c) * LY::KLD + 32 * i + 16 * w.hf);
          s[kb2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, w.q[i], s[kb2], 0, 0, 0);
        }
      }
      w.mask(t, ok, s);
      float top = s[0][0];
#pragma unroll
      for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
        for (int u = 0; u < 16; ++u) top = fmaxf(top, s[kb2][u]);
      top = fmaxf(top, __shfl_xor(top, 32));
      w.rescale(top, m, l, o);
      const float mc = m * a.c;
      bf16x8 pb[4];
#pragma unroll
      for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const float e = fast_exp2(s[kb2][u] * a.c - mc);
          l += e;
          pb[2 * kb2 + u / 8][u % 8] = (bf16)e;
        }
      const char* src = vl + (4 * w.hf + (w.lane & 15) / 4) * LY::VLD + ((w.lane >> 4) & 1) * 32 + (w.lane & 3) * 8;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          const s16x4 v0 = read_tr(src + 16 * ks * LY::VLD + 64 * d);
          const s16x4 v1 = read_tr(src + (16 * ks + 8) * LY::VLD + 64 * d);
          const bf16x4 b0 = __builtin_bit_cast(bf16x4, v0), b1 = __builtin_bit_cast(bf16x4, v1);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              bf16x8{b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]}, pb[ks], o[d], 0, 0, 0);
        }
    }
    store(buf ^ 1, okn);
    ok = okn;
  }
  w.finish(o, m, l);
}

// d = 128, many tiles: eight waves, two blocks under way in each. A wave issues an
// instruction every five cycles or so and a 32x32x16 product occupies the matrix
// unit for 32, so the vector work has to stand between the products of the same
// wave: in step t the products X(t+1) are dealt among the exponentials of block t,
// then the products O += P(t) V(t) among the maxima of X(t+1), and the operands
// come from LDS a few products ahead. Measured per step of 8 waves: 2200 cycles
// for the products (2048 without any gap), 1000 for the pair (below) and 900 of
// wait for the slower half of the waves.
//
// Blocks are loaded into registers two steps ahead and written to LDS one ahead:
// "pair p" is keys p + 1 and values p. Step t, between two barriers, writes pair
// t + 1 (keys t + 2 over keys t, read in step t - 1; values t + 1 over values
// t - 1, likewise) while it reads keys t + 1 and values t.
// 4096 tokens of 16 heads over 16384 keys (481 GFLOP): 495 to 527 us a call by card,
// 913 to 970 TFLOP/s, where the kernel above takes 600 us. Those are 256 workgroups of
// 192 to 256 blocks on 256 CUs: the longest decides, an eighth above the mean.
template <int D, bool WIDE>
__global__ __launch_bounds__(512, 2) void paged_step_kernel(PagedArgs a) {
  using W = TileWork<D, 8, WIDE>;
  using LY = typename W::LY;
  extern __shared__ __align__(16) char lds[];
  W w(a);
  if (w.x.rows <= 0) return;
  const int T = w.T;
  f32x16 o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int u = 0; u < 16; ++u) o[i][u] = 0.f;
  float m = kNoMax, l = 0.f, top = 0.f;             // top: the row's maximum in the next block

  u32x4 kr[LY::ST], vr[LY::ST];
  int pair = 0;                                     // the pair in registers: keys pair + 1, values pair
  int id1 = 0, id2 = 0;                             // table entries of blocks pair + 1 and pair + 2
  unsigned long long ok_now = 0, ok_last = 0;       // keys of blocks pair and pair - 1
  char* vlds = lds + 2 * LY::k_bytes;
  char* k_dst = lds + w.sr * LY::KLD + w.sc * 16;
  char* v_dst = vlds + w.sr * LY::VLD + w.sc * 16;
  // Pair to LDS, the one after it under way. Nothing here depends on how many
  // blocks are left (blocks past the end are not used), so the counts of loads in
  // flight are known and each wait is for its own.
  auto next_pair = [&]() {
    w.clear(ok_now, vr);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i)
      *reinterpret_cast<u32x4*>(k_dst + ((pair + 1) & 1) * LY::k_bytes + LY::RS * i * LY::KLD) = kr[i];
#pragma unroll
    for (int i = 0; i < LY::ST; ++i)
      *reinterpret_cast<u32x4*>(v_dst + (pair & 1) * LY::v_bytes + LY::RS * i * LY::VLD) = vr[i];
    ok_last = ok_now;
    ok_now = w.valid(pair + 1, id1);
    ++pair;
    const uint64_t k_at = w.place(pair + 1, id2, w.k_page, w.k_tok), v_at = w.place(pair, id1, w.v_page, w.v_tok);
    id1 = id2;
    id2 = w.lookup(pair + 2);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) kr[i] = w.load_k(k_at, i);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) vr[i] = w.load_v(v_at, i);
  };
  if (T > 0) {
    const int id0 = w.lookup(0);
    id1 = w.lookup(1);
    id2 = w.lookup(2);
    ok_now = w.valid(0, id0);
    uint64_t k_at = w.place(0, id0, w.k_page, w.k_tok);
    const uint64_t v_at = w.place(0, id0, w.v_page, w.v_tok);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) kr[i] = w.load_k(k_at, i);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) *reinterpret_cast<u32x4*>(k_dst + LY::RS * i * LY::KLD) = kr[i];
    k_at = w.place(1, id1, w.k_page, w.k_tok);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) kr[i] = w.load_k(k_at, i);
#pragma unroll
    for (int i = 0; i < LY::ST; ++i) vr[i] = w.load_v(v_at, i);
  }
  w.have_queries();

  // the blocks [w0, w1) of the workgroup's that some row of the wave sees
  int w0, w1 = w.p_max < 0 ? 0 : (w.p_max >> 6) + 1 - w.first_b;
  w1 = w1 < T ? w1 : T;
  w0 = (w.lo_min >> 6) - w.first_b;
  w0 = w0 > 0 ? w0 : 0;
  if (w0 >= w1) w0 = w1 = T + 2;

  // X^T of block t: product i is channels 16 (i / 2) .. of the half i % 2 of its keys
  constexpr int NK = D / 8, RK = 8, EP = 32 / NK;
  const char* k_src = lds + w.c * LY::KLD + 16 * w.hf;
  auto read_k = [&](const char* kl, int i) {
    return *reinterpret_cast<const bf16x8*>(kl + 32 * (i & 1) * LY::KLD + 32 * (i >> 1));
  };
  // O^T: product i is keys 16 (i / ND) .. of the block, channels 32 (i % ND) ..
  constexpr int ND = D / 32, NV = 4 * ND, RV = 6;
  const char* v_src = vlds + (4 * w.hf + (w.lane & 15) / 4) * LY::VLD + ((w.lane >> 4) & 1) * 32 + (w.lane & 3) * 8;
  auto read_v = [&](const char* vl, int i, s16x4 (&v)[2]) {
    const char* at = vl + 16 * (i / ND) * LY::VLD + 64 * (i % ND);
    v[0] = read_tr(at);
    v[1] = read_tr(at + 8 * LY::VLD);
  };

  // step t: cur holds X(t), nxt takes X(t + 1)
  auto step = [&](int t, f32x16 (&cur)[2], f32x16 (&nxt)[2]) {
    __syncthreads();
    const char* kl = k_src + ((t + 1) & 1) * LY::k_bytes;
    const char* vl = v_src + (t & 1) * LY::v_bytes;
    bf16x8 kf[RK];
    const bool on = t >= w0 && t < w1;
    if (on || t + 1 == w0) {
#pragma unroll
      for (int i = 0; i < RK; ++i) kf[i] = read_k(kl, i);
    }
    next_pair();
    if (on) {
      w.rescale(top, m, l, o);
      const float mc = m * a.c;
      float sum[2] = {0.f, 0.f};
      bf16x8 pb[4];
      s16x4 vf[RV][2];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < 16; ++u) nxt[0][u] = nxt[1][u] = 0.f;
#pragma unroll
      for (int i = 0; i < NK + 2; ++i) {
        if (i < NK) {
          nxt[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i % RK], w.q[i >> 1], nxt[i & 1], 0, 0, 0);
          if (i + RK < NK) kf[i % RK] = read_k(kl, i + RK);
        }
        if (i >= NK - RV && i < NK) read_v(vl, i - (NK - RV), vf[i - (NK - RV)]);
        // element e of cur in three turns: argument, power, sum and rounding
#pragma unroll
        for (int u = 0; u < EP; ++u) {
          if (i < NK) {
            const int e = EP * i + u;
            cur[e >> 4][e & 15] = cur[e >> 4][e & 15] * a.c - mc;
          }
          if (i >= 1 && i <= NK) {
            const int e = EP * (i - 1) + u;
            cur[e >> 4][e & 15] = fast_exp2(cur[e >> 4][e & 15]);
          }
          if (i >= 2) {
            const int e = EP * (i - 2) + u;
            sum[u & 1] += cur[e >> 4][e & 15];
            pb[e >> 3][e & 7] = (bf16)cur[e >> 4][e & 15];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      l += sum[0] + sum[1];
      w.mask(t + 1, ok_last, nxt);
      float top2 = nxt[0][0];
      top = nxt[1][0];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bf16x4 b0 = __builtin_bit_cast(bf16x4, vf[i % RV][0]), b1 = __builtin_bit_cast(bf16x4, vf[i % RV][1]);
        o[i % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            bf16x8{b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]}, pb[i / ND], o[i % ND], 0, 0, 0);
        if (i + RV < NV) read_v(vl, i + RV, vf[i % RV]);
        // from product 2 on, the maxima: X(t + 1) has left the matrix unit by then
        constexpr int MP = (16 + NV - 3) / (NV - 2);
#pragma unroll
        for (int u = 0; u < MP; ++u) {
          const int e = MP * (i - 2) + u;
          if (i >= 2 && e < 16) {
            top2 = fmaxf(top2, nxt[0][e]);
            top = fmaxf(top, nxt[1][e]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      top = fmaxf(top, top2);
      top = fmaxf(top, __shfl_xor(top, 32));
    } else if (t + 1 == w0) {                       // the wave's first block
#pragma unroll
      for (int u = 0; u < 16; ++u) nxt[0][u] = nxt[1][u] = 0.f;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        nxt[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i % RK], w.q[i >> 1], nxt[i & 1], 0, 0, 0);
        if (i + RK < NK) kf[i % RK] = read_k(kl, i + RK);
      }
      w.mask(t + 1, ok_last, nxt);
      top = nxt[0][0];
#pragma unroll
      for (int kb2 = 0; kb2 < 2; ++kb2)
#pragma unroll
        for (int u = 0; u < 16; ++u) top = fmaxf(top, nxt[kb2][u]);
      top = fmaxf(top, __shfl_xor(top, 32));
    }
  };
  f32x16 s0[2], s1[2];
  if (T > 0)
    for (int t = -1; t < T; t += 2) {
      step(t, s0, s1);
      if (t + 1 < T) step(t + 1, s1, s0);
    }
  w.finish(o, m, l);
}

// ---------------------------------------------------------------------------
// Joins the partial results of one (token, query head). Each of WAVES waves takes a
// run of the shares, 64 at a time: a lane per share for the statistics, then the
// shares' outputs weighted by them, 32 loads in flight. The runs' sums meet in LDS;
// the sizes and lengths alone decide the order. Partial index of share i: first for
// i = 0, next + (i - 1) stride from there on.
template <typename E, int D, int WAVES>
__device__ __forceinline__ void join_shares(const PagedArgs& a, int64_t at, int64_t first, int64_t next,
                                            int64_t stride, int count) {
  constexpr int PER = D / 64, U = 8, GROUPS = 4;
  using V = __attribute__((ext_vector_type(PER))) float;
  const int lane = lane_id(), wave = WAVES > 1 ? wave_id() : 0;
  auto slot = [&](int i) { return i == 0 ? first : next + (i - 1) * stride; };
  float M = kLeast, L = 0.f;
  V o = 0.f;
  const int run = (count + WAVES - 1) / WAVES, end = run * (wave + 1) < count ? run * (wave + 1) : count;
  for (int c0 = run * wave; c0 < end; c0 += 64) {
    const int left = end - c0 < 64 ? end - c0 : 64;
    const int64_t own = slot(c0 + (lane < left ? lane : 0));
    const float m = a.pml[own * 2], l = a.pml[own * 2 + 1];
    V v[GROUPS * U];
    auto load = [&](int i0) {
#pragma unroll
      for (int q = 0; q < GROUPS; ++q)
        if (q == 0 || i0 + q * U < left)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = i0 + q * U + u;
            v[q * U + u] = *reinterpret_cast<const V*>(a.po + slot(c0 + (i < left ? i : left - 1)) * D + lane * PER);
          }
    };
    load(0);
    float M1 = m;
#pragma unroll
    for (int w = 1; w < 64; w <<= 1) M1 = fmaxf(M1, __shfl_xor(M1, w));
    M1 = fmaxf(M1, M);
    const float f = fast_exp2((M - M1) * a.c), e = lane < left ? fast_exp2((m - M1) * a.c) : 0.f;
    L = L * f + wave_sum(l * e);
    M = M1;
    o *= f;
    for (int i0 = 0; i0 < left; i0 += GROUPS * U) {
      if (i0) load(i0);
#pragma unroll
      for (int q = 0; q < GROUPS; ++q)
        if (q == 0 || i0 + q * U < left)
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (i0 + q * U + u < left)
              o += v[q * U + u] * __int_as_float(__builtin_amdgcn_readlane(__float_as_int(e), i0 + q * U + u));
    }
  }
  if constexpr (WAVES > 1) {
    __shared__ float ml[WAVES][2];
    __shared__ V part[WAVES][64];
    if (lane == 0) { ml[wave][0] = M; ml[wave][1] = L; }
    part[wave][lane] = o;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) M = fmaxf(M, ml[w][0]);
    L = 0.f;
    o = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float f = fast_exp2((ml[w][0] - M) * a.c);
      L += ml[w][1] * f;
      o += part[w][lane] * f;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  E* out = static_cast<E*>(a.o) + at / a.Hq * a.o_row + at % a.Hq * D + lane * PER;
#pragma unroll
  for (int k = 0; k < PER; ++k) out[k] = from_f32<E>(o[k] * inv);
  if (lane == 0 && a.lse)
    a.lse[at] = log_sum(a, M, L);
}

// The rows of a tile whose keys were shared, as its first share noted it down: one
// to a wave, or, where there are many rows and at most kFewShares shares, eight, four
// at a time with a lane per row and share for the statistics. 4000 tokens over
// themselves, 12 heads of 64 in two shares: 9.6 us, a row to a wave 30; 256 tokens of
// 16 heads of 128 in 16 shares 16 and 9.
constexpr int kFewShares = 16;
template <int D, int ROWS>
__global__ __launch_bounds__(256) void paged_tile_combine_kernel(PagedArgs a) {
  const int* cut = a.cuts + (int64_t)blockIdx.x * kCutInts;
  const int n0 = cut[0], row0 = cut[1], rows = cut[2], h = cut[3], count = cut[4];
  const int64_t stride = (int64_t)a.N * a.Hq;
  auto index = [&](int r) {
    const int row = row0 + r;
    return (int64_t)(n0 + row / a.G) * a.Hq + h * a.G + row % a.G;
  };
  const int first = (blockIdx.y * 4 + wave_id()) * ROWS;
  if (first >= rows) return;
  if constexpr (ROWS == 1) {
    const int64_t at = index(first);
    join_shares<bf16, D, 1>(a, at, at, at + stride, stride, count);
  } else {
    constexpr int PER = D / 64, R = 4, U = 4;       // rows and shares of a round of loads
    using V = __attribute__((ext_vector_type(PER))) float;
    const int lane = lane_id(), own = lane & (kFewShares - 1);
    for (int r0 = first; r0 < first + ROWS && r0 < rows; r0 += R) {
      int64_t at[R];
#pragma unroll
      for (int r = 0; r < R; ++r) at[r] = index(r0 + r < rows ? r0 + r : rows - 1);
      const int mine = r0 + lane / kFewShares;
      const int64_t my = index(mine < rows ? mine : rows - 1);
      const int64_t p = my + (own < count ? own : 0) * stride;
      const float m = a.pml[p * 2], l = a.pml[p * 2 + 1];
      V o[R] = {};
      float M = m;
#pragma unroll
      for (int w = 1; w < kFewShares; w <<= 1) M = fmaxf(M, __shfl_xor(M, w));
      float f = own < count ? fast_exp2((m - M) * a.c) : 0.f, L = l * f;
#pragma unroll
      for (int w = 1; w < kFewShares; w <<= 1) L += __shfl_xor(L, w);
      f *= L == 0.f ? 0.f : 1.f / L;
      for (int i0 = 0; i0 < count; i0 += U) {
        V v[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < R; ++r)
            v[u][r] = *reinterpret_cast<const V*>(
                a.po + (at[r] + (i0 + u < count ? i0 + u : count - 1) * stride) * D + lane * PER);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + u < count)
#pragma unroll
            for (int r = 0; r < R; ++r)
              o[r] += v[u][r] * __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), r * kFewShares + i0 + u));
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r0 + r < rows) {
          bf16* out = static_cast<bf16*>(a.o) + at[r] / a.Hq * a.o_row + at[r] % a.Hq * D + lane * PER;
#pragma unroll
          for (int k = 0; k < PER; ++k) out[k] = (bf16)o[r][k];
        }
      if (a.lse && own == 0 && mine < rows)
        a.lse[my] = log_sum(a, M, L);
    }
  }
}

// The rows of the item, if any, that starts in workgroup blockIdx.x's stretch of the
// row kernel and goes on behind it: what that workgroup noted down. A wave per row
// (d = 64, fp32, 768 workgroups: 5.2 us, 9.5 with WAVES = 4), or a workgroup per row
// where few items leave many shares to each (d = 128, 128 shares: 6.1 us, 12 in a
// wave).
template <typename E, int D, int WAVES>
__global__ __launch_bounds__(256) void paged_rows_combine_kernel(PagedArgs a) {
  using LY = RowsLayout<E, D>;
  const int64_t w = blockIdx.x;
  const int* cut = a.cuts + w * kCutInts;
  const int r = WAVES > 1 ? blockIdx.y : blockIdx.y * 4 + wave_id();
  if (r >= cut[2]) return;
  const int row = cut[1] + r;
  const int64_t at = (int64_t)(cut[0] + row / a.G) * a.Hq + cut[3] * a.G + row % a.G;
  join_shares<E, D, WAVES>(a, at, (2 * w + 1) * LY::BM + r, 2 * (w + 1) * LY::BM + r, 2 * LY::BM, cut[4]);
}

}  // namespace carve
