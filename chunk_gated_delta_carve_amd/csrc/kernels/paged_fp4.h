// Attention of new tokens over a paged cache in 4 bits: what paged_attn.h does, over
// the values that the codes stand for.
#pragma once
#include "fp4.h"
#include "paged_attn.h"

namespace carve {

struct Fp4Args : PagedArgs {           // kc, vc: codes, strides in bytes
  const uint8_t *ks, *vs;
  Fp4Strides k, v;                     // of the scales
};

// A key/value head of such a cache, an entry at a time.
template <typename E, int D>
struct Fp4Entries {
  static constexpr int PER = D / 64;
  const Fp4Args& a;
  const uint8_t *kc, *vc, *ks, *vs;
  __device__ __forceinline__ Fp4Entries(const Fp4Args& a_, int h)
      : a(a_), kc(static_cast<const uint8_t*>(a_.kc) + h * a_.kc_head),
        vc(static_cast<const uint8_t*>(a_.vc) + h * a_.vc_head), ks(a_.ks + h * a_.k.head), vs(a_.vs + h * a_.v.head) {}
  __device__ __forceinline__ float score(int id, int64_t off, const E* q) const {
    const unsigned* c = reinterpret_cast<const unsigned*>(kc + id * a.kc_page + off * a.kc_tok);
    const uint8_t* e = ks + id * a.k.page + off * a.k.tok;
    float s = 0.f;
    for (int i = 0; i < D / 8; ++i) {
      float kx[8], qx[8];
      fp4_open8(c[i], fp4_factor(e[i / 4]), kx);
      if constexpr (sizeof(E) == 2) {
        Piece<E>::open(reinterpret_cast<const u32x4*>(q)[i], qx);
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) qx[u] = q[8 * i + u];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) s += kx[u] * qx[u];
    }
    return s;
  }
  __device__ __forceinline__ void add(int id, int64_t off, float w, float (&o)[PER]) const {
    // lane l has the channels from l PER on: half a byte at d = 64
    const int at = lane_id() * PER;
    const unsigned c = vc[id * a.vc_page + off * a.vc_tok + at / 2];
    const float s = fp4_factor(vs[id * a.v.page + off * a.v.tok + at / kFp4Block]);
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    if constexpr (PER == 2) {
      o[0] += w * v[0];
      o[1] += w * v[1];
    } else {
      o[0] += w * (at & 1 ? v[1] : v[0]);
    }
  }
};

// Few rows, as paged_rows_kernel deals them: 16 rows at a time, four waves taking
// alternate blocks of 32 keys. A lane has key c's channels [g D/4, (g + 1) D/4), one load
// of 16 bytes (8 at d = 64) and one scale, opened to bf16 in registers: the keys as
// operands, the values on their way through the wave's LDS. fp32 queries and weights
// enter the products as three bf16 parts, which hold their 24 bits; the codes are exact.
// (The products that take 4-bit operands as they are drop what lies 2^13 below the largest
// of eight terms, so a sum would not hold 32 bits.)
//
// Bound by memory where there is much (64 sequences of 200 to 8192 keys, 4 heads of 128,
// 147 MB: 33 us, 4.4 TB/s), by an item's chain of trips otherwise: lengths, page, entries,
// some 5 us (4 sequences of 50k to 65k keys of 2 heads, 64 MB: 18 us where the copy's rate
// would give 13). Loading two blocks ahead costs d = 64 its fourth workgroup of a CU (256
// sequences of 1000 keys, 12 heads, 54 us became 59) and gains d = 128 nothing.
template <typename E, int D>
struct RowsFp4 {
  static constexpr int BM = 16, KT = 32, BN = 4 * KT;                            // as RowsLayout
  // workgroups of a CU; one fewer in fp32 would spare a register of d = 128, and took 92 us for
  // 77 (50 sequences of 38 to 75 tokens over 385 to 770 keys, 16 heads on 4 of 128), at d = 64 48 for 41
  static constexpr int PER_CU = D == 128 ? 3 : 4;
  static constexpr int NI = D / 32;                                              // products per block of 16 keys
  static constexpr int NQ = sizeof(E) == 2 ? 1 : 3, NP = sizeof(E) == 2 ? 2 : 3; // parts of q and of the weights
  static constexpr int VLD = 2 * D + 32, OLD = D + 4;
  static constexpr int v_bytes = 4 * KT * VLD, o_bytes = 4 * BM * OLD * 4;
  static constexpr int bytes = v_bytes > o_bytes ? v_bytes : o_bytes;
};

// Three parts of 8 bits, cut off one after the other: their sum is x.
__device__ __forceinline__ void cut_parts(const float (&x)[8], u32x4 (&part)[3]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned a = __float_as_uint(r[2 * i]) & 0xffff0000u, b = __float_as_uint(r[2 * i + 1]) & 0xffff0000u;
      part[p][i] = a >> 16 | b;
      r[2 * i] -= __uint_as_float(a);
      r[2 * i + 1] -= __uint_as_float(b);
    }
}

__device__ __forceinline__ f32x4 mma_bits(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// An item costs a workgroup about as much before and after its blocks as three of them
// (finding it, three dependent loads, joining the waves), so that much is added to its
// blocks where the work is dealt out: short sequences, several to a workgroup, would
// otherwise make the slowest ones. 64 sequences of 200 to 8192 keys, 4 heads of 128: 33.3
// us, without 36.5; 12 heads of 64: 56 and 66.
constexpr int kStart = 3;

// WIDE: pages of 16 tokens and more, so that 16 aligned keys lie in one. A lane looks
// up the page of one of the wave's next 64 runs of 16 keys, and a run's address is a
// scalar to which a lane adds a constant. Otherwise every lane looks up its own keys'.
template <typename E, int D, bool WIDE>
__global__ __launch_bounds__(256, (RowsFp4<E, D>::PER_CU)) void paged_rows_fp4_kernel(Fp4Args a) {
  using LY = RowsFp4<E, D>;
  constexpr int NI = LY::NI, KT = LY::KT, NQ = LY::NQ;
  using Codes = __attribute__((ext_vector_type(NI))) unsigned;
  __shared__ __align__(16) char lds[LY::bytes];
  __shared__ float ms[4][16], ls[4][16];
  __shared__ int bad[16];
  const int lane = lane_id(), wave = wave_id(), c = lane & 15, g = lane >> 4;
  const RowsPlan plan = rows_plan<kStart>(a, LY::BM, LY::BN);
  if (threadIdx.x == 0 && a.po) a.cuts[blockIdx.x] = 0;
  if ((int)blockIdx.x >= plan.shares) return;
  int at_block = plan.start(blockIdx.x);            // in blocks of the plan, kStart more per item than it has
  const int end_block = plan.start(blockIdx.x + 1);
  const int in = 63 - __clzll(__ballot(plan.before <= at_block));
  int s = in * plan.run;
  int seq_block = __builtin_amdgcn_readlane(plan.before, in);
  RowsWork w = plan.work<kStart>(a, s, LY::BM, LY::BN);
  // Strides as registers of their own: the compiler keeps kernel arguments in the groups it
  // loads them in, and parks whole groups in vector registers for want of scalar ones.
  unsigned kpage = a.kc_page, ktok = a.kc_tok, vpage = a.vc_page, vtok = a.vc_tok;
  unsigned kspage = a.k.page, kstok = a.k.tok, vspage = a.v.page, vstok = a.v.tok, pages = a.pages, shift = a.page_shift;
  asm volatile("" : "+s"(kpage), "+s"(ktok), "+s"(vpage), "+s"(vtok), "+s"(kspage), "+s"(kstok), "+s"(vspage),
               "+s"(vstok), "+s"(pages), "+s"(shift));
  const unsigned mask = (1u << shift) - 1;
  const unsigned gc = g * (D / 8), gs = g * (D / 4) / kFp4Block;   // the lane's part of an entry
  // a lane's offset in a run of 16 keys
  const unsigned k_off = c * ktok + gc, ks_off = c * kstok + gs, v_off = c * vtok + gc, vs_off = c * vstok + gs;
  while (at_block < end_block) {
  while (at_block >= seq_block + w.blocks()) {
    seq_block += w.blocks();
    w = plan.work<kStart>(a, ++s, LY::BM, LY::BN);
  }
  const int item = quotient(at_block - seq_block, w.nb), b0 = at_block - seq_block - item * w.nb;
  const int b1 = w.nb - b0 < end_block - at_block ? w.nb : b0 + (end_block - at_block);
  const int last_block = at_block - b0 + w.nb - 1;  // of the item
  at_block += b1 - b0;
  if (b1 <= kStart && !a.whole) continue;           // the blocks that stand for the start alone: the next workgroup's
  const int blk = b0 > kStart ? b0 - kStart : 0;
  const bool whole = a.whole || (blk == 0 && b1 == w.nb);
  const int tile = a.by_hk.div(item), h = item - tile * a.Hk;
  const AttnTile x = tile_of_rows(a, s, w.n0, w.cnt, w.pos0, tile * LY::BM, LY::BM);
  const int first_key = (x.lo / LY::BN + blk) * LY::BN, take = b1 - kStart - blk;
  const int k0 = __builtin_amdgcn_readfirstlane(first_key > x.lo ? first_key : x.lo);
  const int k1 = __builtin_amdgcn_readfirstlane(whole || (x.hi - first_key) / LY::BN < take ? x.hi
                                                                                          : first_key + take * LY::BN);
  const uint8_t* kb = static_cast<const uint8_t*>(a.kc) + h * a.kc_head;
  const uint8_t* vb = static_cast<const uint8_t*>(a.vc) + h * a.vc_head;
  const uint8_t* ksb = a.ks + h * a.k.head;
  const uint8_t* vsb = a.vs + h * a.v.head;
  char* vl = lds + wave * KT * LY::VLD;

  const int* trow = a.table + s * a.table_row;
  constexpr int STEP = 4 * KT;
  int j0 = (k0 / LY::BN) * LY::BN + wave * KT;
  Codes kr[2], vr[2];
  unsigned kf[2], vf[2];                            // scales
  unsigned okn = 0;                                 // which of the 32 keys exist (bit = key)
  int ids = 0, left = 0;                            // WIDE: page of a lane's run, iterations until the next lookup
  int id[2];                                        // else: pages of the lane's keys, looked up a block ahead, since
                                                    // looking at them sooner would wait for the loads under way
  auto lookup = [&](int j) {
    if constexpr (WIDE) {
      const int mine = j + (lane >> 1) * STEP + 16 * (lane & 1);
      ids = trow[(mine < k1 ? mine : k1 - 1) >> shift];
      left = 32;
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int mine = j + 16 * b + c;
        id[b] = trow[(mine < k1 ? mine : k1 - 1) >> shift];
      }
    }
  };
  // No branch between a load and the block's end: a scale would be widened behind it, and
  // waited for.
  auto fetch = [&](int j) {
    if constexpr (WIDE) {
      if (left == 0) lookup(j);
      const int at_id = 64 - 2 * left--;
      okn = 0;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const unsigned page = __builtin_amdgcn_readlane(ids, at_id + b);
        const int first = j + 16 * b;
        const int from = k0 - first < 0 ? 0 : k0 - first < 16 ? k0 - first : 16;
        const int to = k1 - first < from ? from : k1 - first < 16 ? k1 - first : 16;
        okn |= (page < pages ? (1u << to) - (1u << from) : 0u) << (16 * b);
        const unsigned pg = page < pages ? page : 0, off = first & mask;
        // a scalar base and 32 bits of a lane's own, which has to be seen here for the load to take them so
        auto run = [&](const uint8_t* base, unsigned page_bytes, unsigned tok_bytes, unsigned mine) {
          asm volatile("" : "+v"(mine));
          return base + ((uint64_t)pg * page_bytes + (uint64_t)off * tok_bytes) + mine;
        };
        kr[b] = *reinterpret_cast<const Codes*>(run(kb, kpage, ktok, k_off));
        kf[b] = *run(ksb, kspage, kstok, ks_off);
        vr[b] = *reinterpret_cast<const Codes*>(run(vb, vpage, vtok, v_off));
        vf[b] = *run(vsb, vspage, vstok, vs_off);
      }
    } else {
      bool ok[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int mine = j + 16 * b + c;
        ok[b] = mine >= k0 && mine < k1 && (unsigned)id[b] < pages;
        const unsigned pg = ok[b] ? id[b] : 0, off = mine & mask;
        auto key = [&](const uint8_t* base, unsigned page_bytes, unsigned tok_bytes, unsigned part) {
          return base + ((uint64_t)pg * page_bytes + (uint64_t)off * tok_bytes + part);
        };
        kr[b] = *reinterpret_cast<const Codes*>(key(kb, kpage, ktok, gc));
        kf[b] = *key(ksb, kspage, kstok, gs);
        vr[b] = *reinterpret_cast<const Codes*>(key(vb, vpage, vtok, gc));
        vf[b] = *key(vsb, vspage, vstok, gs);
      }
      okn = (unsigned)(__ballot(ok[0]) & 0xffffu) | (unsigned)(__ballot(ok[1]) & 0xffffu) << 16;
      lookup(j + STEP);
    }
  };
  if (j0 < k1) lookup(j0);

  // this lane's row and its queries
  const int row = x.row0 + (c < x.rows ? c : x.rows - 1);
  const int tok = a.by_g.div(row), p = x.pos0 + tok;
  const int p_min = x.pos0 + a.by_g.div(x.row0), p_max = x.pos0 + a.by_g.div(x.row0 + x.rows - 1);
  const int lo = first_seen(a, p, 0), lo_max = first_seen(a, p_max, 0);
  const unsigned seen = p >= lo ? p - lo + 1 : 0;   // keys the row sees, the last of them p
  const E* qp = static_cast<const E*>(a.q) + (int64_t)(x.n0 + tok) * a.q_row + (h * a.G + row - tok * a.G) * D +
                g * (D / 4);
  u32x4 q[NI][NQ];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if constexpr (NQ == 1) {
      q[i][0] = reinterpret_cast<const u32x4*>(qp)[i];
    } else {
      float y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) y[u] = qp[8 * i + u];
      cut_parts(y, q[i]);
    }
  }

  f32x4 o[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i] = zero4();
  float m = kNoMax, l = 0.f;
  if (j0 < k1) fetch(j0);
  for (; j0 < k1; j0 += STEP) {
    const unsigned ok = okn;
    f32x4 sc[2] = {zero4(), zero4()};
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const u32x4 k = fp4_open8(kr[b][i], fp4_factor(kf[b]));
#pragma unroll
        for (int u = 0; u < NQ; ++u) sc[b] = mma_bits(k, q[i][u], sc[b]);
      }
    // values to LDS; rows that do not exist as zeros
    if (ok != 0xffffffffu) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (!((ok >> (16 * b + c)) & 1u)) { vr[b] = Codes(0u); vf[b] = 127; }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < NI; ++i)
        *reinterpret_cast<u32x4*>(vl + (16 * b + c) * LY::VLD + g * (D / 2) + 16 * i) =
            fp4_open8(vr[b][i], fp4_factor(vf[b]));
    if (j0 + STEP < k1) fetch(j0 + STEP);
    // lane: row c, keys 16 b + 4 g + i
    if (ok != 0xffffffffu || j0 + KT - 1 > p_min || j0 < lo_max) {
      const unsigned mine = ok >> (4 * g);
      const int far = p - j0 - 4 * g;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool see = (mine >> (16 * b + i)) & 1u && (unsigned)(far - (16 * b + i)) < seen;
          sc[b][i] = see ? sc[b][i] : -__builtin_inff();
        }
    }
    float top = sc[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[b][i]);
    top = max_groups(top);
    if (__ballot((top - m) * a.c > kSlack)) {
      const float mn = fmaxf(m, top), al = fast_exp2((m - mn) * a.c);
      m = mn;
      l *= al;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i] *= al;
    }
    const float mc = m * a.c;
    float e[8];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[4 * b + i] = fast_exp2(sc[b][i] * a.c - mc);
        l += e[4 * b + i];
      }
    // The weights go in as bf16 parts: two (16 bits) where the output is bf16, which
    // costs nothing beside the loads, three (24) where it is fp32.
    u32x4 pw[LY::NP];
    if constexpr (LY::NP == 3) {
      cut_parts(e, pw);
    } else {
      bf16x8 hi, rest;
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[i] = (bf16)e[i];
      pw[0] = __builtin_bit_cast(u32x4, hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rest[2 * i] = (bf16)(e[2 * i] - __uint_as_float(pw[0][i] << 16));
        rest[2 * i + 1] = (bf16)(e[2 * i + 1] - __uint_as_float(pw[0][i] & 0xffff0000u));
      }
      pw[1] = __builtin_bit_cast(u32x4, rest);
    }
    const char* src = vl + (4 * g + (lane & 15) / 4) * LY::VLD + (lane & 3) * 8;
#pragma unroll
    for (int d = 0; d < D / 16; d += 2) {           // two at a time: a product does not wait for the one before it
      u32x4 v[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x2 v0 = __builtin_bit_cast(u32x2, read_tr(src + 32 * (d + t)));
        const u32x2 v1 = __builtin_bit_cast(u32x2, read_tr(src + 32 * (d + t) + 16 * LY::VLD));
        v[t] = u32x4{v0[0], v0[1], v1[0], v1[1]};
      }
#pragma unroll
      for (int u = 0; u < LY::NP; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) o[d + t] = mma_bits(v[t], pw[u], o[d + t]);
    }
  }

  // join the four waves (the last item's readers are past the barrier that ended it)
  const Fp4Args& z = args_again<Fp4Args>();
  const RowOut<E, D> ro{z, h, whole, (int64_t)(2 * blockIdx.x + (blk > 0 ? 0 : 1)) * LY::BM, 1};
  if (threadIdx.x == 0 && blk == 0 && !whole)
    note_item(z, x, h, plan.share(last_block) - blockIdx.x + 1);
  l = sum_halves(sum_row_pairs(l));
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
    float M = ms[0][r], Lr = 0.f, acc[D / 16];
#pragma unroll
    for (int w = 1; w < 4; ++w) M = fmaxf(M, ms[w][r]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = fast_exp2((ms[w][r] - M) * z.c);
      Lr += ls[w][r] * f;
#pragma unroll
      for (int i = 0; i < D / 16; i += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(ol + (w * 16 + r) * LY::OLD + t * (D / 16) + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[i + u] += v[u] * f;
      }
    }
    const int64_t at = ro.index(x, r);
    bool nf = odd_sum(Lr) || (Lr == 0.f && sees_any(z, x.pos0 + z.by_g.div(x.row0 + r), k0, k1));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) nf = nf || not_finite(acc[i]);
    if (nf) bad[r] = 1;
    if (ro.whole) {
      const float inv = Lr == 0.f ? 0.f : 1.f / Lr;
      E* out = ro.out(at) + t * (D / 16);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) out[i] = from_f32<E>(acc[i] * inv);
    } else {
      f32x4* out = reinterpret_cast<f32x4*>(ro.part(at, r) + t * (D / 16));
#pragma unroll
      for (int i = 0; i < D / 16; i += 4) out[i / 4] = f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
    }
    if (t == 0) ro.stats(at, r, M, Lr);
  }
  __syncthreads();
  for (int i = wave; i < x.rows; i += 4)
    if (bad[i]) careful_row(ro, Fp4Entries<E, D>(z, h), x, i, k0, k1);
  __syncthreads();                                  // the next item writes the same LDS
  }
}

// ---------------------------------------------------------------------------
// Many rows (bf16): the kernels of paged_attn.h over blocks that are opened to bf16 on
// their way from registers to LDS. A thread has 16 channels of a key, 8 bytes and a
// scale: 64 keys of 128 channels are one such piece for each of 512 threads, keys and
// values alike, 16 conversions and four 16-byte stores a step. What bounds those kernels
// bounds these (products, then what stands beside them); a quarter of the loads makes up
// for the conversions: 4096 tokens over 16384 keys, 16 on 4 heads of 128, 477 us (1.0
// PFLOP/s) where the bf16 cache takes 498; 8 prompts, window 1024, 12 on 4 heads of 64, 82
// and 88.
template <int D, int NW, bool WIDE>
struct Fp4Tiles : TileRows<D, NW, Fp4Args> {
  using R = TileRows<D, NW, Fp4Args>;
  using LY = typename R::LY;
  using Cache = Fp4Entries<bf16, D>;
  static constexpr int GPR = D / 16;                // pieces per key
  static constexpr int ST = LY::BN * GPR / LY::NT, RS = LY::NT / GPR, WR = 64 / GPR;   // as TileLayout has them
  struct Chunks { u32x2 codes[ST]; unsigned scale[ST]; };
  struct Place { unsigned page, off; };
  using R::a; using R::h; using R::first_b; using R::pmask;
  const uint8_t *kb, *vb, *ksb, *vsb;
  int sr, sc;

  __device__ __forceinline__ Fp4Tiles(const Fp4Args& a_) : R(a_) {
    kb = static_cast<const uint8_t*>(a.kc) + h * a.kc_head;
    vb = static_cast<const uint8_t*>(a.vc) + h * a.vc_head;
    ksb = a.ks + h * a.k.head;
    vsb = a.vs + h * a.v.head;
    sr = threadIdx.x / GPR;
    sc = threadIdx.x % GPR;
  }
  // Page (0 where there is none) and offset in it of the lane's key of block t.
  __device__ __forceinline__ Place place(int t, int id) const {
    return {(unsigned)id < (unsigned)a.pages ? (unsigned)id : 0u, (unsigned)((first_b + t) * LY::BN + lane_id()) & pmask};
  }
  __device__ __forceinline__ Place place_k(int t, int id) const { return place(t, id); }
  __device__ __forceinline__ Place place_v(int t, int id) const { return place(t, id); }
  // As PlainTiles::load: one load of a wave covers 8 keys (16 at d = 64), and in pages
  // that hold so many the first one's address is a scalar.
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t page, int64_t tok,
                                       const Fp4Strides& s, Place at, Chunks& r) const {
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      if constexpr (WIDE) {
        const int r0 = wave_id() * WR + RS * i;
        const unsigned pg = __builtin_amdgcn_readlane((int)at.page, r0), off = __builtin_amdgcn_readlane((int)at.off, r0);
        const unsigned row = lane_id() / GPR;
        const uint8_t* c = codes + (uint64_t)pg * (unsigned)page + (uint64_t)off * (unsigned)tok;
        const uint8_t* e = scales + (uint64_t)pg * (unsigned)s.page + (uint64_t)off * (unsigned)s.tok;
        r.codes[i] = *reinterpret_cast<const u32x2*>(c + (row * (unsigned)tok + sc * 8));
        r.scale[i] = e[row * (unsigned)s.tok + sc / 2];
      } else {
        const int rr = sr + RS * i;
        const unsigned pg = __shfl((int)at.page, rr), off = __shfl((int)at.off, rr);
        r.codes[i] = *reinterpret_cast<const u32x2*>(codes + ((uint64_t)pg * (unsigned)page +
                                                              (uint64_t)off * (unsigned)tok + sc * 8));
        r.scale[i] = scales[(uint64_t)pg * (unsigned)s.page + (uint64_t)off * (unsigned)s.tok + sc / 2];
      }
    }
  }
  __device__ __forceinline__ void load_k(Place at, Chunks& r) const { load(kb, ksb, a.kc_page, a.kc_tok, a.k, at, r); }
  __device__ __forceinline__ void load_v(Place at, Chunks& r) const { load(vb, vsb, a.vc_page, a.vc_tok, a.v, at, r); }
  // Zeros in the place of values whose key does not exist.
  __device__ __forceinline__ void clear(unsigned long long ok, Chunks& r) const {
    if (ok != ~0ull) {
#pragma unroll
      for (int i = 0; i < ST; ++i)
        if (!((ok >> (sr + RS * i)) & 1ull)) {
          r.codes[i] = u32x2{0, 0};
          r.scale[i] = 127;
        }
    }
  }
  __device__ __forceinline__ void store(char* block, int ld, const Chunks& r) const {
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      char* at = block + (sr + RS * i) * ld + sc * 32;
      const float f = fp4_factor(r.scale[i]);
      *reinterpret_cast<u32x4*>(at) = fp4_open8(r.codes[i][0], f);
      *reinterpret_cast<u32x4*>(at + 16) = fp4_open8(r.codes[i][1], f);
    }
  }
  __device__ __forceinline__ void store_k(char* block, const Chunks& r) const { store(block, LY::KLD, r); }
  __device__ __forceinline__ void store_v(char* block, const Chunks& r) const { store(block, LY::VLD, r); }
};

}  // namespace carve
