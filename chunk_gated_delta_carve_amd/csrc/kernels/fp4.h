// Numbers of 4 bits in blocks of 32 with one scale, and what stores and reads
// them in a paged cache.
//
// A block x[0..31] has the scale 2^e, e the least with max |x| <= 7 2^e. Codes
// are a sign and the grid 0, 0.5, 1, 1.5, 2, 3, 4, 6; the nearest code of x / 2^e
// is off by at most 1 (7 and 5 to 6, half of the widest gap), so letting the
// largest value reach 7 costs nothing over stopping at 6, and halves every other
// value's error in the blocks with a maximum between 6 and 7. The exponent comes
// from the maximum's bits: with M = 2^k (1 + f), e = k - 2 where f <= 3/4, else
// k - 1. It is kept in [-125, 125], so that every value is a normal number or 0,
// and finite. gfx950 converts two values an instruction, either way.
#pragma once
#include "assign.h"
#include "common.h"
#include "rope.h"

namespace carve {

constexpr int kFp4Block = 32;
constexpr unsigned kFp4Bad = 255, kFp4Least = 2, kFp4Most = 252;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// The scale's byte of a block whose largest |x| has these bits.
__device__ __forceinline__ unsigned fp4_scale(unsigned top) {
  if (top >= 0x7f800000u) return kFp4Bad;
  const unsigned k = (top + 0x1fffffu) >> 23;       // exponent, one more where f > 3/4
  const unsigned e = k > 2 ? k - 2 : 0;
  return e < kFp4Least ? kFp4Least : e > kFp4Most ? kFp4Most : e;
}
// As an operand of the conversions, which look at the exponent alone (255: NaN).
__device__ __forceinline__ float fp4_factor(unsigned byte) { return __uint_as_float(byte << 23); }

// max of the lanes of a block's values, W neighbouring lanes to a block (4 or 8)
__device__ __forceinline__ unsigned dpp_max(unsigned x, unsigned y) { return x > y ? x : y; }
template <int CTRL>
__device__ __forceinline__ unsigned dpp_bits(unsigned x) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}
template <int W>
__device__ __forceinline__ unsigned block_max(unsigned x) {
  x = dpp_max(x, dpp_bits<0xB1>(x));                // lane xor 1
  x = dpp_max(x, dpp_bits<0x4E>(x));                // xor 2
  if constexpr (W > 4) x = dpp_max(x, dpp_bits<0x141>(x));   // mirrored in 8 lanes: the other quad's
  return x;
}

// A lane's 16-byte piece of a row (V values, 32 / V lanes to a block): its codes in
// the low 4 V bits, and the block's scale byte.
template <typename E>
__device__ __forceinline__ unsigned fp4_close(u32x4 raw, unsigned& byte) {
  constexpr int V = Piece<E>::V;
  unsigned top = 0, c = 0;
  if constexpr (V == 8) {                           // bf16: two maxima at a time, and converted as they are
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    auto size = [](unsigned x) { return __builtin_bit_cast(u16x2, x & 0x7fff7fffu); };
    const u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(size(raw[0]), size(raw[1])),
                                              __builtin_elementwise_max(size(raw[2]), size(raw[3])));
    top = (unsigned)(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) top = dpp_max(top, raw[i] & 0x7fffffffu);
  }
  byte = fp4_scale(block_max<kFp4Block / V>(top));
  const float s = fp4_factor(byte);
  if constexpr (V == 8) {
    auto two = [](unsigned x) { return __builtin_bit_cast(bf16x2, x); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(raw[0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(raw[1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(raw[2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, two(raw[3]), s, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(raw[0]), __uint_as_float(raw[1]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(raw[2]), __uint_as_float(raw[3]), s, 1);
  }
  return byte == kFp4Bad ? 0u : c;
}

// Eight codes as values.
__device__ __forceinline__ u32x4 fp4_open8(unsigned c, float s) {
  auto two = [](bf16x2 x) { return __builtin_bit_cast(unsigned, x); };
  return u32x4{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
               two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
}
__device__ __forceinline__ void fp4_open8(unsigned c, float s, float (&x)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
              d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  x[0] = a[0]; x[1] = a[1]; x[2] = b[0]; x[3] = b[1];
  x[4] = d[0]; x[5] = d[1]; x[6] = e[0]; x[7] = e[1];
}

// Where a head's codes and scales of an entry are.
struct Fp4Strides { int64_t page, tok, head; };

struct Fp4AppendArgs {
  AppendArgs a;                        // kc, vc: codes, strides in bytes
  uint8_t *ks, *vs;
  Fp4Strides k, v;                     // of the scales
};

// Where a new token goes: its position and its entry in the cache, page -1 where it has none.
struct TokenPlace { int64_t pos, page, off; };
constexpr int64_t kNoToken = INT64_MIN;             // position of a token behind the last sequence

// Where the TOK tokens from n0 on go, lane l for token l % TOK. What tells their sequences
// is loaded ahead of the wave's rows, since loads come back in the order they went out: up
// to 64 sequences a lane has one of them, beyond a lane looks its token's up.
template <int TOK>
struct TokenSeeker {
  int s, c0, c1, kv;
  __device__ __forceinline__ TokenSeeker(const AppendArgs& a, int n0) {
    const int n = n0 + lane_id() % TOK;
    s = a.cu ? lane_id() : n;
    if (a.cu && a.S > 64) s = last_at(a.cu, a.S, (unsigned)n);
    s = s < a.S ? s : a.S - 1;
    c0 = a.cu ? a.cu[s] : s;
    c1 = a.cu ? a.cu[s + 1] : s + 1;
    kv = a.kv_lens[s];
  }
  __device__ __forceinline__ TokenPlace places(const AppendArgs& a, int n0) const {
    const int n = n0 + lane_id() % TOK;
    int in = s, b = c0, e = c1, len = kv;
    if (a.cu && a.S <= 64) {
#pragma unroll
      for (int k = 0; k < TOK; ++k) {
        const int over = __popcll(__ballot(lane_id() < a.S && c1 <= n0 + k)), t = over < a.S ? over : a.S - 1;
        const int tb = __builtin_amdgcn_readlane(c0, t), te = __builtin_amdgcn_readlane(c1, t);
        const int tl = __builtin_amdgcn_readlane(kv, t);
        const bool mine = lane_id() % TOK == k;
        in = mine ? t : in; b = mine ? tb : b; e = mine ? te : e; len = mine ? tl : len;
      }
    }
    TokenPlace x{kNoToken, -1, 0};
    if (n >= a.N || n < b || n >= e) return x;      // behind the last sequence
    x.pos = (int64_t)len - e + n;
    const int64_t slot = x.pos >> a.page_shift;
    if (x.pos >= 0 && slot < a.width) x.page = a.table[in * a.table_row + slot];
    if (x.page >= a.pages) x.page = -1;
    x.off = x.pos & ((1 << a.page_shift) - 1);
    return x;
  }
};

// A wave has 64 U pieces of each of TOK neighbouring tokens (q's, k's and v's heads): all
// of the rows are under way while lanes look for the tokens' places. A block's lanes (4, or
// 8 in fp32) find its largest value by lane exchanges; each stores its own codes, the first
// the scale. Bound by instructions, then by the trips to memory that wait for each other
// (lengths; rows and page; the stores): 22,044 tokens of 8 heads of 128 in bf16 (57 MB read
// and written) took 28 us with a 64-bit product for every stride and piece, 18 with a
// token's part as scalars and a head's found once for all tokens, and take 15 (3.8 TB/s)
// with sequences found in one trip and without what norm and rotation need (TURN) where
// there is neither (16.3 with it); 64 single tokens 3.5.
template <typename E, int D, int U, int TOK, bool TURN>
__global__ __launch_bounds__(256) void paged_append_fp4_kernel(Fp4AppendArgs f) {
  const AppendArgs& a = f.a;
  constexpr int V = Piece<E>::V, LPR = D / V;
  const int n0 = (blockIdx.x * 4 + wave_id()) * TOK;
  if (n0 >= a.N) return;
  const TokenSeeker<TOK> seek(a, n0);
  const Turn<E, D> t(a.rot, a.interleaved);
  const int heads = a.Hq + 2 * a.Hk;
  u32x4 raw[TOK][U];
  int hh[U];
  // a head's place within an entry's page and token, found once for all tokens
  uint64_t code_at[U], scale_at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    hh[u] = ((blockIdx.y * U + u) * 64 + lane_id()) / LPR;
    const int h = hh[u] < heads ? hh[u] : heads - 1;
    const bool isq = h < a.Hq, isk = h < a.Hq + a.Hk;
    const E* src = isq ? static_cast<const E*>(a.q) : static_cast<const E*>(isk ? a.k : a.v);
    const unsigned hk = isq ? h : h - a.Hq - (isk ? 0 : a.Hk), row = isq ? a.q_row : isk ? a.k_row : a.v_row;
    src += hk * D + t.c * V;
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
      const unsigned n = n0 + k < a.N ? n0 + k : a.N - 1;
      raw[k][u] = *reinterpret_cast<const u32x4*>(src + (uint64_t)n * row);
    }
    code_at[u] = (uint64_t)hk * (unsigned)(isk ? a.kc_head : a.vc_head) + t.c * (V / 2);
    scale_at[u] = (uint64_t)hk * (unsigned)(isk ? f.k.head : f.v.head) + t.c / (kFp4Block / V);
  }
  u32x4 wq{}, wk{};
  if constexpr (TURN) { wq = weight_piece<E, D>(a.wq, t.c); wk = weight_piece<E, D>(a.wk, t.c); }
  const TokenPlace mine = seek.places(a, n0);
#pragma unroll
  for (int k = 0; k < TOK; ++k) {
    const int64_t n = n0 + k;
    // the token's place is the wave's: scalars
    const int pos_hi = __builtin_amdgcn_readlane((int)(mine.pos >> 32), k);
    const int64_t pos = (int64_t)pos_hi << 32 | (unsigned)__builtin_amdgcn_readlane((int)mine.pos, k);
    if (pos == kNoToken) continue;                  // behind the last sequence
    const int page = __builtin_amdgcn_readlane((int)mine.page, k);
    const unsigned off = __builtin_amdgcn_readlane((int)mine.off, k), pg = page >= 0 ? page : 0;
    auto token = [&](void* base, int64_t page_bytes, int64_t tok_bytes) {
      return static_cast<uint8_t*>(base) + (uint64_t)pg * (unsigned)page_bytes + (uint64_t)off * (unsigned)tok_bytes;
    };
    uint8_t *kc = token(a.kc, a.kc_page, a.kc_tok), *vc = token(a.vc, a.vc_page, a.vc_tok);
    uint8_t *ks = token(f.ks, f.k.page, f.k.tok), *vs = token(f.vs, f.v.page, f.v.tok);
    float cs[V], sn[V];
    if constexpr (TURN) t.angles(a.cos, a.sin, a.rot, a.table_len, pos, false, cs, sn);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hh[u];
      const bool isq = h < a.Hq, isk = h < a.Hq + a.Hk;
      u32x4 y = raw[k][u];
      if constexpr (TURN) {
        if (__ballot(isk)) {
          const u32x4 z = norm_rope_piece<E, D>(y, t, isq ? wq : wk, cs, sn, a.norm, a.eps);
          y = isk ? z : y;
        }
      }
      if (isq) *reinterpret_cast<u32x4*>(static_cast<E*>(a.qo) + n * a.qo_row + h * D + t.c * V) = y;
      if (page < 0 || !__ballot(!isq)) continue;
      unsigned byte;
      const unsigned codes = fp4_close<E>(y, byte);
      if (isq || h >= heads) continue;
      uint8_t *c = (isk ? kc : vc) + code_at[u], *s = (isk ? ks : vs) + scale_at[u];
      if constexpr (V == 8) *reinterpret_cast<unsigned*>(c) = codes;
      else *reinterpret_cast<uint16_t*>(c) = (uint16_t)codes;
      if (t.c % (kFp4Block / V) == 0) *s = (uint8_t)byte;
    }
  }
}

struct Fp4ReadArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const int64_t* slots;
  void *k, *v;
  Fp4Strides kcs, kss, vcs, vss;
  int64_t k_row, v_row, entries;       // entries: pages page_size
  int N, Hk, heads, page_shift;        // heads: of k and v, those that are asked for
};

// A piece is 16 bytes of output; the pieces of all slots and heads (a slot's k heads,
// then its v heads) are laid end to end over the workgroups, kReadPieces of them in
// flight to a lane, and the tokens of a workgroup's use the lines they read together.
// Bound by memory: 235,608 slots of 2 heads of 128 in bf16 (307 MB) 61 us, 5.0 TB/s; a
// wave to a slot, which leaves one load under way, took 105.
constexpr int kReadPieces = 4, kReadThreads = 256;
template <typename E, int D>
__global__ __launch_bounds__(kReadThreads) void paged_read_fp4_kernel(Fp4ReadArgs a) {
  constexpr int V = Piece<E>::V, LPR = D / V, U = kReadPieces;
  const unsigned per = a.heads * LPR;               // pieces of a slot
  const int64_t first = (int64_t)blockIdx.x * (kReadThreads * U), n0 = first / per;
  const unsigned rest = (unsigned)(first - n0 * per);
  const unsigned mask = (1u << a.page_shift) - 1;
  int64_t n[U], slot[U];
  unsigned piece[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned i = rest + u * kReadThreads + threadIdx.x, k = i / per;
    n[u] = n0 + k;
    piece[u] = i - k * per;
    slot[u] = n[u] < a.N ? a.slots[n[u]] : -1;
  }
  unsigned codes[U], byte[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned hh = piece[u] / LPR, c = piece[u] % LPR;
    const bool isk = a.k && hh < (unsigned)a.Hk;
    const unsigned h = isk || !a.k ? hh : hh - a.Hk;
    codes[u] = byte[u] = 0;
    if (slot[u] >= 0 && slot[u] < a.entries) {
      const unsigned page = (unsigned)(slot[u] >> a.page_shift), off = (unsigned)slot[u] & mask;
      auto entry = [&](const uint8_t* base, const Fp4Strides& s) {
        return base + ((uint64_t)page * (unsigned)s.page + (uint64_t)off * (unsigned)s.tok + (uint64_t)h * (unsigned)s.head);
      };
      const uint8_t* pc = entry(isk ? a.kc : a.vc, isk ? a.kcs : a.vcs);
      if constexpr (V == 8) codes[u] = reinterpret_cast<const unsigned*>(pc)[c];
      else codes[u] = reinterpret_cast<const uint16_t*>(pc)[c];
      byte[u] = entry(isk ? a.ks : a.vs, isk ? a.kss : a.vss)[c / (kFp4Block / V)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (n[u] >= a.N) continue;
    const unsigned hh = piece[u] / LPR, c = piece[u] % LPR;
    const bool isk = a.k && hh < (unsigned)a.Hk;
    const unsigned h = isk || !a.k ? hh : hh - a.Hk;
    E* dst = isk ? static_cast<E*>(a.k) + n[u] * a.k_row + h * D : static_cast<E*>(a.v) + n[u] * a.v_row + h * D;
    u32x4 y;
    if constexpr (V == 8) {
      y = fp4_open8(codes[u], fp4_factor(byte[u]));
    } else {
      float x[8];
      fp4_open8(codes[u], fp4_factor(byte[u]), x);
      y = Piece<float>::close({x[0], x[1], x[2], x[3]});
    }
    *reinterpret_cast<u32x4*>(dst + c * V) = y;
  }
}

}  // namespace carve
