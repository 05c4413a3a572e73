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
  float x[V];
  Piece<E>::open(raw, x);
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) top = dpp_max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  byte = fp4_scale(block_max<kFp4Block / V>(top));
  const float s = fp4_factor(byte);
  unsigned c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
  if constexpr (V == 8) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
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

// As paged_append_kernel: one wave per token and 64 U pieces of its rows. A block's
// lanes (4, or 8 in fp32) find its largest value by lane exchanges; each stores its
// own codes, the first the scale.
template <typename E, int D, int U>
__global__ __launch_bounds__(256) void paged_append_fp4_kernel(Fp4AppendArgs f) {
  const AppendArgs& a = f.a;
  constexpr int V = Piece<E>::V, LPR = D / V;
  const int n = blockIdx.x * 4 + wave_id();
  if (n >= a.N) return;
  // the rows leave before the token's place is looked for, three loads that wait for each other
  const Turn<E, D> t(a.rot, a.interleaved);
  const int heads = a.Hq + 2 * a.Hk;
  u32x4 raw[U];
  int hh[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    hh[u] = ((blockIdx.y * U + u) * 64 + lane_id()) / LPR;
    const int h = hh[u] < heads ? hh[u] : heads - 1;
    const E* src = h < a.Hq ? static_cast<const E*>(a.q) + n * a.q_row + h * D
                   : h < a.Hq + a.Hk ? static_cast<const E*>(a.k) + n * a.k_row + (h - a.Hq) * D
                                     : static_cast<const E*>(a.v) + n * a.v_row + (h - a.Hq - a.Hk) * D;
    raw[u] = *reinterpret_cast<const u32x4*>(src + t.c * V);
  }
  const u32x4 wq = weight_piece<E, D>(a.wq, t.c), wk = weight_piece<E, D>(a.wk, t.c);
  const TokenPlace at = token_place(a, n);
  if (at.pos == kNoToken) return;                   // behind the last sequence
  float cs[V], sn[V];
  t.angles(a.cos, a.sin, a.rot, a.table_len, at.pos, false, cs, sn);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = hh[u];
    const u32x4 y = norm_rope_piece<E, D>(raw[u], t, h < a.Hq ? wq : wk, cs, sn, a.norm, a.eps);
    const bool isk = h < a.Hq + a.Hk;
    unsigned byte;
    const unsigned codes = fp4_close<E>(isk ? y : raw[u], byte);
    if (h < a.Hq) {
      *reinterpret_cast<u32x4*>(static_cast<E*>(a.qo) + n * a.qo_row + h * D + t.c * V) = y;
    } else if (h < heads && at.page >= 0) {
      const int hk = h - a.Hq - (isk ? 0 : a.Hk);
      uint8_t* c = isk ? static_cast<uint8_t*>(a.kc) + at.page * a.kc_page + at.off * a.kc_tok + hk * a.kc_head
                       : static_cast<uint8_t*>(a.vc) + at.page * a.vc_page + at.off * a.vc_tok + hk * a.vc_head;
      uint8_t* s = isk ? f.ks + at.page * f.k.page + at.off * f.k.tok + hk * f.k.head
                       : f.vs + at.page * f.v.page + at.off * f.v.tok + hk * f.v.head;
      if constexpr (V == 8) reinterpret_cast<unsigned*>(c)[t.c] = codes;
      else reinterpret_cast<uint16_t*>(c)[t.c] = (uint16_t)codes;
      if (t.c % (kFp4Block / V) == 0) s[t.c / (kFp4Block / V)] = (uint8_t)byte;
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
// Bound by memory: READ_NUMBERS
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
