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
    // lane l has channels l PER on: half a byte at d = 64
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

// A wave per (token, query head), key by key.
template <typename E, int D>
__global__ __launch_bounds__(256) void paged_each_fp4_kernel(Fp4Args a) {
  const int n = blockIdx.x, qh = blockIdx.y * 4 + wave_id();
  if (qh >= a.Hq) return;
  int s = n, n0 = n, cnt = 1;
  if (a.cu) {
    s = find_sequence(a.cu, a.S, n);
    if (s >= a.S || n < a.cu[s]) return;
    n0 = a.cu[s];
    cnt = (a.cu[s + 1] < a.N ? a.cu[s + 1] : a.N) - n0;
  }
  const int h = qh / a.G;
  const AttnTile x = tile_of_rows(a, s, n0, cnt, first_position(a, s, cnt), (n - n0) * a.G + qh % a.G, 1);
  const RowOut<E, D> ro{a, h, true, 0, 0};
  careful_row(ro, Fp4Entries<E, D>(a, h), x, 0, x.lo, x.hi);
}

}  // namespace carve
