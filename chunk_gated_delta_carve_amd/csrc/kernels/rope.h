// Per-head norm and rotation of queries and keys (forward and gradient), and
// the append of keys and values to a paged cache with both applied on the way.
//
// A row is one head of one token, x in R^d. With r = (mean x^2 + eps)^{-1/2}
// (1 without the norm) and per-channel weights w (1 when absent):
//   z = x r w,   y = R(p) z
// where R(p) turns `rot` / 2 pairs of channels by the angles of position p,
// whose cosines and sines the caller tabulates. Pairs are (i, i + rot/2), or
// (2i, 2i + 1) when interleaved; channels from `rot` on are not turned.
// Gradient: dz = R(p)^T dy, dw = sum over rows of dz x r, and with n = x r,
// dn = dz w:  dx = r (dn - n mean(dn n)).
//
// Every lane holds one 16-byte piece of a row, so a row is D sizeof(E) / 16
// neighbouring lanes, its sums are lane exchanges inside them, and in the
// half-split form a lane gets its partner channels from the lane that holds them:
// each input byte is read once. Forward, a wave takes the heads of one token, so
// the position, the angles and (for the cache) the page are found once for up to
// 256 pieces. All of it is bound by memory once an instruction count of about 120
// per piece is out of the way: a wave per token took the forward pass of 8192
// tokens, 24 heads of 64 from 15.6 us (a lane per row piece, 250 instructions) to
// 12.4 us.
#pragma once
#include "common.h"

namespace carve {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

struct RopeArgs {
  const void *q, *k, *wq, *wk;         // inputs and their weights (NULL: ones)
  const float *cos, *sin;              // [table_len][rot / 2]
  const int* positions;                // [N], or NULL: token n is at n mod T
  void *qo, *ko;                       // forward: outputs; backward: gradients of the outputs (read)
  void *dq, *dk;                       // backward: gradients of q and k
  float* part;                         // backward: per-block weight sums [blocks][d]
  int64_t N, q_row, k_row, qo_row, ko_row, dq_row, dk_row;   // elements between tokens
  int T, Hq, Hk, rot, table_len;
  int blocks_q, blocks;                // blocks [0, blocks_q) take q's rows, the rest k's
  int interleaved, norm;
  float eps;
};

template <typename E> struct Piece;    // 16 bytes of a row
template <> struct Piece<bf16> {
  static constexpr int V = 8;
  __device__ __forceinline__ static void open(u32x4 r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(r[i] << 16);
      x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static u32x4 close(const float (&x)[8]) {   // the one rounding: nearest even
    const bf16x8 b = {(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3], (bf16)x[4], (bf16)x[5], (bf16)x[6], (bf16)x[7]};
    return __builtin_bit_cast(u32x4, b);
  }
};
template <> struct Piece<float> {
  static constexpr int V = 4;
  __device__ __forceinline__ static void open(u32x4 r, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r[i]);
  }
  __device__ __forceinline__ static u32x4 close(const float (&x)[4]) {
    return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
  }
};

// sum over the W neighbouring lanes of a row (W = 8, 16 or 32), in each of them
template <int W>
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_mov<0xB1>(x);                            // lane xor 1
  x += dpp_mov<0x4E>(x);                            // xor 2: the quads' sums
  x += dpp_mov<0x141>(x);                           // mirrored in 8 lanes: the other quad's
  if constexpr (W > 8) x += dpp_mov<0x140>(x);      // mirrored in 16
  if constexpr (W > 16) x = sum_row_pairs(x);
  return x;
}

// What a lane does in a rotation: which piece it holds, which lane holds the
// partners of its channels, and where its angles are.
template <typename E, int D>
struct Turn {
  static constexpr int V = Piece<E>::V, LPR = D / V;
  int c, partner;
  int angle;                           // first table column
  bool turns, all;                     // whether the piece is rotated at all; whether every piece of a row is
  bool inter;
  float sign;                          // half-split: -1 in the first half, +1 in the second
  __device__ __forceinline__ Turn(int rot, bool interleaved) : inter(interleaved) {
    const int lane = lane_id(), half = rot / 2 / V;          // pieces per half
    c = lane % LPR;
    turns = c * V < rot;
    all = rot == D;
    if (inter) {
      partner = lane; angle = c * (V / 2); sign = 0.f;
    } else {
      const bool up = c >= half;
      partner = !turns ? lane : up ? lane - half : lane + half;
      angle = (up ? c - half : c) * V;
      sign = up ? 1.f : -1.f;
    }
  }
  // Cosines of the lane's channels at position p and sines with the sign that
  // y = z cos + partner sin has them with (back: of the inverse rotation). A
  // position outside the table turns by NaN, so its outputs are NaN.
  __device__ __forceinline__ void angles(const float* cos, const float* sin, int rot, int table_len, int64_t p,
                                         bool back, float (&cs)[V], float (&sn)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
    if (!turns) return;
    if (p < 0 || p >= table_len) {
#pragma unroll
      for (int i = 0; i < V; ++i) cs[i] = sn[i] = __builtin_nanf("");
      return;
    }
    const float* pc = cos + p * (rot / 2) + angle;
    const float* ps = sin + p * (rot / 2) + angle;
    const float b = back ? -1.f : 1.f;
    if (inter) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        cs[2 * i] = cs[2 * i + 1] = pc[i];
        sn[2 * i] = -b * ps[i];
        sn[2 * i + 1] = b * ps[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(pc + i), y = *reinterpret_cast<const f32x4*>(ps + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) { cs[i + j] = x[j]; sn[i + j] = b * sign * y[j]; }
      }
    }
  }
  // y = z cos + partner sin, rounded in this order for every caller
  __device__ __forceinline__ void turn(const float (&z)[V], const float (&cs)[V], const float (&sn)[V],
                                       float (&y)[V]) const {
#pragma clang fp contract(off)
    float zp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) zp[i] = inter ? z[i ^ 1] : __shfl(z[i], partner);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = __builtin_fmaf(z[i], cs[i], zp[i] * sn[i]);
    if (!all) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = turns ? y[i] : z[i];
    }
  }
};

// A lane's piece of a weight vector, or of ones.
template <typename E, int D>
__device__ __forceinline__ u32x4 weight_piece(const void* w, int c) {
  constexpr unsigned one = sizeof(E) == 2 ? 0x3f803f80u : 0x3f800000u;
  return w ? static_cast<const u32x4*>(w)[c] : u32x4{one, one, one, one};
}

// The one place that norms and rotates forward, for both entry points that do:
// products and sums are fused where they say so and nowhere else, so both give
// the same bits.
template <typename E, int D>
__device__ __forceinline__ u32x4 norm_rope_piece(u32x4 raw, const Turn<E, D>& t, u32x4 weight,
                                                 const float (&cs)[Piece<E>::V], const float (&sn)[Piece<E>::V],
                                                 bool norm, float eps) {
#pragma clang fp contract(off)
  constexpr int V = Piece<E>::V, LPR = D / V;
  float x[V], y[V];
  Piece<E>::open(raw, x);
  if (norm) {
    float w[V];
    Piece<E>::open(weight, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss = __builtin_fmaf(x[i], x[i], ss);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum<LPR>(ss), 1.f / D, eps));   // within 2^-23
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = x[i] * r * w[i];
  }
  t.turn(x, cs, sn, y);
  return Piece<E>::close(y);
}

constexpr int kRopeThreads = 256, kRopePieces = 4;   // most pieces per lane of a forward wave

// One wave per token and 64 U pieces of its rows (q's heads, then k's).
template <typename E, int D, int U>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(RopeArgs a) {
  constexpr int V = Piece<E>::V, LPR = D / V;
  const int64_t n = (int64_t)blockIdx.x * (kRopeThreads / 64) + wave_id();
  if (n >= a.N) return;
  const Turn<E, D> t(a.rot, a.interleaved);
  const int heads = a.Hq + a.Hk;
  u32x4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int hh = ((blockIdx.y * U + u) * 64 + lane_id()) / LPR, h = hh < heads ? hh : heads - 1;
    const E* src = h < a.Hq ? static_cast<const E*>(a.q) + n * a.q_row + h * D
                            : static_cast<const E*>(a.k) + n * a.k_row + (h - a.Hq) * D;
    raw[u] = *reinterpret_cast<const u32x4*>(src + t.c * V);
  }
  const int64_t p = a.positions ? a.positions[n] : n % a.T;
  float cs[V], sn[V];
  t.angles(a.cos, a.sin, a.rot, a.table_len, p, false, cs, sn);
  const u32x4 wq = weight_piece<E, D>(a.wq, t.c), wk = weight_piece<E, D>(a.wk, t.c);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = ((blockIdx.y * U + u) * 64 + lane_id()) / LPR;
    const u32x4 y = norm_rope_piece<E, D>(raw[u], t, h < a.Hq ? wq : wk, cs, sn, a.norm, a.eps);
    if (h >= heads) continue;
    E* dst = h < a.Hq ? static_cast<E*>(a.qo) + n * a.qo_row + h * D
                      : static_cast<E*>(a.ko) + n * a.ko_row + (h - a.Hq) * D;
    *reinterpret_cast<u32x4*>(dst + t.c * V) = y;
  }
}

// Gradient: the blocks of each tensor walk its rows with a grid stride; a lane
// meets the same channels in every row, so it sums its dw in registers and the
// block's row slots are added once at the end. Per-block sums go to `part` and
// norm_rope_dw_kernel adds them in a fixed order: no atomics, the same bits
// every call. B4 T8192, 20 heads of 128 (507 MB): 104 us, 4.9 TB/s, and 5 us for
// the sums.
template <typename E, int D>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_bwd_kernel(RopeArgs a) {
  constexpr int V = Piece<E>::V, LPR = D / V, RPB = kRopeThreads / LPR;
  const bool isq = (int)blockIdx.x < a.blocks_q;
  const unsigned H = isq ? a.Hq : a.Hk;
  const int64_t rows = a.N * H, x_row = isq ? a.q_row : a.k_row, dy_row = isq ? a.qo_row : a.ko_row,
                dx_row = isq ? a.dq_row : a.dk_row;
  const E* x_ = static_cast<const E*>(isq ? a.q : a.k);
  const E* dy_ = static_cast<const E*>(isq ? a.qo : a.ko);
  E* dx_ = static_cast<E*>(isq ? a.dq : a.dk);
  const void* w = isq ? a.wq : a.wk;
  const Turn<E, D> t(a.rot, a.interleaved);
  float wo[V], dw[V];
  Piece<E>::open(weight_piece<E, D>(w, t.c), wo);
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = 0.f;
  const int block = isq ? blockIdx.x : blockIdx.x - a.blocks_q, blocks = isq ? a.blocks_q : a.blocks - a.blocks_q;
  for (int64_t row = (int64_t)block * RPB + threadIdx.x / LPR; row - threadIdx.x / LPR < rows;
       row += (int64_t)blocks * RPB) {
    const bool in = row < rows;                    // lanes past the end run along (the shuffles need whole rows)
    const int64_t rr = in ? row : rows - 1;
    const int64_t n = (unsigned)rr / H;
    const int64_t h = (unsigned)rr - (unsigned)n * H;
    const u32x4 xr = *reinterpret_cast<const u32x4*>(x_ + n * x_row + h * D + t.c * V);
    const u32x4 gr = *reinterpret_cast<const u32x4*>(dy_ + n * dy_row + h * D + t.c * V);
    const int64_t p = a.positions ? a.positions[n] : (unsigned)n % (unsigned)a.T;
    float cs[V], sn[V], x[V], g[V], dz[V];
    t.angles(a.cos, a.sin, a.rot, a.table_len, p, true, cs, sn);
    Piece<E>::open(xr, x);
    Piece<E>::open(gr, g);
    t.turn(g, cs, sn, dz);
    if (a.norm) {
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) { ss += x[i] * x[i]; dot += dz[i] * wo[i] * x[i]; }
      ss = row_sum<LPR>(ss);
      dot = row_sum<LPR>(dot);
      const float r = __builtin_amdgcn_rsqf(ss * (1.f / D) + a.eps);
      const float m = dot * r * (1.f / D);         // mean(dn n)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float nn = x[i] * r;
        if (in) dw[i] += dz[i] * nn;
        dz[i] = r * (dz[i] * wo[i] - nn * m);
      }
    }
    if (in) *reinterpret_cast<u32x4*>(dx_ + n * dx_row + h * D + t.c * V) = Piece<E>::close(dz);
  }
  if (!w || !a.part) return;                       // uniform over the block
  __shared__ float sum[RPB * D];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[threadIdx.x / LPR * D + t.c * V + i] = dw[i];
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kRopeThreads) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < RPB; ++j) s += sum[j * D + i];
    a.part[(int64_t)blockIdx.x * D + i] = s;
  }
}

constexpr int kDwThreads = 1024, kDwCols = 8;

// Sums the per-block weight gradients: one block per 8 columns of dq_weight
// (blockIdx.y = 0) or dk_weight (1), 128 strips of blocks per column.
template <int D>
__global__ __launch_bounds__(kDwThreads) void norm_rope_dw_kernel(const float* part, int blocks_q, int blocks,
                                                                  float* dwq, float* dwk) {
  constexpr int S = kDwThreads / kDwCols;
  float* out = blockIdx.y ? dwk : dwq;
  if (!out) return;
  const int b0 = blockIdx.y ? blocks_q : 0, b1 = blockIdx.y ? blocks : blocks_q;
  const int col = threadIdx.x % kDwCols, strip = threadIdx.x / kDwCols;
  float s = 0.f;
  for (int b = b0 + strip; b < b1; b += S) s += part[(int64_t)b * D + blockIdx.x * kDwCols + col];
  __shared__ float sum[S][kDwCols];
  sum[strip][col] = s;
  __syncthreads();
  for (int h = S / 2; h > 0; h >>= 1) {
    if (strip < h) sum[strip][col] += sum[strip + h][col];
    __syncthreads();
  }
  if (strip == 0) out[blockIdx.x * kDwCols + col] = sum[0][col];
}

// ---------------------------------------------------------------------------
// Paged caches

// Index of the sequence that holds token n, by 64-way probing of the offsets
// cu[0 .. S]: the number of s with cu[s + 1] <= n. S when n lies behind the last
// sequence. Wave-uniform; the whole wave takes part.
__device__ __forceinline__ int find_sequence(const int* cu, int S, int n) {
  int lo = 0, len = S;                              // the answer is in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int at = (lane_id() + 1) * step;          // probes sequence lo + at - 1
    const bool past = at <= len && cu[lo + at] <= n;
    const int k = __popcll(__ballot(past));         // that many probes lie before n
    lo += k * step;
    len = step - 1 < len - k * step ? step - 1 : len - k * step;
  }
  return lo;
}

struct AppendArgs {
  const void *k, *v, *q, *wq, *wk;
  const float *cos, *sin;
  const int *cu, *kv_lens, *table;
  void *kc, *vc, *qo;
  int64_t k_row, v_row, q_row, qo_row, table_row;
  int64_t kc_page, kc_tok, kc_head, vc_page, vc_tok, vc_head;
  int N, S, Hq, Hk, rot, table_len, width, pages, page_shift;
  int interleaved, norm;
  float eps;
};

// One wave per token and 64 U pieces of its rows (q's, k's and v's heads): the
// sequence, position and page are found once per wave. A token whose position
// is negative, lies past the block table or falls on a page number outside the
// cache is not stored. 17k tokens of 24 heads of 128 (222 MB): 41 us, 5.4 TB/s.
template <typename E, int D, int U>
__global__ __launch_bounds__(256) void paged_append_kernel(AppendArgs a) {
  constexpr int V = Piece<E>::V, LPR = D / V;
  const int n = blockIdx.x * 4 + wave_id();
  if (n >= a.N) return;
  int s = n, i = 0, cnt = 1;
  if (a.cu) {
    s = find_sequence(a.cu, a.S, n);
    if (s < a.S) { i = n - a.cu[s]; cnt = a.cu[s + 1] - a.cu[s]; }
  }
  if (s >= a.S || i < 0) return;                    // behind the last sequence
  const int64_t pos = (int64_t)a.kv_lens[s] - cnt + i;
  const int64_t slot = pos >> a.page_shift;
  int page = -1;
  if (pos >= 0 && slot < a.width) page = a.table[s * a.table_row + slot];
  const bool stored = page >= 0 && page < a.pages;
  const int64_t off = pos & ((1 << a.page_shift) - 1);
  const Turn<E, D> t(a.rot, a.interleaved);
  const int heads = a.Hq + 2 * a.Hk;
  float cs[V], sn[V];
  t.angles(a.cos, a.sin, a.rot, a.table_len, pos, false, cs, sn);
  const u32x4 wq = weight_piece<E, D>(a.wq, t.c), wk = weight_piece<E, D>(a.wk, t.c);
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
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = hh[u];
    const u32x4 y = norm_rope_piece<E, D>(raw[u], t, h < a.Hq ? wq : wk, cs, sn, a.norm, a.eps);
    if (h < a.Hq) {
      *reinterpret_cast<u32x4*>(static_cast<E*>(a.qo) + n * a.qo_row + h * D + t.c * V) = y;
    } else if (h < heads && stored) {
      const bool isk = h < a.Hq + a.Hk;
      E* dst = isk ? static_cast<E*>(a.kc) + page * a.kc_page + off * a.kc_tok + (h - a.Hq) * a.kc_head
                   : static_cast<E*>(a.vc) + page * a.vc_page + off * a.vc_tok + (h - a.Hq - a.Hk) * a.vc_head;
      *reinterpret_cast<u32x4*>(dst + t.c * V) = isk ? y : raw[u];
    }
  }
}

}  // namespace carve
