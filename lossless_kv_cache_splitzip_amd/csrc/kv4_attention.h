// Attention over the 4-bit cache (splitzip_kv4_attention).
//
// Everything is held transposed: S^T = K Q^T and O^T = V^T P^T, on 16x16x32
// matrix instructions.  The contraction index of such a product may be
// permuted at will as long as both operands agree, which is what makes the
// cache's bytes fit the operands without a shuffle:
//   * K as the left operand: lane (i, j) (i = lane % 16, j = lane / 16) holds
//     8 channels of key i.  Its channels are a run of min(32, D/4), one wide
//     load of K codes, all under one scale byte; the products' channel order
//     is (step, j, 8 channels) and Q is loaded in the same order.
//   * S^T leaves lane (n, j) with the logits of query row n and keys 4j ..
//     4j + 3 of each 16: two such tiles are the right operand of O^T for 32
//     keys in the order (j: 4 of the first 16, 4 of the second 16).
//   * V^T as the left operand needs 8 tokens of one channel per lane in that
//     order: the cache's V section keeps 4 tokens x D/16 channels together, so
//     a lane loads them at once, converts pairs of channels under each
//     token's scale and exchanges halves between tokens.
// E2M1 values times powers of two are exact in BF16, and so are products of
// BF16 in FP32.  FP16 queries (11 bits) are carried as two BF16 terms, exactly.
#ifndef SPLITZIP_KV4_ATTENTION_H
#define SPLITZIP_KV4_ATTENTION_H

#include "kv4_common.h"

namespace kv4 {

constexpr int kAttThreads = 256;  // 4 waves

// Workgroups that the GPU holds at once (256 compute units): the kernel for few
// rows 3 a unit, by its registers; the one for many 2, by its LDS.
constexpr uint32_t kFewSlots = 768, kManySlots = 512;
// Pieces of the weights' sums: nothing to join, so shorter ones, fewer where the
// rows' operands take more registers.  480, 768, 1000, 1536 in all: 32.9, 29.8,
// 28.8, 29.0 us (32 sequences of 4 rows), 12.5, 12.1, 14.4, 15.7 (24 of 35 rows).
constexpr uint32_t kMassPieces = 1536, kMassPiecesRows = 768;
// Up to so many rows every wave converts the cache for itself, in row tiles of
// 32 (the second tile's reads are L2's): no barriers and more bytes under way.
// 64 rows of 128 channels, 16 x 8192 slots: 74 us against 82 through LDS; 128
// rows: 165 against 132.
constexpr uint32_t kFewRows = 64;
// Up to this length a workgroup takes a head's slots whole: a second launch to
// join pieces costs the host more than they save the GPU (1000 slots: equal).
constexpr uint32_t kWholeLen = 1024;

struct AttArgs {
  Batch a;
  const uint8_t* q;
  uint64_t q_row, q_head;  // strides in elements
  uint8_t* out;
  float* lse;
  const float* mass;
  float* mass_out;
  float* part_o;    // [piece][head][rows_max][D] unnormalised sums
  float* part_ml;   // [piece][head][rows_max][2] largest logit (base 2), sum
  float* row_lse;   // [seq][head][rows_max] log2 of the sums, for the weights
  float* mass_part; // [part][seq][head][max_len] weights of a part of the rows
  uint32_t mass_parts;
  uint32_t q_heads, group;
  uint32_t rows_max;  // rows (token, head of the group) of the longest sequence
  uint32_t pieces;    // wanted in all (Piece); 0: sequences stay whole
  float scale2;       // scale * log2 e
};

// The long axis is cut into pieces of one length for all sequences, chosen on
// the device from the lengths themselves: max_len is only a bound, and with
// pieces cut from it a ragged batch would leave most workgroups idle.  At least
// one piece a sequence, a multiple of 128 slots each, at most pieces + n_seqs
// in all.
struct Piece {
  uint32_t seq, index, count;  // of its sequence
  uint32_t first;              // the sequence's first piece
  uint32_t len;                // slots of a piece
  Seq s;
};

// The piece x (want_seq false), or the pieces of sequence x; every wave finds
// it for itself.  seq = n_seqs: there is no such piece.
__device__ inline Piece piece_of(const Batch& a, uint32_t pieces, uint32_t x, bool want_seq) {
  const uint32_t lane = threadIdx.x & 63;
  // what a batch of up to 64 sequences is described by, in one round of loads
  auto at = [&](uint32_t b, int32_t& len, int32_t& row0, int32_t& end) {
    const bool in = b < a.n_seqs;
    len = in ? a.lens[b] : 0;
    row0 = a.cu ? (in ? a.cu[b] : 0) : (int32_t)b;
    end = a.cu ? (in ? a.cu[b + 1] : 0) : (int32_t)b + 1;
  };
  auto checked = [&](int32_t n) { return n < 0 || n > (int32_t)a.max_len ? 0u : (uint32_t)n; };
  int32_t len0, row00, end0;
  at(lane, len0, row00, end0);
  Piece p;
  p.len = 1u << 30;
  if (pieces) {
    uint64_t total = 0;
    for (uint32_t b = 0; b < a.n_seqs; b += 64) {
      const uint32_t n = checked(b == 0 ? len0 : b + lane < a.n_seqs ? a.lens[b + lane] : 0);
      // 64 lengths of up to 2^30 each, summed in two halves
      total += wave_last(wave_scan(n & 0xFFFFu)) + ((uint64_t)wave_last(wave_scan(n >> 16)) << 16);
    }
    p.len = (uint32_t)min((total / pieces + 128) / 128 * 128, (uint64_t)1 << 30);
  }
  uint32_t before = 0;
  for (uint32_t b = 0; b < a.n_seqs; b += 64) {
    int32_t len = len0, row0 = row00, end = end0;
    if (b > 0) at(b + lane, len, row0, end);
    const uint32_t count = b + lane < a.n_seqs ? max(1u, (checked(len) + p.len - 1) / p.len) : 0u;
    const uint32_t upto = wave_scan(count);
    const uint64_t hit = __ballot(want_seq ? b + lane == x : before + upto > x);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      p.seq = b + l;
      p.count = (uint32_t)__builtin_amdgcn_readlane((int)count, l);
      p.first = before + (uint32_t)__builtin_amdgcn_readlane((int)upto, l) - p.count;
      p.index = want_seq ? 0 : x - p.first;
      p.s = seq_from(a, __builtin_amdgcn_readlane(len, l), __builtin_amdgcn_readlane(row0, l),
                     __builtin_amdgcn_readlane(end, l));
      return p;
    }
    before += wave_last(upto);
  }
  p.seq = a.n_seqs;
  p.index = p.count = p.first = 0;
  p.s = Seq{0, 0, 0, false};
  return p;
}

// Channels of product step m for lane quarter j: an 8-channel run.
template <int D>
__device__ inline uint32_t chan_of(uint32_t m, uint32_t j) {
  constexpr uint32_t W = D / 4 < 32 ? D / 4 : 32;
  return m * 8 / W * (4 * W) + j * W + m * 8 % W;
}

__device__ inline float max_quarters(float v) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

__device__ inline float sum_quarters(float v) {
  auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

__device__ inline uint32_t pack_bf16(float a, float b) {  // round to nearest even
  bf16x2 p;
  p[0] = (__bf16)a;
  p[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, p);
}

__device__ inline float bf16_lo(uint32_t p) { return __uint_as_float(p << 16); }
__device__ inline float bf16_hi(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

__device__ inline f32x4 mma(const u32x4 a, const u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Query rows as an operand: row r = token * group + head in the group, step m.
// Rows beyond `rows` are zero.  lo: what BF16 leaves of FP16 values.
template <int D, bool kHalf>
__device__ inline void load_q_step(const AttArgs& g, const Seq& s, uint32_t head, uint32_t r, uint32_t rows, uint32_t j,
                                   uint32_t m, u32x4& hi, u32x4& lo) {
  const uint32_t tok = r / g.group, hg = r % g.group;
  const uint8_t* p = g.q + 2 * (((uint64_t)s.row0 + tok) * g.q_row + (uint64_t)(head * g.group + hg) * g.q_head);
  u32x4 x = {0, 0, 0, 0};
  if (r < rows) x = *reinterpret_cast<const u32x4*>(p + 2 * chan_of<D>(m, j));
  if constexpr (kHalf) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = (float)__builtin_bit_cast(_Float16, (uint16_t)x[e]);
      const float b = (float)__builtin_bit_cast(_Float16, (uint16_t)(x[e] >> 16));
      hi[e] = pack_bf16(a, b);
      lo[e] = pack_bf16(a - bf16_lo(hi[e]), b - bf16_hi(hi[e]));
    }
  } else {
    hi = x;
  }
}

template <int D, bool kHalf>
__device__ inline void load_q(const AttArgs& g, const Seq& s, uint32_t head, uint32_t r, uint32_t rows, uint32_t j,
                              u32x4 hi[D / 32], u32x4 lo[D / 32]) {
#pragma unroll
  for (int m = 0; m < D / 32; ++m) load_q_step<D, kHalf>(g, s, head, r, rows, j, m, hi[m], lo[m]);
}

// One lane's share of 16 keys: K codes of its key and quarter, V codes of 4
// tokens and D/16 channels, and their scales.
template <int D>
struct Raw {
  uint32_t k[D / 32], v[D / 32];
  uint32_t ks, vs;
};

// A lane's offsets in the bytes of 16 slots: the same for all, so a load is a
// scalar base and a constant register.
template <int D>
struct LaneAt {
  using L = Layout<D>;
  uint32_t k, v, ks, vs;
  __device__ LaneAt(uint32_t i, uint32_t j)
      : k(i * L::kCode + j * (D == 64 ? 8 : 16)),
        v(L::v_piece(4 * j, i)),
        ks(i * L::kScale + (D == 64 ? j >> 1 : j)),
        vs(L::v_scale(4 * j, i * L::kScale / 16)) {}
};

template <bool kOnce, class T>
__device__ inline T get(const uint8_t* p) {
  if constexpr (kOnce) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  return *reinterpret_cast<const T*>(p);
}

// Lane (i, j)'s bytes of the 16 slots at `t` (in a page, uniform) of `base`.
// kOnce: no other workgroup reads these codes (non-temporal: 96 -> 87 us on
// 374 MB of scattered pages); the scales share their lines with other slots'.
// kOnceK: nor K's.
template <int D, bool kOnce, bool kV = true, bool kOnceK = kOnce>
__device__ inline void load_raw(const uint8_t* base, uint32_t shift, uint32_t t, const LaneAt<D>& at, Raw<D>& r) {
  using L = Layout<D>;
  const uint8_t* k = base + t * L::kCode;
  const uint8_t* v = k + L::v_codes(shift);
  const uint8_t* ks = base + L::k_scales(shift) + t * L::kScale;
  const uint8_t* vs = base + L::v_scales(shift) + t * L::kScale;
  if constexpr (D == 64) {
    *reinterpret_cast<u32x2*>(r.k) = get<kOnceK, u32x2>(k + at.k);
    r.ks = ks[at.ks];
    if constexpr (kV) *reinterpret_cast<u32x2*>(r.v) = get<kOnce, u32x2>(v + at.v);
  } else if constexpr (D == 128) {
    *reinterpret_cast<u32x4*>(r.k) = get<kOnceK, u32x4>(k + at.k);
    r.ks = ks[at.ks];
    if constexpr (kV) *reinterpret_cast<u32x4*>(r.v) = get<kOnce, u32x4>(v + at.v);
  } else {
    *reinterpret_cast<u32x4*>(r.k) = get<kOnceK, u32x4>(k + at.k);
    *reinterpret_cast<u32x4*>(r.k + 4) = get<kOnceK, u32x4>(k + at.k + 64);
    r.ks = ks[at.ks] | (uint32_t)ks[at.ks + 4] << 8;
    if constexpr (kV) {
      *reinterpret_cast<u32x4*>(r.v) = get<kOnce, u32x4>(v + at.v);
      *reinterpret_cast<u32x4*>(r.v + 4) = get<kOnce, u32x4>(v + at.v + 16);
    }
  }
  if constexpr (kV) r.vs = *reinterpret_cast<const uint32_t*>(vs + at.vs);
}

// Step m's left operand of S^T.
template <int D>
__device__ inline u32x4 k_operand(const Raw<D>& r, int m) {
  const float s = scale_of(D == 256 ? (m < 4 ? r.ks & 0xFFu : r.ks >> 8) : r.ks);
  u32x4 o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.k[m], s, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.k[m], s, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.k[m], s, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.k[m], s, 3));
  return o;
}

// Byte `kB` of codes (2 channels of one token) under scale s.
template <int kB>
__device__ inline uint32_t v_pair(uint32_t codes, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, kB));
}

template <int D, int kTok, int kPair>
__device__ inline uint32_t v_at(const Raw<D>& r, float s) {  // channels 2 kPair, 2 kPair + 1 of token kTok
  constexpr int at = kTok * (D / 32) + kPair;
  return v_pair<at % 4>(r.v[at / 4], s);
}

// Left operands of O^T for the lane's channels 2 kPair and 2 kPair + 1 (x, y)
// from 4 tokens of each of two tiles.
template <int D, int kPair>
__device__ inline void v_operands(const Raw<D>& a, const float sa[4], const Raw<D>& b, const float sb[4], u32x4& x,
                                  u32x4& y) {
  const uint32_t a0 = v_at<D, 0, kPair>(a, sa[0]), a1 = v_at<D, 1, kPair>(a, sa[1]);
  const uint32_t a2 = v_at<D, 2, kPair>(a, sa[2]), a3 = v_at<D, 3, kPair>(a, sa[3]);
  const uint32_t b0 = v_at<D, 0, kPair>(b, sb[0]), b1 = v_at<D, 1, kPair>(b, sb[1]);
  const uint32_t b2 = v_at<D, 2, kPair>(b, sb[2]), b3 = v_at<D, 3, kPair>(b, sb[3]);
  x[0] = __builtin_amdgcn_perm(a1, a0, 0x05040100);
  x[1] = __builtin_amdgcn_perm(a3, a2, 0x05040100);
  x[2] = __builtin_amdgcn_perm(b1, b0, 0x05040100);
  x[3] = __builtin_amdgcn_perm(b3, b2, 0x05040100);
  y[0] = __builtin_amdgcn_perm(a1, a0, 0x07060302);
  y[1] = __builtin_amdgcn_perm(a3, a2, 0x07060302);
  y[2] = __builtin_amdgcn_perm(b1, b0, 0x07060302);
  y[3] = __builtin_amdgcn_perm(b3, b2, 0x07060302);
}

__device__ inline void v_scales4(uint32_t vs, float s[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) s[t] = scale_of((vs >> (8 * t)) & 0xFFu);
}

// Clears the tokens t0 + 0..3 at or beyond `end`: a slot that no row may see
// can hold anything, and 0 times a NaN is a NaN.
template <int D>
__device__ inline void clear_v(Raw<D>& r, uint32_t t0, uint32_t end) {
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {
    if constexpr (D == 64) {
      if (t0 + 2 * w >= end) r.v[w] &= 0xFFFF0000u;
      if (t0 + 2 * w + 1 >= end) r.v[w] &= 0xFFFFu;
    } else {
      if (t0 + w * 4 / (D / 32) >= end) r.v[w] = 0;
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
    if (t0 + t >= end) r.vs = (r.vs & ~(0xFFu << (8 * t))) | 127u << (8 * t);
}

template <int D, int kPair, int kRows>
__device__ inline void pv_step(const Raw<D>& a, const float sa[4], const Raw<D>& b, const float sb[4],
                               const u32x4 (&p)[kRows], const u32x4 (&pl)[kRows], f32x4 (&o)[kRows][D / 16]) {
  if constexpr (kPair < D / 32) {
    u32x4 x, y;
    v_operands<D, kPair>(a, sa, b, sb, x, y);
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      o[n][2 * kPair] = mma(x, p[n], o[n][2 * kPair]);
      o[n][2 * kPair + 1] = mma(y, p[n], o[n][2 * kPair + 1]);
      o[n][2 * kPair] = mma(x, pl[n], o[n][2 * kPair]);
      o[n][2 * kPair + 1] = mma(y, pl[n], o[n][2 * kPair + 1]);
    }
    pv_step<D, kPair + 1, kRows>(a, sa, b, sb, p, pl, o);
  }
}

// One lane's 4 tokens of V as halves of operands: channel c at to[c][.][lane][.].
template <int D, int kPair>
__device__ inline void v_to_lds(const Raw<D>& r, const float s[4], u32x2* to) {
  if constexpr (kPair < D / 32) {
    const uint32_t a0 = v_at<D, 0, kPair>(r, s[0]), a1 = v_at<D, 1, kPair>(r, s[1]);
    const uint32_t a2 = v_at<D, 2, kPair>(r, s[2]), a3 = v_at<D, 3, kPair>(r, s[3]);
    to[(2 * kPair) * 128] = u32x2{__builtin_amdgcn_perm(a1, a0, 0x05040100), __builtin_amdgcn_perm(a3, a2, 0x05040100)};
    to[(2 * kPair + 1) * 128] =
        u32x2{__builtin_amdgcn_perm(a1, a0, 0x07060302), __builtin_amdgcn_perm(a3, a2, 0x07060302)};
    v_to_lds<D, kPair + 1>(r, s, to);
  }
}

__device__ inline void store2(uint8_t* out, uint64_t elem, bool half, float a, float b) {
  uint32_t w;
  if (half)
    w = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) | (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
  else
    w = pack_bf16(a, b);
  *reinterpret_cast<uint32_t*>(out + 2 * elem) = w;
}

// One workgroup: the slots of one piece, 16 kRows query rows of one KV head of
// one sequence.  Each wave takes every 4th tile of 32 slots with a softmax of
// its own; the four are joined through LDS.
// kAgain: the weights' kernel reads K again, so the caches are to keep it (32 x
// 8192 slots: 79 -> 77 us, 8 x 32768: 64 -> 62).
template <int D, int kRows, bool kHalf, bool kAgain>
__global__ __launch_bounds__(kAttThreads, D == 256 ? 1 : kRows == 1 || D == 64 ? 3 : 2) void kv4_attend_kernel(AttArgs g) {
  constexpr int kSteps = D / 32;
  __shared__ float sh_o[4][16][D + 4];
  __shared__ float sh_m[4][16 * kRows], sh_l[4][16 * kRows];
  const Batch& a = g.a;
  const uint32_t head = blockIdx.y, tile = blockIdx.z;
  const uint32_t tid = threadIdx.x, lane = tid & 63, i = lane & 15, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Piece pc = piece_of(a, g.pieces, blockIdx.x, false);
  const uint32_t b = pc.seq;
  if (b >= a.n_seqs) return;
  const Seq s = pc.s;
  if (!s.ok && tid == 0) corrupt(a.status);
  const uint32_t rows = (uint32_t)s.rows * g.group, r0 = tile * 16 * kRows;
  if (r0 >= rows) return;
  // what each row sees: row r's last slot is len - rows + token
  const int32_t before = s.len - s.rows;
  const int32_t newest = before + (int32_t)(min(r0 + 16 * kRows, rows) - 1) / (int32_t)g.group;
  const uint32_t seen = newest < 0 ? 0u : (uint32_t)newest + 1;  // slots that any row of this tile sees
  const uint32_t c0 = pc.index * pc.len, c1 = min(seen, c0 + pc.len);
  if (c0 >= c1 && c0 > 0) return;  // the first piece writes what rows without slots get

  u32x4 qh[kRows][kSteps], ql[kRows][kSteps];
  int32_t lim[kRows];
  f32x4 o[kRows][D / 16];
  float m[kRows], l[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const uint32_t r = r0 + 16 * n + i;
    load_q<D, kHalf>(g, s, head, r, rows, j, qh[n], ql[n]);
    lim[n] = before + (int32_t)(r / g.group) + 1;
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[n][t] = f32x4{0, 0, 0, 0};
  }
  // This wave's tiles: 32 slots at first + 128 it.  Lane 2 it + h holds the
  // page of tile it's half h, for 32 tiles at a time, so that a tile's address
  // never waits for the block table.
  const uint32_t in_page = (1u << a.page_shift) - 1;
  const uint32_t first = c0 + 32 * wave, n_tiles = first < c1 ? (c1 - first + 127) / 128 : 0;
  // a half tile wholly behind the end loads the last slots there are instead, unused
  auto slot_of = [&](uint32_t it, uint32_t h) { return min(first + 128 * it + 16 * h, (c1 - 1) & ~15u); };
  const LaneAt<D> lane_at(i, j);
  uint32_t pages = 0;
  auto load_pages = [&](uint32_t it) {
    if (n_tiles > 0) pages = page_of(a, b, slot_of(min(it + (lane >> 1), n_tiles - 1), lane & 1) >> a.page_shift);
  };
  auto load_tile = [&](uint32_t it, Raw<D> (&r)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t p = (uint32_t)__builtin_amdgcn_readlane((int)pages, (int)(2 * (it & 31) + h)) & ~kBadPage;
      const uint8_t* base = a.pages + ((uint64_t)p * a.n_heads + head) * a.page_bytes;
      load_raw<D, kRows == 1, true, kRows == 1 && !kAgain>(base, a.page_shift, __builtin_amdgcn_readfirstlane(slot_of(it, h)) & in_page, lane_at, r[h]);
    }
  };
  auto compute = [&](uint32_t it, Raw<D> (&cur)[2]) {
    const uint32_t at = first + 128 * it;
    f32x4 x[kRows][2];
#pragma unroll
    for (int n = 0; n < kRows; ++n) x[n][0] = x[n][1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 k = k_operand<D>(cur[h], st);
#pragma unroll
        for (int n = 0; n < kRows; ++n) {
          x[n][h] = mma(k, qh[n][st], x[n][h]);
          if constexpr (kHalf) x[n][h] = mma(k, ql[n][st], x[n][h]);
        }
      }
    if ((int32_t)(at + 32) > before) {  // some row does not see all of the tile
#pragma unroll
      for (int n = 0; n < kRows; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((int32_t)(at + 16 * h + 4 * j + e) >= lim[n]) x[n][h][e] = -INFINITY;
    }
    if (at + 32 > c1) {
#pragma unroll
      for (int h = 0; h < 2; ++h) clear_v<D>(cur[h], at + 16 * h + 4 * j, c1);
    }
    u32x4 p[kRows], pl[kRows];
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      float top = m[n];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, x[n][h][e]);
      top = max_quarters(top);
      if (__any(top > m[n])) {  // the running maximum grew for some row: rescale
        const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[n] - top) * g.scale2);
        m[n] = top;
        l[n] *= f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) o[n][t] *= f;
      }
      const float shift = m[n] == -INFINITY ? 0.0f : m[n] * g.scale2;
      float w[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[4 * h + e] = __builtin_amdgcn_exp2f(fmaf(x[n][h][e], g.scale2, -shift));
          l[n] += w[4 * h + e];
        }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[n][e] = pack_bf16(w[2 * e], w[2 * e + 1]);
        // what BF16 leaves of the weights: 16 bits in all
        pl[n][e] = pack_bf16(w[2 * e] - bf16_lo(p[n][e]), w[2 * e + 1] - bf16_hi(p[n][e]));
      }
    }
    float sa[4], sb[4];
    v_scales4(cur[0].vs, sa);
    v_scales4(cur[1].vs, sb);
    pv_step<D, 0, kRows>(cur[0], sa, cur[1], sb, p, pl, o);
  };
  // Loads run a tile ahead of the products, in two sets of registers.  They
  // are issued whether or not there is a next tile: behind a branch the wait
  // for this tile's bytes would be one for the next tile's as well.
  Raw<D> even[2], odd[2];
  load_pages(0);
  auto step = [&](uint32_t it, Raw<D> (&cur)[2], Raw<D> (&nxt)[2]) {
    const uint32_t ahead = min(it + 1, n_tiles - 1);
    if (((it + 1) & 31) == 0) load_pages(ahead);
    load_tile(ahead, nxt);
    compute(it, cur);
  };
  if (n_tiles > 0) {
    load_tile(0, even);
    uint32_t it = 0;
    for (; it + 2 <= n_tiles; it += 2) {
      step(it, even, odd);
      step(it + 1, odd, even);
    }
    if (it < n_tiles) compute(it, even);
  }

  // join the four waves
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    l[n] = sum_quarters(l[n]);
    if (j == 0) {
      sh_m[wave][16 * n + i] = m[n];
      sh_l[wave][16 * n + i] = l[n];
    }
  }
  __syncthreads();
  const uint32_t row_base = (b * a.n_heads + head) * g.rows_max;  // fits: checked on the host
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    float top = sh_m[0][16 * n + i];
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, sh_m[w][16 * n + i]);
    const float f = m[n] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m[n] - top) * g.scale2);
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sh_o[wave][i][(4 * j + e) * (D / 16) + t] = o[n][t][e] * f;
    __syncthreads();
    const uint32_t row = tid >> 4, r = r0 + 16 * n + row;
    if (r < rows) {
      float mm[4], all = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) all = fmaxf(all, mm[w] = sh_m[w][16 * n + row]);
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (mm[w] != -INFINITY) sum += sh_l[w][16 * n + row] * __builtin_amdgcn_exp2f((mm[w] - all) * g.scale2);
      const uint32_t tok = r / g.group, qh_at = head * g.group + r % g.group;
      const uint64_t out_row = ((uint64_t)s.row0 + tok) * g.q_heads + qh_at;
      const uint64_t part = ((uint64_t)blockIdx.x * a.n_heads + head) * g.rows_max + r;
      const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
      for (uint32_t c = 2 * (tid & 15); c < (uint32_t)D; c += 32) {
        float u = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          u += sh_o[w][row][c];
          v += sh_o[w][row][c + 1];
        }
        if (pc.count == 1) {
          store2(g.out, out_row * D + c, kHalf, u * inv, v * inv);
        } else {
          g.part_o[part * D + c] = u;
          g.part_o[part * D + c + 1] = v;
        }
      }
      if ((tid & 15) == 0) {
        const float top2 = all * g.scale2;
        if (pc.count == 1) {
          const float lse2 = sum == 0.0f ? -INFINITY : top2 + __builtin_amdgcn_logf(sum);
          if (g.lse) g.lse[out_row] = lse2 * 0.69314718055994531f;
          if (g.row_lse) g.row_lse[row_base + r] = lse2;
        } else {
          g.part_ml[2 * part] = top2;
          g.part_ml[2 * part + 1] = sum;
        }
      }
    }
    __syncthreads();
  }
}

// Query rows of a wave of the kernel for many rows: those of 256 channels fill
// twice the registers.
template <int D>
constexpr int kWaveRows = D == 256 ? 16 : 32;

// Many rows: 128 query rows of one KV head, 32 a wave, over a piece's slots.
// The four waves convert 64 slots at a time into LDS, 16 slots each, in the
// order in which the matrix instructions take their operands (a lane's 16
// bytes side by side: no bank conflicts on either side), and share them: a
// conversion serves 128 rows.  Two buffers, one barrier a tile; the codes of
// the tile after the next are on their way meanwhile.  Heads run fastest over
// the grid, so that one head's row tiles meet in one XCD's L2 (8 heads), and
// the last rows, which see the most, come first.
template <int D, bool kHalf>
__global__ __launch_bounds__(kAttThreads, 2) void kv4_extend_kernel(AttArgs g) {
  constexpr int kSteps = D / 32, kChans = D / 16, kN = kWaveRows<D> / 16;
  // 16s of slots of a tile, its slots, its 32s.  256 channels: half a tile, so that two workgroups share a compute
  // unit (6000 slots' prompts: 895 -> 631 us); two waves then have the keys and two the values to convert
  constexpr int kKeys = D == 256 ? 2 : 4, kTile = 16 * kKeys, kPairs = kKeys / 2;
  __shared__ u32x4 sh_k[2][kKeys][kSteps][64];
  __shared__ u32x2 sh_v[2][kPairs][kChans][64][2];
  const Batch& a = g.a;
  const uint32_t head = blockIdx.x, tile = gridDim.y - 1 - blockIdx.y;
  const uint32_t tid = threadIdx.x, lane = tid & 63, i = lane & 15, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Piece pc = piece_of(a, g.pieces, blockIdx.z, false);
  const uint32_t b = pc.seq;
  if (b >= a.n_seqs) return;
  const Seq s = pc.s;
  if (!s.ok && tid == 0) corrupt(a.status);
  const uint32_t rows = (uint32_t)s.rows * g.group, r0 = tile * 4 * kWaveRows<D>;
  if (r0 >= rows) return;
  const int32_t before = s.len - s.rows;
  auto seen_by = [&](uint32_t r) -> uint32_t {  // slots that row r sees
    const int32_t n = before + (int32_t)(min(r, rows - 1) / g.group) + 1;
    return n < 0 ? 0u : (uint32_t)n;
  };
  const uint32_t seen = seen_by(r0 + 4 * kWaveRows<D> - 1);
  const uint32_t c0 = pc.index * pc.len, c1 = min(seen, c0 + pc.len);
  if (c0 >= c1 && c0 > 0) return;  // the first piece writes what rows without slots get
  const uint32_t w0 = r0 + kWaveRows<D> * wave;  // this wave's rows
  const uint32_t w_first = seen_by(w0), w_last = w0 < rows ? seen_by(w0 + kWaveRows<D> - 1) : 0;

  u32x4 qh[kN][kSteps], ql[kN][kSteps];
  int32_t lim[kN];
  f32x4 o[kN][kChans];
  float m[kN], l[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const uint32_t r = w0 + 16 * n + i;
    load_q<D, kHalf>(g, s, head, r, rows, j, qh[n], ql[n]);
    lim[n] = before + (int32_t)(r / g.group) + 1;
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int t = 0; t < kChans; ++t) o[n][t] = f32x4{0, 0, 0, 0};
  }
  // this wave's 16 slots of a tile; lane t holds the page of tile t, 64 tiles at a time
  const uint32_t in_page = (1u << a.page_shift) - 1, n_tiles = c1 > c0 ? (c1 - c0 + kTile - 1) / kTile : 0,
                 mine = wave % kKeys;
  const LaneAt<D> lane_at(i, j);
  auto slot_of = [&](uint32_t t) { return min(c0 + kTile * t + 16 * mine, (c1 - 1) & ~15u); };
  uint32_t pages = 0;
  auto load_pages = [&](uint32_t t) { pages = page_of(a, b, slot_of(min(t + lane, n_tiles - 1)) >> a.page_shift); };
  Raw<D> raw;
  auto load_tile = [&](uint32_t t) {
    const uint32_t p = (uint32_t)__builtin_amdgcn_readlane((int)pages, (int)(t & 63)) & ~kBadPage;
    load_raw<D, false>(a.pages + ((uint64_t)p * a.n_heads + head) * a.page_bytes, a.page_shift,
                       __builtin_amdgcn_readfirstlane(slot_of(t)) & in_page, lane_at, raw);
  };
  auto convert = [&](uint32_t t) {  // raw -> LDS
    const uint32_t at = c0 + kTile * t + 16 * mine, buf = t & 1;
    if (at + 16 > c1) clear_v<D>(raw, at + 4 * j, c1);
    if (kKeys == 4 || wave < 2) {
#pragma unroll
      for (int st = 0; st < kSteps; ++st) sh_k[buf][mine][st][lane] = k_operand<D>(raw, st);
    }
    if (kKeys == 4 || wave >= 2) {
      float sv[4];
      v_scales4(raw.vs, sv);
      v_to_lds<D, 0>(raw, sv, &sh_v[buf][mine >> 1][0][lane][mine & 1]);
    }
  };
  if (n_tiles > 0) {
    load_pages(0);
    load_tile(0);
    convert(0);
    load_tile(min(1u, n_tiles - 1));
  }
  for (uint32_t t = 0; t < n_tiles; ++t) {
    __syncthreads();
    const uint32_t at = c0 + kTile * t, buf = t & 1;
    if (at < w_last) {
      f32x4 x[kN][kKeys];
#pragma unroll
      for (int kt = 0; kt < kKeys; ++kt)
#pragma unroll
        for (int n = 0; n < kN; ++n) x[n][kt] = f32x4{0, 0, 0, 0};
      // steps outside: 8 sums in turn, so that none waits for its own last product
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
#pragma unroll
        for (int kt = 0; kt < kKeys; ++kt) {
          const u32x4 k = sh_k[buf][kt][st][lane];
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            x[n][kt] = mma(k, qh[n][st], x[n][kt]);
            if constexpr (kHalf) x[n][kt] = mma(k, ql[n][st], x[n][kt]);
          }
        }
      if (at + kTile > w_first) {  // some row does not see all of the tile
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int kt = 0; kt < kKeys; ++kt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((int32_t)(at + 16 * kt + 4 * j + e) >= lim[n]) x[n][kt][e] = -INFINITY;
      }
      u32x4 p[kN][kPairs], pl[kN][kPairs];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        float top = m[n];
#pragma unroll
        for (int kt = 0; kt < kKeys; ++kt)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, x[n][kt][e]);
        top = max_quarters(top);
        if (__any(top > m[n])) {
          const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[n] - top) * g.scale2);
          m[n] = top;
          l[n] *= f;
#pragma unroll
          for (int c = 0; c < kChans; ++c) o[n][c] *= f;
        }
        const float shift = m[n] == -INFINITY ? 0.0f : m[n] * g.scale2;
#pragma unroll
        for (int kt = 0; kt < kKeys; ++kt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float w0_ = __builtin_amdgcn_exp2f(fmaf(x[n][kt][2 * h], g.scale2, -shift));
            const float w1_ = __builtin_amdgcn_exp2f(fmaf(x[n][kt][2 * h + 1], g.scale2, -shift));
            l[n] += w0_ + w1_;
            const uint32_t hi = pack_bf16(w0_, w1_);
            p[n][kt >> 1][2 * (kt & 1) + h] = hi;
            // FP16 results need more of the weights than BF16 holds
            if constexpr (kHalf) pl[n][kt >> 1][2 * (kt & 1) + h] = pack_bf16(w0_ - bf16_lo(hi), w1_ - bf16_hi(hi));
          }
      }
#pragma unroll
      for (int h = 0; h < kPairs; ++h)
#pragma unroll
        for (int c = 0; c < kChans; ++c) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(&sh_v[buf][h][c][lane][0]);
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            o[n][c] = mma(v, p[n][h], o[n][c]);
            if constexpr (kHalf) o[n][c] = mma(v, pl[n][h], o[n][c]);
          }
        }
    }
    if (t + 1 < n_tiles) {
      convert(t + 1);
      const uint32_t ahead = min(t + 2, n_tiles - 1);
      if (((t + 2) & 63) == 0) load_pages(ahead);
      load_tile(ahead);
    }
  }
  // lane (i, j) holds channels (4j + e) D/16 .. of row i
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    l[n] = sum_quarters(l[n]);
    const uint32_t r = w0 + 16 * n + i;
    if (r >= rows) continue;
    const uint64_t out_row = ((uint64_t)s.row0 + r / g.group) * g.q_heads + head * g.group + r % g.group;
    const uint64_t part = ((uint64_t)blockIdx.z * a.n_heads + head) * g.rows_max + r;
    const float sum = l[n], inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t c = (4 * j + e) * kChans;
      if (pc.count == 1) {
#pragma unroll
        for (int t = 0; t < kChans; t += 2)
          store2(g.out, out_row * D + c + t, kHalf, o[n][t][e] * inv, o[n][t + 1][e] * inv);
      } else {
#pragma unroll
        for (int t = 0; t < kChans; t += 4)
          *reinterpret_cast<f32x4*>(g.part_o + part * D + c + t) =
              f32x4{o[n][t][e], o[n][t + 1][e], o[n][t + 2][e], o[n][t + 3][e]};
      }
    }
    if (j == 0) {
      const float top2 = m[n] * g.scale2;
      if (pc.count == 1) {
        const float lse2 = sum == 0.0f ? -INFINITY : top2 + __builtin_amdgcn_logf(sum);
        if (g.lse) g.lse[out_row] = lse2 * 0.69314718055994531f;
        if (g.row_lse) g.row_lse[(b * a.n_heads + head) * g.rows_max + r] = lse2;
      } else {
        g.part_ml[2 * part] = top2;
        g.part_ml[2 * part + 1] = sum;
      }
    }
  }
}

// Joins the pieces: D / 4 lanes hold a row's channels.  kSpread (few rows): the
// workgroup's lane groups share one row's pieces and are joined through LDS;
// else every group has a row of its own.
template <int D, bool kHalf, bool kSpread>
__global__ __launch_bounds__(256) void kv4_join_kernel(AttArgs g) {
  constexpr uint32_t kLanes = D / 4, kGroups = 256 / kLanes, kAhead = 4;
  __shared__ f32x4 sh_o[kSpread ? kGroups : 1][kLanes];
  __shared__ float sh_m[kGroups], sh_l[kGroups];
  const Batch& a = g.a;
  const uint32_t head = blockIdx.y;
  const uint32_t lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const Piece pc = piece_of(a, g.pieces, blockIdx.z, true);
  if (pc.count == 1) return;  // written by the attention itself
  const Seq s = pc.s;
  const uint32_t r = kSpread ? blockIdx.x : blockIdx.x * kGroups + group, rows = (uint32_t)s.rows * g.group;
  if (kSpread ? r >= rows : blockIdx.x * kGroups >= rows) return;
  const int32_t newest = s.len - s.rows + (int32_t)(r / g.group);
  const uint32_t seen = newest < 0 ? 0u : (uint32_t)newest + 1;
  // pieces with slots of this row
  const uint32_t n = r < rows ? max(1u, (seen + pc.len - 1) / pc.len) : 0;
  const uint32_t begin = kSpread ? group : 0, step = kSpread ? kGroups : 1;
  const uint64_t first = ((uint64_t)pc.first * a.n_heads + head) * g.rows_max + r, next = (uint64_t)a.n_heads * g.rows_max;
  float top = -INFINITY, sum = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (uint32_t k = begin; k < n; k += kAhead * step) {
    float mk[kAhead], lk[kAhead];
    f32x4 ok[kAhead];
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) {  // the loads of a round are under way together
      const uint64_t at = first + (uint64_t)min(k + u * step, n - 1) * next;
      mk[u] = k + u * step < n ? g.part_ml[2 * at] : -INFINITY;
      lk[u] = g.part_ml[2 * at + 1];
      ok[u] = *reinterpret_cast<const f32x4*>(g.part_o + at * D + 4 * lane);
    }
    float now = top;
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) now = fmaxf(now, mk[u]);
    if (now == -INFINITY) continue;
    const float f = __builtin_amdgcn_exp2f(top - now);
    top = now;
    sum *= f;
    o *= f;
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) {
      const float fk = __builtin_amdgcn_exp2f(mk[u] - now);  // 0 for a piece without slots of the row
      sum += lk[u] * fk;
      o += ok[u] * fk;
    }
  }
  if constexpr (kSpread) {
    sh_o[group][lane] = o;
    if (lane == 0) {
      sh_m[group] = top;
      sh_l[group] = sum;
    }
    __syncthreads();
    if (group != 0) return;
    for (uint32_t k = 1; k < kGroups; ++k) top = fmaxf(top, sh_m[k]);
    sum = 0.0f;
    o = f32x4{0, 0, 0, 0};
    for (uint32_t k = 0; k < kGroups; ++k) {
      if (sh_m[k] == -INFINITY) continue;
      const float f = __builtin_amdgcn_exp2f(sh_m[k] - top);
      sum += sh_l[k] * f;
      o += sh_o[k][lane] * f;
    }
  }
  if (r >= rows) return;
  const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
  const uint64_t out_row = ((uint64_t)s.row0 + r / g.group) * g.q_heads + head * g.group + r % g.group;
  store2(g.out, out_row * D + 4 * lane, kHalf, o[0] * inv, o[1] * inv);
  store2(g.out, out_row * D + 4 * lane + 2, kHalf, o[2] * inv, o[3] * inv);
  if (lane == 0) {
    const float lse2 = sum == 0.0f ? -INFINITY : top + __builtin_amdgcn_logf(sum);
    if (g.lse) g.lse[out_row] = lse2 * 0.69314718055994531f;
    if (g.row_lse) g.row_lse[(pc.seq * a.n_heads + head) * g.rows_max + r] = lse2;
  }
}

// The weights that the slots drew: the logits again (K is half of the cache,
// and keeping them would cost 4 bytes for each of its rows), p = 2^(x - lse) and
// its sum over the rows in a fixed order.  Here the products are S = Q K^T, so
// that a lane has one key and four rows: two exchanges sum a key's column.
//
// Few rows: Q stays in registers, a wave takes 64 slots at a time.
template <int D, int kRows, bool kHalf>
__global__ __launch_bounds__(kAttThreads, 2) void kv4_mass_kernel(AttArgs g) {
  constexpr int kSteps = D / 32;
  const Batch& a = g.a;
  const uint32_t head = blockIdx.y;
  const uint32_t tid = threadIdx.x, lane = tid & 63, i = lane & 15, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Piece pc = piece_of(a, g.pieces, blockIdx.x, false);
  const uint32_t b = pc.seq;
  if (b >= a.n_seqs) return;
  const Seq s = pc.s;
  if (!s.ok) return;
  const uint32_t c0 = pc.index * pc.len, c1 = min((uint32_t)s.len, c0 + pc.len);
  const uint32_t first = c0 + 64 * wave;
  if (first >= c1) return;
  const uint32_t n_tiles = (c1 - first + 255) / 256;
  const uint32_t rows = (uint32_t)s.rows * g.group;
  const int32_t before = s.len - s.rows;
  u32x4 qh[kRows][kSteps], ql[kRows][kSteps];
  float lse2[kRows][4];
  int32_t lim[kRows][4];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    load_q<D, kHalf>(g, s, head, 16 * n + i, rows, j, qh[n], ql[n]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t r = 16 * n + 4 * j + e;
      lse2[n][e] = r < rows ? g.row_lse[(b * a.n_heads + head) * g.rows_max + r] : INFINITY;
      lim[n][e] = r < rows ? before + (int32_t)(r / g.group) + 1 : 0;
    }
  }
  const uint32_t in_page = (1u << a.page_shift) - 1;
  const LaneAt<D> lane_at(i, j);
  // lane 4 t + h holds the page of tile t's quarter h, for 16 tiles at a time
  auto slot_of = [&](uint32_t t, uint32_t h) { return min(first + 256 * t + 16 * h, (c1 - 1) & ~15u); };
  uint32_t pages = 0;
  auto load_pages = [&](uint32_t t) { pages = page_of(a, b, slot_of(min(t + (lane >> 2), n_tiles - 1), lane & 3) >> a.page_shift); };
  auto page_at = [&](uint32_t t, uint32_t h) { return (uint32_t)__builtin_amdgcn_readlane((int)pages, (int)(4 * (t & 15) + h)); };
  auto load_tile = [&](uint32_t t, Raw<D> (&r)[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      load_raw<D, true, false>(a.pages + ((uint64_t)(page_at(t, h) & ~kBadPage) * a.n_heads + head) * a.page_bytes, a.page_shift,
                               __builtin_amdgcn_readfirstlane(slot_of(t, h)) & in_page, lane_at, r[h]);
  };
  // this lane's slot of a tile, as an index of the mass arrays; none where there is nothing to write
  constexpr uint64_t kNone = ~0ull;
  auto own_at = [&](uint32_t t) -> uint64_t {
    const uint32_t p = j == 0 ? page_at(t, 0) : j == 1 ? page_at(t, 1) : j == 2 ? page_at(t, 2) : page_at(t, 3);
    const uint32_t slot = first + 256 * t + lane;
    if (slot >= c1 || (p & kBadPage)) return kNone;
    return (((uint64_t)p * a.n_heads + head) << a.page_shift) + (slot & in_page);
  };
  auto compute = [&](uint32_t t, Raw<D> (&r)[4], uint64_t to, float old) {
    const uint32_t at = first + 256 * t;
    float own = 0.0f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      f32x4 x[kRows];
#pragma unroll
      for (int n = 0; n < kRows; ++n) x[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 k = k_operand<D>(r[h], st);
#pragma unroll
        for (int n = 0; n < kRows; ++n) {
          x[n] = mma(qh[n][st], k, x[n]);
          if constexpr (kHalf) x[n] = mma(ql[n][st], k, x[n]);
        }
      }
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < kRows; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = __builtin_amdgcn_exp2f(fmaf(x[n][e], g.scale2, -lse2[n][e]));
          sum += (int32_t)(at + 16 * h + i) < lim[n][e] ? w : 0.0f;
        }
      sum = sum_quarters(sum);
      own = (uint32_t)h == j ? sum : own;
    }
    if (to != kNone) g.mass_out[to] = old + own;
  };
  Raw<D> even[4], odd[4];
  auto step = [&](uint32_t t, Raw<D> (&cur)[4], Raw<D> (&nxt)[4]) {
    const uint64_t to = own_at(t);
    const float old = to != kNone ? g.mass[to] : 0.0f;
    const uint32_t ahead = min(t + 1, n_tiles - 1);
    if (((t + 1) & 15) == 0) load_pages(ahead);
    load_tile(ahead, nxt);
    compute(t, cur, to, old);
  };
  load_pages(0);
  load_tile(0, even);
  for (uint32_t t = 0; t < n_tiles; t += 2) {
    step(t, even, odd);
    if (t + 1 < n_tiles) step(t + 1, odd, even);
  }
}

// Many rows: 64 slots a wave stay in registers as operands, the query rows come
// through LDS, 32 at a time for the four waves' 256 slots.  Where slots alone make too few workgroups the rows are shared too, and
// kv4_mass_sum_kernel adds their parts.
template <int D, bool kHalf>
__global__ __launch_bounds__(kAttThreads, D == 256 ? 1 : 2) void kv4_mass_rows_kernel(AttArgs g) {
  constexpr int kSteps = D / 32, kTerms = kHalf ? 2 : 1, kMine = 2 * kSteps / 4;  // operands that a wave stages
  __shared__ u32x4 sh_q[2][kTerms][2 * kSteps][64];
  __shared__ float sh_lse[2][32];
  const Batch& a = g.a;
  const uint32_t head = blockIdx.x, b = blockIdx.z % a.n_seqs, part = blockIdx.z / a.n_seqs;
  const uint32_t tid = threadIdx.x, lane = tid & 63, i = lane & 15, j = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Seq s = seq_of(a, b);
  if (!s.ok) return;
  const uint32_t w_at = blockIdx.y * 256, at = w_at + 64 * wave, len = (uint32_t)s.len;
  if (w_at >= len) return;
  const uint32_t all_rows = (uint32_t)s.rows * g.group;
  const int32_t before = s.len - s.rows;
  const uint32_t in_page = (1u << a.page_shift) - 1;
  const LaneAt<D> lane_at(i, j);
  u32x4 k[4][kSteps];
  uint32_t page[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t t = __builtin_amdgcn_readfirstlane(min(at + 16 * h, (len - 1) & ~15u));
    page[h] = page_of(a, b, t >> a.page_shift);
    Raw<D> raw;
    load_raw<D, true, false>(a.pages + ((uint64_t)(page[h] & ~kBadPage) * a.n_heads + head) * a.page_bytes, a.page_shift,
                             t & in_page, lane_at, raw);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) k[h][st] = k_operand<D>(raw, st);
  }
  // from the first rows that see any of the workgroup's slots, this part's rounds of 32
  const int32_t tok0 = (int32_t)w_at - before;
  const uint32_t from = tok0 > 0 ? (uint32_t)tok0 * g.group / 32 * 32 : 0;
  const uint32_t share = (all_rows > from ? (all_rows - from + 32 * g.mass_parts - 1) / (32 * g.mass_parts) : 0) * 32;
  const uint32_t begin = from + part * share, rows = min(all_rows, begin + share);
  u32x4 mh[kMine], ml[kMine];
  float m_lse = 0.0f;
  auto fetch = [&](uint32_t r0) {  // rows r0 .. r0 + 31 (none beyond the last): global -> registers
#pragma unroll
    for (int f = 0; f < kMine; ++f) {
      const uint32_t id = wave + 4 * f, r = r0 + 16 * (id / kSteps) + i;
      load_q_step<D, kHalf>(g, s, head, r, rows, j, id % kSteps, mh[f], ml[f]);
    }
    if (tid < 32) {
      float v = r0 + tid < rows ? g.row_lse[(b * a.n_heads + head) * g.rows_max + r0 + tid] : INFINITY;
      if (v == -INFINITY) v = INFINITY;  // a row without slots adds nothing
      m_lse = v;
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int f = 0; f < kMine; ++f) {
      sh_q[buf][0][wave + 4 * f][lane] = mh[f];
      if constexpr (kHalf) sh_q[buf][1][wave + 4 * f][lane] = ml[f];
    }
    if (tid < 32) sh_lse[buf][tid] = m_lse;
  };
  float sum[4] = {};
  auto compute = [&](uint32_t r0, int buf) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint32_t ra = r0 + 16 * n;
      if (ra >= rows) continue;
      const int32_t seen = before + (int32_t)(ra / g.group) + 1;                               // by the first row
      const int32_t most = before + (int32_t)(min(ra + 16, rows) - 1) / (int32_t)g.group + 1;  // and the last
      if (most <= (int32_t)at) continue;
      f32x4 x[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) x[h] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 q = sh_q[buf][0][n * kSteps + st][lane];
#pragma unroll
        for (int h = 0; h < 4; ++h) x[h] = mma(q, k[h][st], x[h]);
        if constexpr (kHalf) {
          const u32x4 ql = sh_q[buf][1][n * kSteps + st][lane];
#pragma unroll
          for (int h = 0; h < 4; ++h) x[h] = mma(ql, k[h][st], x[h]);
        }
      }
      const f32x4 lse2 = *reinterpret_cast<const f32x4*>(&sh_lse[buf][16 * n + 4 * j]);
      if (seen < (int32_t)at + 64) {  // some row does not see all of the slots
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t lim = before + (int32_t)((ra + 4 * j + e) / g.group) + 1;
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if ((int32_t)(at + 16 * h + i) >= lim || ra + 4 * j + e >= rows) x[h][e] = -INFINITY;
        }
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_exp2f(fmaf(x[h][e], g.scale2, -lse2[e]));
        sum[h] += (w[0] + w[1]) + (w[2] + w[3]);
      }
    }
  };
  if (begin < rows) {
    fetch(begin);
    put(0);
  }
  auto round = [&](uint32_t r0, int buf) {
    __syncthreads();
    if (r0 + 32 < rows) fetch(r0 + 32);
    compute(r0, buf);
    if (r0 + 32 < rows) put(buf ^ 1);
  };
  for (uint32_t r0 = begin; r0 < rows; r0 += 64) {
    round(r0, 0);
    if (r0 + 32 < rows) round(r0 + 32, 1);
  }
  float own = 0.0f;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float v = sum_quarters(sum[h]);
    own = (uint32_t)h == j ? v : own;
  }
  if (at + lane >= len) return;
  if (g.mass_parts > 1) {
    g.mass_part[(((uint64_t)part * a.n_seqs + b) * a.n_heads + head) * a.max_len + at + lane] = own;
    return;
  }
  const uint32_t p = j == 0 ? page[0] : j == 1 ? page[1] : j == 2 ? page[2] : page[3];
  if (p & kBadPage) return;
  const uint64_t to = (((uint64_t)p * a.n_heads + head) << a.page_shift) + ((at + lane) & in_page);
  g.mass_out[to] = g.mass[to] + own;
}

__global__ __launch_bounds__(256) void kv4_mass_sum_kernel(AttArgs g) {
  const Batch& a = g.a;
  const uint32_t slot = blockIdx.x * 256 + threadIdx.x, head = blockIdx.y, b = blockIdx.z;
  const Seq s = seq_of(a, b);
  if (!s.ok || slot >= (uint32_t)s.len) return;
  float sum = 0.0f;
  for (uint32_t p = 0; p < g.mass_parts; ++p)
    sum += g.mass_part[(((uint64_t)p * a.n_seqs + b) * a.n_heads + head) * a.max_len + slot];
  const uint32_t page = page_of(a, b, slot >> a.page_shift);
  if (page & kBadPage) return;
  const uint64_t to = (((uint64_t)page * a.n_heads + head) << a.page_shift) + (slot & ((1u << a.page_shift) - 1));
  g.mass_out[to] = g.mass[to] + sum;
}

// How a call is cut: rows per workgroup, pieces of the long axis.
struct Plan {
  uint32_t group, rows_max, row_tiles, tile_rows, pieces, grid;
  bool mass_rows;       // the weights' kernel for many rows
  uint32_t mass_parts;  // its shares of the rows
  uint64_t part_o, part_ml, row_lse, mass_part, bytes;  // offsets in the work area
};

inline bool plan_of(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, uint32_t q_heads, bool mass, Plan* p) {
  if (q_heads == 0 || q_heads % c->n_heads || q_heads / c->n_heads > kMaxGroup) return false;
  p->group = q_heads / c->n_heads;
  const uint64_t rows = (uint64_t)b->max_new * p->group;
  // rows of a workgroup: few rows have the cache converted by every wave for itself, many share it through LDS
  p->tile_rows = rows <= 16 ? 16 : c->head_dim == 256 ? 64 : rows <= kFewRows ? 32 : 128;
  const uint64_t tiles = up(rows, p->tile_rows) / p->tile_rows, n = (uint64_t)b->n_seqs * c->n_heads * rows;
  if (tiles > 65535 || n >= (1ull << 32)) return false;
  p->rows_max = (uint32_t)rows;
  p->row_tiles = (uint32_t)tiles;
  const uint64_t across = (uint64_t)c->n_heads * (tiles ? tiles : 1);
  const uint64_t round = (p->tile_rows >= 64 ? kManySlots : kFewSlots) / across;
  uint64_t pieces = round >= 4ull * b->n_seqs ? round - b->n_seqs : 2 * round;
  if (pieces < b->n_seqs) pieces = round ? b->n_seqs : 0;  // 0: enough rows to fill the GPU, no cut
  if (p->tile_rows <= 32 && b->max_len <= kWholeLen) pieces = 0;
  if (p->tile_rows >= 64 && pieces + b->n_seqs > 65535) pieces = 0;  // a grid's third dimension
  // pieces are 128 slots or more
  const uint64_t most = (uint64_t)b->n_seqs * (up(b->max_len ? b->max_len : 1, 128) / 128);
  p->grid = pieces == 0 ? b->n_seqs : (uint32_t)(pieces + b->n_seqs < most ? pieces + b->n_seqs : most);
  p->pieces = (uint32_t)pieces;
  const uint64_t parts = p->grid > b->n_seqs ? (uint64_t)p->grid * c->n_heads * rows : 0;
  p->part_o = 0;
  p->part_ml = up(parts * c->head_dim * 4, 256);
  p->row_lse = p->part_ml + up(parts * 8, 256);
  p->mass_part = p->row_lse + (mass ? up(n * 4, 256) : 0);
  p->mass_rows = rows > (c->head_dim == 256 ? 16 : 64);
  p->mass_parts = 1;
  if (mass && p->mass_rows && n > 0) {
    const uint64_t blocks = (uint64_t)b->n_seqs * c->n_heads * ((b->max_len + 255) / 256);
    uint64_t parts_wanted = blocks >= kManySlots || blocks == 0 ? 1 : 2 * kManySlots / blocks;
    if (parts_wanted > (rows + 127) / 128) parts_wanted = (rows + 127) / 128;
    if (parts_wanted * b->n_seqs > 65535) parts_wanted = 1;
    p->mass_parts = (uint32_t)parts_wanted;
  }
  p->bytes = p->mass_part + (p->mass_parts > 1 ? up((uint64_t)p->mass_parts * b->n_seqs * c->n_heads * b->max_len * 4, 256) : 0);
  if (p->bytes < 256) p->bytes = 256;
  return true;
}

template <int D, bool kHalf>
int attend(const Plan& p, const splitzip_kv4_batch* b, const AttArgs& g, hipStream_t stream) {
  const dim3 grid(p.grid, g.a.n_heads, p.row_tiles);
  // no row at all: only the weights' arrays are copied
  if (p.rows_max > 0 && p.tile_rows >= 64) kv4_extend_kernel<D, kHalf><<<dim3(g.a.n_heads, p.row_tiles, p.grid), kAttThreads, 0, stream>>>(g);
  if constexpr (D != 256) {
    if (p.rows_max > 0 && p.tile_rows == 32) kv4_attend_kernel<D, 2, kHalf, false><<<grid, kAttThreads, 0, stream>>>(g);
  }
  if (p.rows_max > 0 && p.tile_rows == 16) {
    if (g.mass_out) kv4_attend_kernel<D, 1, kHalf, true><<<grid, kAttThreads, 0, stream>>>(g);
    else kv4_attend_kernel<D, 1, kHalf, false><<<grid, kAttThreads, 0, stream>>>(g);
  }
  if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  if (p.rows_max > 0 && p.grid > b->n_seqs) {
    // a workgroup a row until those fill the GPU
    if ((uint64_t)p.rows_max * g.a.n_heads * g.a.n_seqs <= 2048) {
      kv4_join_kernel<D, kHalf, true><<<dim3(p.rows_max, g.a.n_heads, g.a.n_seqs), 256, 0, stream>>>(g);
    } else {
      const uint32_t per = 1024 / D;
      kv4_join_kernel<D, kHalf, false>
          <<<dim3((p.rows_max + per - 1) / per, g.a.n_heads, g.a.n_seqs), 256, 0, stream>>>(g);
    }
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  }
  if (g.mass_out && b->max_len > 0) {
    const uint32_t rows = p.rows_max;
    if (!p.mass_rows) {
      // pieces of their own
      AttArgs m = g;
      const uint64_t most = (uint64_t)b->n_seqs * ((b->max_len + 127) / 128);
      uint64_t pieces = (rows <= 16 ? kMassPieces : kMassPiecesRows) / g.a.n_heads + 1;
      if (pieces < b->n_seqs) pieces = b->n_seqs;
      m.pieces = (uint32_t)pieces;
      const dim3 grid((uint32_t)(pieces + b->n_seqs < most ? pieces + b->n_seqs : most), g.a.n_heads);
      if (rows <= 16) kv4_mass_kernel<D, 1, kHalf><<<grid, kAttThreads, 0, stream>>>(m);
      if constexpr (D != 256) {
        if (rows > 48) kv4_mass_kernel<D, 4, kHalf><<<grid, kAttThreads, 0, stream>>>(m);
        else if (rows > 32) kv4_mass_kernel<D, 3, kHalf><<<grid, kAttThreads, 0, stream>>>(m);
        else if (rows > 16) kv4_mass_kernel<D, 2, kHalf><<<grid, kAttThreads, 0, stream>>>(m);
      }
    } else {
      kv4_mass_rows_kernel<D, kHalf>
          <<<dim3(g.a.n_heads, (b->max_len + 255) / 256, g.a.n_seqs * p.mass_parts), kAttThreads, 0, stream>>>(g);
      if (p.mass_parts > 1)
        kv4_mass_sum_kernel<<<dim3((b->max_len + 255) / 256, g.a.n_heads, g.a.n_seqs), 256, 0, stream>>>(g);
    }
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  }
  return SPLITZIP_OK;
}

}  // namespace kv4

extern "C" {

size_t splitzip_kv4_attention_work_bytes(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch,
                                         uint32_t n_q_heads, int with_mass) {
  using namespace kv4;
  Plan p;
  if (!cache_ok(cache) || !batch_ok(cache, batch, true) || !plan_of(cache, batch, n_q_heads, with_mass != 0, &p)) return 0;
  return p.bytes;
}

int splitzip_kv4_attention(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype,
                           const void* d_q, size_t q_row_stride, size_t q_head_stride, uint32_t n_q_heads, float scale,
                           void* d_out, float* d_lse, const float* d_mass, float* d_mass_out, void* d_work,
                           size_t work_bytes, int32_t* d_status, hipStream_t stream) {
  using namespace kv4;
  if (!cache_ok(cache) || !batch_ok(cache, batch, true)) return SPLITZIP_E_INVALID;
  if (dtype != SPLITZIP_BF16 && dtype != SPLITZIP_KV4_FP16) return SPLITZIP_E_INVALID;
  Plan p;
  if (!plan_of(cache, batch, n_q_heads, d_mass_out != nullptr, &p)) return SPLITZIP_E_INVALID;
  if (!(scale > 0.0f) || !(scale <= 3.0e38f) || !al(d_q, 16) || ((q_row_stride | q_head_stride) & 7) || !al(d_out, 16) ||
      !al(d_lse, 4) || !al(d_mass, 4) || !al(d_mass_out, 4) || !al(d_work, 256) || !al(d_status, 4) ||
      (d_mass == nullptr) != (d_mass_out == nullptr))
    return SPLITZIP_E_INVALID;
  if (batch->n_rows > 0 && (!d_q || !d_out)) return SPLITZIP_E_INVALID;
  if (batch->n_seqs == 0 || (batch->n_rows == 0 && !d_mass_out)) return SPLITZIP_OK;
  if (!d_work) return SPLITZIP_E_INVALID;
  if (work_bytes < p.bytes) return SPLITZIP_E_CAPACITY;
  AttArgs g = {};
  g.a = batch_of(cache, batch, d_status);
  g.q = static_cast<const uint8_t*>(d_q);
  g.q_row = q_row_stride;
  g.q_head = q_head_stride;
  g.out = static_cast<uint8_t*>(d_out);
  g.lse = d_lse;
  g.mass = d_mass;
  g.mass_out = d_mass_out;
  uint8_t* w = static_cast<uint8_t*>(d_work);
  g.part_o = reinterpret_cast<float*>(w + p.part_o);
  g.part_ml = reinterpret_cast<float*>(w + p.part_ml);
  g.row_lse = d_mass_out ? reinterpret_cast<float*>(w + p.row_lse) : nullptr;
  g.mass_part = reinterpret_cast<float*>(w + p.mass_part);
  g.mass_parts = p.mass_parts;
  g.q_heads = n_q_heads;
  g.group = p.group;
  g.rows_max = p.rows_max;
  g.pieces = p.pieces;
  g.scale2 = scale * 1.44269504088896341f;
  const bool half = dtype == SPLITZIP_KV4_FP16;
  if (cache->head_dim == 64) return half ? attend<64, true>(p, batch, g, stream) : attend<64, false>(p, batch, g, stream);
  if (cache->head_dim == 128)
    return half ? attend<128, true>(p, batch, g, stream) : attend<128, false>(p, batch, g, stream);
  return half ? attend<256, true>(p, batch, g, stream) : attend<256, false>(p, batch, g, stream);
}

}  // extern "C"

#endif
