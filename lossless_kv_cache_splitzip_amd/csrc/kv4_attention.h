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

constexpr int kAttThreads = 256;  // 4 waves, each with key tiles of its own

struct AttArgs {
  Batch a;
  const uint8_t* q;
  uint64_t q_row, q_head;  // strides in elements
  uint8_t* out;
  float* lse;
  const float* mass;
  float* mass_out;
  float* part_o;    // [seq][head][split][rows_pad][D] unnormalised sums
  float* part_ml;   // [seq][head][split][rows_pad][2] largest logit (base 2), sum
  float* row_lse;   // [seq][head][rows_pad] log2 of the sums, for the weights
  uint32_t q_heads, group;
  uint32_t rows_pad;    // rows (token, head of the group) of the longest sequence, a multiple of 16
  uint32_t splits;      // of the long axis
  uint32_t split_len;   // slots each, a multiple of 128
  float scale2;         // scale * log2 e
};

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

// Query rows as the right operand: row r = token * group + head in the group.
// Rows beyond `rows` are zero.  lo: what BF16 leaves of FP16 values.
template <int D, bool kHalf>
__device__ inline void load_q(const AttArgs& g, const Seq& s, uint32_t head, uint32_t r, uint32_t rows, uint32_t j,
                              u32x4 hi[D / 32], u32x4 lo[D / 32]) {
  const uint32_t tok = r / g.group, hg = r % g.group;
  const uint8_t* p = g.q + 2 * (((uint64_t)s.row0 + tok) * g.q_row + (uint64_t)(head * g.group + hg) * g.q_head);
#pragma unroll
  for (int m = 0; m < D / 32; ++m) {
    u32x4 x = {0, 0, 0, 0};
    if (r < rows) x = *reinterpret_cast<const u32x4*>(p + 2 * chan_of<D>(m, j));
    if constexpr (kHalf) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = (float)__builtin_bit_cast(_Float16, (uint16_t)x[e]);
        const float b = (float)__builtin_bit_cast(_Float16, (uint16_t)(x[e] >> 16));
        hi[m][e] = pack_bf16(a, b);
        lo[m][e] = pack_bf16(a - bf16_lo(hi[m][e]), b - bf16_hi(hi[m][e]));
      }
    } else {
      hi[m] = x;
    }
  }
}

// One lane's share of 16 keys: K codes of its key and quarter, V codes of 4
// tokens and D/16 channels, and their scales.
template <int D>
struct Raw {
  uint32_t k[D / 32], v[D / 32];
  uint32_t ks, vs;
};

// Lane (i, j)'s bytes of the 16 slots at `t` (in a page) of `base`.
template <int D>
__device__ inline void load_raw(const uint8_t* base, uint32_t shift, uint32_t t, uint32_t i, uint32_t j, Raw<D>& r,
                                bool want_v = true) {
  using L = Layout<D>;
  const uint8_t* k = base + (t + i) * L::kCode;
  const uint8_t* ks = base + L::k_scales(shift) + (t + i) * L::kScale;
  const uint8_t* v = base + L::v_codes(shift) + L::v_piece(t + 4 * j, i);
  const uint8_t* vs = base + L::v_scales(shift) + L::v_scale(t + 4 * j, i * L::kScale / 16);
  if constexpr (D == 64) {
    *reinterpret_cast<u32x2*>(r.k) = *reinterpret_cast<const u32x2*>(k + 8 * j);
    r.ks = ks[j >> 1];
    if (want_v) *reinterpret_cast<u32x2*>(r.v) = *reinterpret_cast<const u32x2*>(v);
  } else if constexpr (D == 128) {
    *reinterpret_cast<u32x4*>(r.k) = *reinterpret_cast<const u32x4*>(k + 16 * j);
    r.ks = ks[j];
    if (want_v) *reinterpret_cast<u32x4*>(r.v) = *reinterpret_cast<const u32x4*>(v);
  } else {
    *reinterpret_cast<u32x4*>(r.k) = *reinterpret_cast<const u32x4*>(k + 16 * j);
    *reinterpret_cast<u32x4*>(r.k + 4) = *reinterpret_cast<const u32x4*>(k + 64 + 16 * j);
    r.ks = ks[j] | (uint32_t)ks[4 + j] << 8;
    if (want_v) {
      *reinterpret_cast<u32x4*>(r.v) = *reinterpret_cast<const u32x4*>(v);
      *reinterpret_cast<u32x4*>(r.v + 4) = *reinterpret_cast<const u32x4*>(v + 16);
    }
  }
  if (want_v) r.vs = *reinterpret_cast<const uint32_t*>(vs);
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

template <int D, int kPair, int kRows, bool kTwo>
__device__ inline void pv_step(const Raw<D>& a, const float sa[4], const Raw<D>& b, const float sb[4],
                               const u32x4 (&p)[kRows], const u32x4 (&pl)[kRows], f32x4 (&o)[kRows][D / 16]) {
  if constexpr (kPair < D / 32) {
    u32x4 x, y;
    v_operands<D, kPair>(a, sa, b, sb, x, y);
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      o[n][2 * kPair] = mma(x, p[n], o[n][2 * kPair]);
      o[n][2 * kPair + 1] = mma(y, p[n], o[n][2 * kPair + 1]);
      if constexpr (kTwo) {
        o[n][2 * kPair] = mma(x, pl[n], o[n][2 * kPair]);
        o[n][2 * kPair + 1] = mma(y, pl[n], o[n][2 * kPair + 1]);
      }
    }
    pv_step<D, kPair + 1, kRows, kTwo>(a, sa, b, sb, p, pl, o);
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

// One workgroup: the slots of one split, 16 kRows query rows of one KV head of
// one sequence.  Each wave takes every 4th tile of 32 slots with a softmax of
// its own; the four are joined through LDS.
template <int D, int kRows, bool kHalf>
__global__ __launch_bounds__(kAttThreads) void kv4_attend_kernel(AttArgs g) {
  constexpr int kSteps = D / 32;
  __shared__ float sh_o[4][16][D + 4];
  __shared__ float sh_m[4][16 * kRows], sh_l[4][16 * kRows];
  const Batch& a = g.a;
  const uint32_t split = blockIdx.x, b = blockIdx.z;
  const uint32_t head = blockIdx.y % a.n_heads, tile = blockIdx.y / a.n_heads;
  const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, j = lane >> 4;
  const Seq s = seq_of(a, b);
  if (!s.ok && tid == 0) corrupt(a.status);
  const uint32_t rows = (uint32_t)s.rows * g.group, r0 = tile * 16 * kRows;
  if (r0 >= rows) return;
  // what each row sees: row r's last slot is len - rows + token
  const int32_t before = s.len - s.rows;
  const int32_t newest = before + (int32_t)(min(r0 + 16 * kRows, rows) - 1) / (int32_t)g.group;
  const uint32_t seen = newest < 0 ? 0u : (uint32_t)newest + 1;  // slots that any row of this tile sees
  const uint32_t c0 = split * g.split_len, c1 = min(seen, c0 + g.split_len);
  if (c0 >= c1 && split > 0) return;  // split 0 writes what rows without slots get

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
  const uint32_t in_page = (1u << a.page_shift) - 1;
  auto load_tile = [&](uint32_t at, Raw<D> (&r)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // a half tile wholly behind the end loads the last slots there are instead, unused
      const uint32_t t = __builtin_amdgcn_readfirstlane(min(at + 16 * h, (c1 - 1) & ~15u));
      const uint32_t p = page_of(a, b, t >> a.page_shift);
      const uint8_t* base = a.pages + ((uint64_t)p * a.n_heads + head) * a.page_bytes;
      load_raw<D>(base, a.page_shift, t & in_page, i, j, r[h]);
    }
  };
  Raw<D> cur[2], nxt[2];
  uint32_t at = c0 + 32 * wave;
  if (at < c1) load_tile(at, nxt);
  for (; at < c1; at += 128) {
    cur[0] = nxt[0];
    cur[1] = nxt[1];
    if (at + 128 < c1) load_tile(at + 128, nxt);
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
    pv_step<D, 0, kRows, true>(cur[0], sa, cur[1], sb, p, pl, o);
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
  const uint32_t row_base = (b * a.n_heads + head) * g.rows_pad;  // fits: checked on the host
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
      const uint64_t part = ((uint64_t)(b * a.n_heads + head) * g.splits + split) * g.rows_pad + r;
      const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
      for (uint32_t c = 2 * (tid & 15); c < (uint32_t)D; c += 32) {
        float u = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          u += sh_o[w][row][c];
          v += sh_o[w][row][c + 1];
        }
        if (g.splits == 1) {
          store2(g.out, out_row * D + c, kHalf, u * inv, v * inv);
        } else {
          g.part_o[part * D + c] = u;
          g.part_o[part * D + c + 1] = v;
        }
      }
      if ((tid & 15) == 0) {
        const float top2 = all * g.scale2;
        if (g.splits == 1) {
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

// Joins the splits: one row (query head of a token) per D / 4 lanes.
template <int D, bool kHalf>
__global__ __launch_bounds__(256) void kv4_join_kernel(AttArgs g) {
  constexpr uint32_t kLanes = D / 4;
  const Batch& a = g.a;
  const uint32_t b = blockIdx.z, head = blockIdx.y;
  const uint32_t r = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes, c = 4 * (threadIdx.x % kLanes);
  const Seq s = seq_of(a, b);
  if (r >= (uint32_t)s.rows * g.group) return;
  const int32_t newest = s.len - s.rows + (int32_t)(r / g.group);
  const uint32_t seen = newest < 0 ? 0u : (uint32_t)newest + 1;
  const uint32_t n = max(1u, (seen + g.split_len - 1) / g.split_len);  // splits with slots of this row
  const uint64_t first = (uint64_t)(b * a.n_heads + head) * g.splits * g.rows_pad + r;
  float top = -INFINITY;
  for (uint32_t k = 0; k < n; ++k) top = fmaxf(top, g.part_ml[2 * (first + (uint64_t)k * g.rows_pad)]);
  float sum = 0.0f;
  f32x4 o = {0, 0, 0, 0};
  for (uint32_t k = 0; k < n; ++k) {
    const uint64_t at = first + (uint64_t)k * g.rows_pad;
    const float mk = g.part_ml[2 * at];
    if (mk == -INFINITY) continue;
    const float f = __builtin_amdgcn_exp2f(mk - top);
    sum += g.part_ml[2 * at + 1] * f;
    o += *reinterpret_cast<const f32x4*>(g.part_o + at * D + c) * f;
  }
  const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
  const uint64_t out_row = ((uint64_t)s.row0 + r / g.group) * g.q_heads + head * g.group + r % g.group;
  store2(g.out, out_row * D + c, kHalf, o[0] * inv, o[1] * inv);
  store2(g.out, out_row * D + c + 2, kHalf, o[2] * inv, o[3] * inv);
  if (c == 0) {
    const float lse2 = sum == 0.0f ? -INFINITY : top + __builtin_amdgcn_logf(sum);
    if (g.lse) g.lse[out_row] = lse2 * 0.69314718055994531f;
    if (g.row_lse) g.row_lse[(b * a.n_heads + head) * g.rows_pad + r] = lse2;
  }
}

// Adds the weights that each slot drew: the logits again (K is half of the
// cache), p = 2^(x - lse) and its sum over the rows, in a fixed order.  A wave
// has 32 slots.
template <int D, bool kHalf>
__global__ __launch_bounds__(kAttThreads) void kv4_mass_kernel(AttArgs g) {
  constexpr int kSteps = D / 32;
  const Batch& a = g.a;
  const uint32_t b = blockIdx.z, head = blockIdx.y;
  const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, j = lane >> 4;
  const Seq s = seq_of(a, b);
  if (!s.ok) return;
  const uint32_t at = (blockIdx.x * 4 + wave) * 32, len = (uint32_t)s.len;
  if (at >= len) return;
  const uint32_t rows = (uint32_t)s.rows * g.group;
  const int32_t before = s.len - s.rows;
  const uint32_t in_page = (1u << a.page_shift) - 1;
  Raw<D> raw[2];
  uint32_t page[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t t = __builtin_amdgcn_readfirstlane(min(at + 16 * h, (len - 1) & ~15u));
    page[h] = page_of(a, b, t >> a.page_shift);
    load_raw<D>(a.pages + ((uint64_t)page[h] * a.n_heads + head) * a.page_bytes, a.page_shift, t & in_page, i, j,
                raw[h], false);
  }
  float add[2][4] = {};
  for (uint32_t r0 = 0; r0 < rows; r0 += 16) {
    if (before + (int32_t)(min(r0 + 16, rows) - 1) / (int32_t)g.group < (int32_t)at) continue;  // rows before these slots
    u32x4 qh[kSteps], ql[kSteps];
    const uint32_t r = r0 + i;
    load_q<D, kHalf>(g, s, head, r, rows, j, qh, ql);
    const int32_t lim = before + (int32_t)(r / g.group) + 1;
    const float lse2 = r < rows ? g.row_lse[(b * a.n_heads + head) * g.rows_pad + r] : INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 x = {0, 0, 0, 0};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 k = k_operand<D>(raw[h], st);
        x = mma(k, qh[st], x);
        if constexpr (kHalf) x = mma(k, ql[st], x);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r < rows && (int32_t)(at + 16 * h + 4 * j + e) < lim)
          add[h][e] += __builtin_amdgcn_exp2f(fmaf(x[e], g.scale2, -lse2));
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = add[h][e];
#pragma unroll
      for (int k = 1; k < 16; k *= 2) v += __shfl_xor(v, k, 64);
      const uint32_t slot = at + 16 * h + 4 * j + e;
      if (i == 0 && slot < len) {
        const uint64_t to = (((uint64_t)page[h] * a.n_heads + head) << a.page_shift) + (slot & in_page);
        g.mass_out[to] = g.mass[to] + v;
      }
    }
}

// How a call is cut: rows per workgroup, splits of the long axis.
struct Plan {
  uint32_t group, rows_pad, row_tiles, tile_rows, splits, split_len;
  uint64_t part_o, part_ml, row_lse, bytes;  // offsets in the work area
};

inline bool plan_of(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, uint32_t q_heads, bool mass, Plan* p) {
  if (q_heads == 0 || q_heads % c->n_heads || q_heads / c->n_heads > kMaxGroup) return false;
  p->group = q_heads / c->n_heads;
  const uint64_t rows = (uint64_t)b->max_new * p->group;
  p->tile_rows = rows <= 16 || c->head_dim == 256 ? 16 : 32;  // 32 rows of 256 channels do not fit the registers
  p->rows_pad = (uint32_t)up(rows, 64);
  p->row_tiles = (uint32_t)(up(rows, p->tile_rows) / p->tile_rows);
  const uint64_t heads = (uint64_t)b->n_seqs * c->n_heads;
  // about 1024 workgroups (4 on each compute unit), 128 slots or more each
  const uint64_t total = heads * p->row_tiles * b->max_len;
  uint64_t len = up(total / 1024 + 1, 128);
  if (len > b->max_len) len = up(b->max_len ? b->max_len : 1, 128);
  p->split_len = (uint32_t)len;
  p->splits = (uint32_t)((b->max_len + len - 1) / len);
  if (p->splits == 0) p->splits = 1;
  const uint64_t n = heads * p->rows_pad, parts = p->splits > 1 ? n * p->splits : 0;
  if (n >= (1ull << 32) || (uint64_t)p->row_tiles * c->n_heads > 65535) return false;
  p->part_o = 0;
  p->part_ml = up(parts * c->head_dim * 4, 256);
  p->row_lse = p->part_ml + up(parts * 8, 256);
  p->bytes = p->row_lse + (mass ? up(n * 4, 256) : 0);
  if (p->bytes < 256) p->bytes = 256;
  return true;
}

template <int D, bool kHalf>
int attend(const Plan& p, const splitzip_kv4_batch* b, const AttArgs& g, hipStream_t stream) {
  const dim3 grid(p.splits, p.row_tiles * g.a.n_heads, g.a.n_seqs);
  if constexpr (D != 256) {
    if (p.tile_rows == 32) kv4_attend_kernel<D, 2, kHalf><<<grid, kAttThreads, 0, stream>>>(g);
  }
  if (p.tile_rows == 16) kv4_attend_kernel<D, 1, kHalf><<<grid, kAttThreads, 0, stream>>>(g);
  if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  if (p.splits > 1) {
    const uint32_t per = 256 / (D / 4);
    kv4_join_kernel<D, kHalf>
        <<<dim3((b->max_new * p.group + per - 1) / per, g.a.n_heads, g.a.n_seqs), 256, 0, stream>>>(g);
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  }
  if (g.mass_out && b->max_len > 0) {
    kv4_mass_kernel<D, kHalf><<<dim3((b->max_len + 127) / 128, g.a.n_heads, g.a.n_seqs), kAttThreads, 0, stream>>>(g);
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
  g.q_heads = n_q_heads;
  g.group = p.group;
  g.rows_pad = p.rows_pad;
  g.splits = p.splits;
  g.split_len = p.split_len;
  g.scale2 = scale * 1.44269504088896341f;
  const bool half = dtype == SPLITZIP_KV4_FP16;
  if (cache->head_dim == 64) return half ? attend<64, true>(p, batch, g, stream) : attend<64, false>(p, batch, g, stream);
  if (cache->head_dim == 128)
    return half ? attend<128, true>(p, batch, g, stream) : attend<128, false>(p, batch, g, stream);
  return half ? attend<256, true>(p, batch, g, stream) : attend<256, false>(p, batch, g, stream);
}

}  // extern "C"

#endif
