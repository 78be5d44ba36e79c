// The 4-bit cache's encoder and decoder (splitzip_kv4_append, splitzip_kv4_read).
//
// A lane holds 8 channels of one row of one head: one wide load, one code
// dword.  Lanes run over 4 rows first, then over the channels, so the stores of
// a wave fill runs of both code sections: V codes interleave 4 tokens
// (kv4_common.h), K codes are a token's row.  A block of 32 channels is then 4
// lanes, 4 apart in a row of 16, whose largest magnitude two row rotations give.
// Both kernels move each byte once and are bound by memory, for a few rows by
// the launch and the chain lengths -> block table -> page (64 rows: 4.0 and 3.5
// us).  21,249 rows of 8 heads of 128 BF16 channels: append 25 us for 111 MB,
// read 20.5 us for 110 MB.
#ifndef SPLITZIP_KV4_CODEC_H
#define SPLITZIP_KV4_CODEC_H

#include <type_traits>

#include "kv4_common.h"

namespace kv4 {

constexpr int kRowThreads = 256;
constexpr uint64_t kEnoughWaves = 4096;  // 1024 to 8192 measure alike
// Where 4 rows take at most so many lanes, a wave has 8 or 16 rows (177,803 rows
// of one head, append and read: 64 channels 56 -> 37 us, 128 60 -> 54; at 256
// lanes 95 -> 90 for BF16, but 50 -> 52.6 for 48,756 rows of E5M2).
constexpr uint32_t kNarrowLanes = 128;

struct RowArgs {
  Batch a;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* k_out;
  uint8_t* v_out;
  uint64_t k_row, k_head, v_row, v_head;  // strides in elements
  uint32_t rows, width;                   // a wave's packed rows: 4, 8 or 16; lanes that 4 rows take
  uint32_t chunks, per_wave, waves;       // of those rows: pieces of 64 lanes, how many a wave does, waves
  const int32_t* positions;
  float* mass;
  int32_t* pos;
};

// 8 elements of type T (a splitzip type) as they lie in memory.
template <int T>
using Eight = std::conditional_t<T == SPLITZIP_FP8_E5M2, u32x2, u32x4>;

template <int T>
__device__ inline Eight<T> load8(const uint8_t* p, uint64_t elem) {
  return __builtin_nontemporal_load(reinterpret_cast<const Eight<T>*>(p + (T == SPLITZIP_FP8_E5M2 ? 1 : 2) * elem));
}

// And as 16-bit floats, BF16 or (E5M2 is the upper half of one) FP16.
template <int T>
__device__ inline u32x4 as16(const Eight<T> q) {
  if constexpr (T == SPLITZIP_FP8_E5M2)
    return u32x4{__builtin_amdgcn_perm(0, q[0], 0x010C000C), __builtin_amdgcn_perm(0, q[0], 0x030C020C),
                 __builtin_amdgcn_perm(0, q[1], 0x010C000C), __builtin_amdgcn_perm(0, q[1], 0x030C020C)};
  else
    return q;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ inline u16x2 max2(uint32_t a, uint32_t b) {
  return __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
}

// The largest of 8 magnitudes (their bits compare as integers).
__device__ inline uint32_t top8(const u32x4 q) {
  const uint32_t m = 0x7FFF7FFFu;
  const u16x2 t = __builtin_elementwise_max(max2(q[0] & m, q[1] & m), max2(q[2] & m, q[3] & m));
  return t[0] > t[1] ? t[0] : t[1];
}

// The largest of the 4 lanes 4 apart in this lane's row of 16.
__device__ inline uint32_t max_of_block(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124 /* row_ror:4 */, 0xF, 0xF, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128 /* row_ror:8 */, 0xF, 0xF, false);
  return v > o ? v : o;
}

// Codes of this lane's 8 channels and the scale byte of their block (all 4
// lanes of a block take part).  The instruction rounds BF16 and FP16 to E2M1
// under the scale, to nearest even and saturating, infinities too.
template <int T>
__device__ inline uint32_t encode8(u32x4 q, uint32_t& scale, bool& odd) {
  constexpr uint32_t kInf = T == SPLITZIP_BF16 ? 0x7F80u : 0x7C00u;
  uint32_t top = max_of_block(top8(q));
  if (__any(top >= kInf)) {  // rare: NaN becomes 0, and neither it nor infinity counts for the scale
    odd = top >= kInf;
    u32x4 finite = q;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t half = 0xFFFFu << (16 * (i & 1)), m = (q[i / 2] >> (16 * (i & 1))) & 0x7FFFu;
      if (m > kInf) q[i / 2] &= ~half;
      if (m >= kInf) finite[i / 2] &= ~half;
    }
    top = max_of_block(top8(finite));
  }
  // the least e with max < 7 * 2^e: 7/4 of a power of two is the border
  const uint32_t bits = T == SPLITZIP_BF16 ? top << 16 : __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)top));
  int s = (int)(bits >> 23) - 2 + ((bits & 0x7FFFFFu) >= 0x600000u ? 1 : 0);
  s = s < 1 ? 1 : s > 252 ? 252 : s;
  scale = (uint32_t)s;
  const float f = scale_of(scale);
  const uint32_t q0 = q[0], q1 = q[1], q2 = q[2], q3 = q[3];
  uint32_t c = 0;
  if constexpr (T == SPLITZIP_BF16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, q0), f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, q1), f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, q2), f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, q3), f, 3);
  } else {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, q0), f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, q1), f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, q2), f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, q3), f, 3);
  }
  return c;
}

// A wave of the row kernels has 4 packed rows and some of their heads, or where
// heads are few 8 or 16 rows with all of them: lanes run over 4 rows first, then
// over 8 channels each, the heads, and the next 4 rows, in chunks of 64 lanes.
// What belongs to the rows is looked up once, by the lanes of their numbers.
// Rows that start at a multiple of 4 slots fill whole words of the V codes,
// others two parts of them.  The grid goes by the packed rows alone, however
// ragged the batch.
struct Place {
  uint32_t row;       // packed
  uint32_t slot, t;   // its slot, in the sequence and in the page
  uint32_t page;      // kBadPage: no slot, or a page number outside the pool
};

// The sequence of a packed row: the first whose rows end behind it.  64
// sequences are looked at in one round of loads, with one vote a row.
__device__ inline uint32_t seq_of_row(const Batch& a, uint32_t row0, uint32_t t, uint32_t rows) {
  if (!a.cu) return row0 + t;
  const uint32_t lane = threadIdx.x & 63;
  uint32_t seq = a.n_seqs;
  for (uint32_t b = 0; b < a.n_seqs; b += 64) {
    const int32_t end = b + lane < a.n_seqs ? a.cu[b + lane + 1] : 0;
    uint32_t mine = a.n_seqs;
    for (uint32_t g = 0; g < rows; g += 4) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const uint64_t hit = __ballot(b + lane < a.n_seqs && end > (int32_t)(row0 + g + k));
        if (g + k == t && hit) mine = b + (uint32_t)__builtin_ctzll(hit);
      }
    }
    if (mine < seq) seq = mine;
    if (__all(seq < a.n_seqs)) break;
  }
  return seq;
}

__device__ inline Place place_of(const Batch& a, uint32_t row0, uint32_t rows) {
  const uint32_t t = threadIdx.x & (rows - 1);
  Place p = {row0 + t, 0, 0, kBadPage};
  const uint32_t b = seq_of_row(a, row0, t, rows);
  if (p.row >= a.n_rows || b >= a.n_seqs) return p;
  const Seq s = seq_of(a, b);
  if (!s.ok || s.rows > s.len || p.row < (uint32_t)s.row0 || p.row >= (uint32_t)(s.row0 + s.rows)) return p;
  p.slot = (uint32_t)(s.len - s.rows) + (p.row - (uint32_t)s.row0);
  p.t = p.slot & ((1u << a.page_shift) - 1);
  p.page = page_of(a, b, p.slot >> a.page_shift);
  return p;
}

// A lane's 4 rows (of the wave's), head and 8 channels (8u ..) in a chunk;
// `in`: there are such.
template <int D, bool kNarrow>
struct Col {
  uint32_t group = 0, head, u;
  bool in;
  __device__ Col(const RowArgs& r, uint32_t chunk) {
    uint32_t col = chunk * 64 + (threadIdx.x & 63);
    if constexpr (kNarrow) {
      group = (col >= r.width ? 1 : 0) + (col >= 2 * r.width ? 1 : 0) + (col >= 3 * r.width ? 1 : 0);
      col -= group * r.width;
    }
    head = col / (D / 2);
    u = col % (D / 2) >> 2;
    in = head < r.a.n_heads && (!kNarrow || 4 * group < r.rows);
  }
  // What the lane of this lane's row holds: all 64 lanes ask.
  __device__ uint32_t of_row(const RowArgs& r, uint32_t v) const {
    return kNarrow ? (uint32_t)__shfl((int)v, (int)(4 * group + (threadIdx.x & 3))) : v;
  }
};

constexpr uint32_t kTogetherRows = 4;  // chunks whose loads are under way together

// Reports sequences out of bounds: the last workgroup's job, as a bad one may
// have no row that finds it.
__device__ inline void report_bad(const Batch& a) {
  if (blockIdx.x != gridDim.x - 1 || !a.status) return;
  for (uint32_t b = threadIdx.x; b < a.n_seqs; b += kRowThreads) {
    const Seq s = seq_of(a, b);
    if (!s.ok || s.rows > s.len) corrupt(a.status);
  }
}

template <int D, int T, bool kNarrow>
__global__ __launch_bounds__(kRowThreads) void kv4_append_kernel(RowArgs r) {
  using L = Layout<D>;
  const Batch& a = r.a;
  report_bad(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6));
  const uint32_t rows = kNarrow ? r.rows : 4;
  const uint32_t row0 = wave / r.waves * rows, first = wave % r.waves * r.per_wave, end = min(first + r.per_wave, r.chunks);
  if (row0 >= a.n_rows) return;
  Eight<T> kq[kTogetherRows], vq[kTogetherRows];
  auto load = [&](uint32_t c) {  // rows that turn out to have no slot, too
#pragma unroll
    for (uint32_t n = 0; n < kTogetherRows; ++n) {
      const Col<D, kNarrow> col(r, c + n);
      const uint64_t row = row0 + 4 * col.group + (threadIdx.x & 3);
      kq[n] = vq[n] = Eight<T>{};
      if (c + n < end && col.in && row < a.n_rows) {
        kq[n] = load8<T>(r.k, row * r.k_row + col.head * r.k_head + 8 * col.u);
        vq[n] = load8<T>(r.v, row * r.v_row + col.head * r.v_head + 8 * col.u);
      }
    }
  };
  load(first);
  const Place p = place_of(a, row0, rows);
  const uint32_t sh = a.page_shift;
  const int32_t position = r.positions && r.pos && p.page != kBadPage ? r.positions[p.row] : (int32_t)p.slot;
  bool odd = false;
  for (uint32_t c = first; c < end; c += kTogetherRows) {
    if (c > first) load(c);
#pragma unroll
    for (uint32_t n = 0; n < kTogetherRows; ++n) {
      if (c + n >= end) break;
      const Col<D, kNarrow> col(r, c + n);
      const uint32_t page = col.of_row(r, p.page), t = col.of_row(r, p.t);
      const int32_t at_position = (int32_t)col.of_row(r, (uint32_t)position);
      uint32_t ks, vs;
      bool k_odd = false, v_odd = false;
      const uint32_t kc = encode8<T>(as16<T>(kq[n]), ks, k_odd), vc = encode8<T>(as16<T>(vq[n]), vs, v_odd);
      if (page == kBadPage || !col.in) continue;
      odd |= k_odd | v_odd;
      uint8_t* base = a.pages + (uint64_t)page * a.n_heads * a.page_bytes + col.head * a.page_bytes;
      *reinterpret_cast<uint32_t*>(base + t * L::kCode + 4 * col.u) = kc;
      uint8_t* v = base + L::v_codes(sh);
      if constexpr (D == 64) {  // 8 channels are two pieces of 2 bytes
        *reinterpret_cast<uint16_t*>(v + L::v_piece(t, 2 * col.u)) = (uint16_t)vc;
        *reinterpret_cast<uint16_t*>(v + L::v_piece(t, 2 * col.u + 1)) = (uint16_t)(vc >> 16);
      } else if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(v + L::v_piece(t, col.u)) = vc;
      } else {  // half a piece of 8 bytes
        *reinterpret_cast<uint32_t*>(v + L::v_piece(t, col.u >> 1) + 4 * (col.u & 1)) = vc;
      }
      if ((col.u & 3) == 0) {
        base[L::k_scales(sh) + t * L::kScale + col.u / 4] = (uint8_t)ks;
        base[L::v_scales(sh) + L::v_scale(t, col.u / 4)] = (uint8_t)vs;
      }
      if (col.u == 0) {
        const uint64_t at = (((uint64_t)page * a.n_heads + col.head) << sh) + t;
        if (r.mass) r.mass[at] = 0.0f;
        if (r.pos) r.pos[at] = at_position;
      }
    }
  }
  if (odd && a.status) {
    int32_t none = SPLITZIP_OK;
    __hip_atomic_compare_exchange_strong(a.status, &none, SPLITZIP_E_NONFINITE, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
  }
}

// 8 codes of one block as 8 values of type T, 16 bytes.
template <int T>
__device__ inline u32x4 decode8(uint32_t c, uint32_t scale) {
  const float f = scale_of(scale);
  u32x4 o;
  if constexpr (T == SPLITZIP_BF16) {  // two bits of precision: exact
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 3));
  } else {
    auto two = [](bf16x2 p) {
      const uint32_t lo = __builtin_bit_cast(uint16_t, (_Float16)(float)p[0]);
      const uint32_t hi = __builtin_bit_cast(uint16_t, (_Float16)(float)p[1]);
      return lo | hi << 16;
    };
    o[0] = two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 0));
    o[1] = two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 1));
    o[2] = two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 2));
    o[3] = two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, f, 3));
  }
  return o;
}

// The rows are not read again here: past the caches (24,348 rows: 45.8 -> 29.4 us between other work).
__device__ inline void put16(uint8_t* p, u32x4 v) { __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p)); }

template <int D, int T, bool kNarrow>
__global__ __launch_bounds__(kRowThreads) void kv4_read_kernel(RowArgs r) {
  using L = Layout<D>;
  const Batch& a = r.a;
  report_bad(a);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6));
  const uint32_t rows = kNarrow ? r.rows : 4;
  const uint32_t row0 = wave / r.waves * rows, first = wave % r.waves * r.per_wave, end = min(first + r.per_wave, r.chunks);
  if (row0 >= a.n_rows) return;
  const Place p = place_of(a, row0, rows);
  if (!__any(p.page != kBadPage)) return;
  const uint32_t sh = a.page_shift;
  for (uint32_t c = first; c < end; c += kTogetherRows) {
    uint32_t kc[kTogetherRows], vc[kTogetherRows], ks[kTogetherRows], vs[kTogetherRows];
    bool on[kTogetherRows];
#pragma unroll
    for (uint32_t n = 0; n < kTogetherRows; ++n) {
      const Col<D, kNarrow> col(r, c + n);
      const uint32_t page = col.of_row(r, p.page), t = col.of_row(r, p.t);
      kc[n] = vc[n] = ks[n] = vs[n] = 0;
      on[n] = c + n < end && col.in && page != kBadPage;
      if (!on[n]) continue;
      const uint8_t* base = a.pages + (uint64_t)page * a.n_heads * a.page_bytes + col.head * a.page_bytes;
      if (r.k_out) {
        kc[n] = *reinterpret_cast<const uint32_t*>(base + t * L::kCode + 4 * col.u);
        ks[n] = base[L::k_scales(sh) + t * L::kScale + col.u / 4];
      }
      if (r.v_out) {
        const uint8_t* v = base + L::v_codes(sh);
        if constexpr (D == 64) {
          vc[n] = *reinterpret_cast<const uint16_t*>(v + L::v_piece(t, 2 * col.u)) |
                  (uint32_t) * reinterpret_cast<const uint16_t*>(v + L::v_piece(t, 2 * col.u + 1)) << 16;
        } else if constexpr (D == 128) {
          vc[n] = *reinterpret_cast<const uint32_t*>(v + L::v_piece(t, col.u));
        } else {
          vc[n] = *reinterpret_cast<const uint32_t*>(v + L::v_piece(t, col.u >> 1) + 4 * (col.u & 1));
        }
        vs[n] = base[L::v_scales(sh) + L::v_scale(t, col.u / 4)];
      }
    }
#pragma unroll
    for (uint32_t n = 0; n < kTogetherRows; ++n) {
      const Col<D, kNarrow> col(r, c + n);
      if (!on[n]) continue;
      const uint64_t row = row0 + 4 * col.group + (threadIdx.x & 3);
      const uint64_t at = (row * a.n_heads + col.head) * D + 8 * col.u;
      if (r.k_out) put16(r.k_out + 2 * at, decode8<T>(kc[n], ks[n]));
      if (r.v_out) put16(r.v_out + 2 * at, decode8<T>(vc[n], vs[n]));
    }
  }
}

// Workgroups for all packed rows (0: more than 2^24); a wave takes one chunk of
// 64 lanes where rows are few, up to 8 where there are more than enough (21,251
// rows of 8 heads: append 31 -> 25 us, read 22 -> 20.5): of 4 rows, or where
// these have fewer, of 8 or 16.
inline uint32_t row_blocks(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, RowArgs* r) {
  r->width = c->n_heads * (c->head_dim / 2);
  r->rows = 4;
  while (r->rows < 16 && r->rows / 4 * r->width <= kNarrowLanes && b->n_rows >= 2 * r->rows * kEnoughWaves) r->rows *= 2;
  const uint64_t groups = ((uint64_t)b->n_rows + r->rows - 1) / r->rows;
  r->chunks = (r->rows / 4 * r->width + 63) / 64;
  const uint64_t all = groups * r->chunks;
  r->per_wave = all >= 8 * kEnoughWaves ? 8 : all >= 4 * kEnoughWaves ? 4 : all >= 2 * kEnoughWaves ? 2 : 1;
  if (r->rows > 4) r->per_wave = r->chunks;
  r->waves = (r->chunks + r->per_wave - 1) / r->per_wave;
  const uint64_t n = up(groups * r->waves, kRowThreads / 64) / (kRowThreads / 64);
  return n < (1ull << 24) ? (uint32_t)n : 0;
}

template <template <int, int, bool> class Launch, int T, bool N>
void dispatch_dim(uint32_t dim, const RowArgs& r, dim3 grid, hipStream_t stream) {
  if (dim == 64) Launch<64, T, N>::go(r, grid, stream);
  else if (dim == 128) Launch<128, T, N>::go(r, grid, stream);
  else Launch<256, T, N>::go(r, grid, stream);
}

template <template <int, int, bool> class Launch, bool N>
int dispatch_type(uint32_t dim, int dtype, const RowArgs& r, dim3 grid, hipStream_t stream) {
  if (dtype == SPLITZIP_BF16) dispatch_dim<Launch, SPLITZIP_BF16, N>(dim, r, grid, stream);
  else if (dtype == SPLITZIP_KV4_FP16) dispatch_dim<Launch, SPLITZIP_KV4_FP16, N>(dim, r, grid, stream);
  else dispatch_dim<Launch, SPLITZIP_FP8_E5M2, N>(dim, r, grid, stream);
  return hipGetLastError() == hipSuccess ? SPLITZIP_OK : SPLITZIP_E_HIP;
}

template <template <int, int, bool> class Launch>
int dispatch(uint32_t dim, int dtype, const RowArgs& r, dim3 grid, hipStream_t stream) {
  return r.rows > 4 ? dispatch_type<Launch, true>(dim, dtype, r, grid, stream)
                    : dispatch_type<Launch, false>(dim, dtype, r, grid, stream);
}

template <int D, int T, bool N>
struct Append {
  static void go(const RowArgs& r, dim3 grid, hipStream_t s) { kv4_append_kernel<D, T, N><<<grid, kRowThreads, 0, s>>>(r); }
};
template <int D, int T, bool N>
struct Read {
  static void go(const RowArgs& r, dim3 grid, hipStream_t s) {
    if constexpr (T != SPLITZIP_FP8_E5M2) kv4_read_kernel<D, T, N><<<grid, kRowThreads, 0, s>>>(r);
  }
};

}  // namespace kv4

extern "C" {

size_t splitzip_kv4_page_bytes(uint32_t head_dim, uint32_t page_tokens) {
  if (!kv4::dim_ok(head_dim) || !kv4::page_ok(page_tokens)) return 0;
  return (size_t)head_dim * page_tokens / 16 * 17;
}

int splitzip_kv4_append(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype, const void* d_k,
                        size_t k_row_stride, size_t k_head_stride, const void* d_v, size_t v_row_stride,
                        size_t v_head_stride, const int32_t* d_positions, float* d_mass, int32_t* d_pos,
                        int32_t* d_status, hipStream_t stream) {
  using namespace kv4;
  if (!cache_ok(cache) || !batch_ok(cache, batch, true)) return SPLITZIP_E_INVALID;
  if (dtype != SPLITZIP_BF16 && dtype != SPLITZIP_KV4_FP16 && dtype != SPLITZIP_FP8_E5M2) return SPLITZIP_E_INVALID;
  const size_t unit = dtype == SPLITZIP_FP8_E5M2 ? 8 : 16;
  if (!al(d_k, unit) || !al(d_v, unit) || ((k_row_stride | k_head_stride | v_row_stride | v_head_stride) & 7) ||
      !al(d_positions, 4) || !al(d_mass, 4) || !al(d_pos, 4) || !al(d_status, 4))
    return SPLITZIP_E_INVALID;
  if (batch->n_rows > 0 && (!d_k || !d_v)) return SPLITZIP_E_INVALID;
  if (batch->n_rows == 0 || batch->n_seqs == 0) return SPLITZIP_OK;
  RowArgs r = {};
  const uint32_t x = row_blocks(cache, batch, &r);
  if (x == 0) return SPLITZIP_E_INVALID;
  r.a = batch_of(cache, batch, d_status);
  r.k = static_cast<const uint8_t*>(d_k);
  r.v = static_cast<const uint8_t*>(d_v);
  r.k_row = k_row_stride;
  r.k_head = k_head_stride;
  r.v_row = v_row_stride;
  r.v_head = v_head_stride;
  r.positions = d_positions;
  r.mass = d_mass;
  r.pos = d_pos;
  return dispatch<Append>(cache->head_dim, dtype, r, dim3(x), stream);
}

int splitzip_kv4_read(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype, void* d_k,
                      void* d_v, int32_t* d_status, hipStream_t stream) {
  using namespace kv4;
  if (!cache_ok(cache) || !batch_ok(cache, batch, true)) return SPLITZIP_E_INVALID;
  if (dtype != SPLITZIP_BF16 && dtype != SPLITZIP_KV4_FP16) return SPLITZIP_E_INVALID;
  if (!al(d_k, 16) || !al(d_v, 16) || !al(d_status, 4)) return SPLITZIP_E_INVALID;
  if (batch->n_rows == 0 || batch->n_seqs == 0 || (!d_k && !d_v)) return SPLITZIP_OK;
  RowArgs r = {};
  const uint32_t x = row_blocks(cache, batch, &r);
  if (x == 0) return SPLITZIP_E_INVALID;
  r.a = batch_of(cache, batch, d_status);
  r.k_out = static_cast<uint8_t*>(d_k);
  r.v_out = static_cast<uint8_t*>(d_v);
  return dispatch<Read>(cache->head_dim, dtype, r, dim3(x), stream);
}

}  // extern "C"

#endif
