// The 4-bit cache's encoder and decoder (splitzip_kv4_append, splitzip_kv4_read).
//
// A lane holds 8 channels of one token of one head: one wide load, one code
// dword.  Lanes run over 4 tokens first, then over the
// channels, so the stores of a wave fill whole runs of both code sections: V
// codes interleave 4 tokens (kv4_common.h), K codes are a token's row.  A block
// of 32 channels is then 4 lanes, 4 apart in a row of 16, whose largest
// magnitude two row rotations give.  Both kernels move each byte once and are
// bound by memory (or, for single tokens, by the launch).
#ifndef SPLITZIP_KV4_CODEC_H
#define SPLITZIP_KV4_CODEC_H

#include "kv4_common.h"

namespace kv4 {

constexpr int kRowThreads = 256;

struct RowArgs {
  Batch a;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* k_out;
  uint8_t* v_out;
  uint64_t k_row, k_head, v_row, v_head;  // strides in elements
  const int32_t* positions;
  float* mass;
  int32_t* pos;
};

// 8 elements of type T (a splitzip type) as floats, exactly.
template <int T>
__device__ inline void load8(const uint8_t* p, uint64_t elem, float x[8]) {
  if constexpr (T == SPLITZIP_BF16) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p + 2 * elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(q[i] << 16);
      x[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  } else if constexpr (T == SPLITZIP_KV4_FP16) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p + 2 * elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)q[i]);
      x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(q[i] >> 16));
    }
  } else {  // E5M2 is the upper half of an FP16
    const u32x2 q = *reinterpret_cast<const u32x2*>(p + elem);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(((q[i / 4] >> (8 * (i % 4))) & 0xFFu) << 8));
  }
}

// The largest of the 4 lanes 4 apart in this lane's row of 16.
__device__ inline uint32_t max_of_block(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124 /* row_ror:4 */, 0xF, 0xF, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128 /* row_ror:8 */, 0xF, 0xF, false);
  return v > o ? v : o;
}

// Codes of this lane's 8 channels and the scale byte of their block (all 4
// lanes of a block take part).  Magnitudes compare as integers.
__device__ inline uint32_t encode8(float x[8], uint32_t& scale, bool& odd) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    if (m >= 0x7F800000u) {
      odd = true;
      if (m > 0x7F800000u) x[i] = 0.0f;
    } else {
      top = m > top ? m : top;
    }
  }
  top = max_of_block(top);
  // the least e with max < 7 * 2^e: 7/4 of a power of two is the border
  int s = (int)(top >> 23) - 2 + ((top & 0x7FFFFFu) >= 0x600000u ? 1 : 0);
  s = s < 1 ? 1 : s > 252 ? 252 : s;
  scale = (uint32_t)s;
  const float f = scale_of(scale);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], f, 3);
  return c;
}

// Where a lane of the row kernels works: its token, head and 8 channels.
struct Place {
  uint32_t b, slot, head, u;  // u: channels 8u .. 8u + 7
  uint64_t row;               // packed row
  uint8_t* base;              // the head's bytes in the slot's page
  uint32_t t;                 // slot in the page
  uint32_t page;
  bool on;  // false: nothing to do, or a page number outside the pool
};

// The sequence of a packed row: the first whose rows end behind it.  64
// sequences are looked at in one round of loads; the rows of a wave differ by
// 3 at most, so one vote a row.
__device__ inline uint32_t seq_of_row(const Batch& a, uint32_t row0, uint32_t t) {
  if (!a.cu) return row0 + t;
  const uint32_t lane = threadIdx.x & 63;
  uint32_t seq = a.n_seqs;
  for (uint32_t b = 0; b < a.n_seqs; b += 64) {
    const int32_t end = b + lane < a.n_seqs ? a.cu[b + lane + 1] : 0;
    uint32_t mine = a.n_seqs;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint64_t hit = __ballot(b + lane < a.n_seqs && end > (int32_t)(row0 + k));
      if (k == t && hit) mine = b + (uint32_t)__builtin_ctzll(hit);
    }
    if (mine < seq) seq = mine;
    if (__all(seq < a.n_seqs)) break;
  }
  return seq;
}

// Work item w: 4 packed rows, a head, 8 channels: D / 2 lanes for a head's 4
// rows, rows fastest.  V codes keep 4 slots together, so rows that start at a
// multiple of 4 fill whole words of 16 bytes, others two parts of them.  The
// grid goes by the rows alone, whatever the batch's raggedness.
template <int D>
__device__ inline Place place_of(const Batch& a, uint64_t w) {
  Place p;
  constexpr uint32_t kLanes = D / 2;
  const uint32_t gh = (uint32_t)(w / kLanes), lane = (uint32_t)(w % kLanes), t = lane & 3;
  const uint32_t row0 = gh / a.n_heads * 4;
  p.head = gh % a.n_heads;
  p.u = lane >> 2;
  p.row = row0 + t;
  p.on = false;
  // a wave's lanes may be of two heads (D = 64), of one group of rows unless the heads end: take the first lane's
  const uint32_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)row0);
  uint32_t b = seq_of_row(a, first, t);
  if (__any(row0 != first)) {
    const uint32_t last = (uint32_t)__builtin_amdgcn_readlane((int)row0, 63);
    const uint32_t b2 = seq_of_row(a, last, t);
    if (row0 != first) b = b2;
  }
  if (p.row >= a.n_rows || b >= a.n_seqs) return p;
  const Seq s = seq_of(a, b);
  if (!s.ok || s.rows > s.len || p.row < (uint32_t)s.row0 || p.row >= (uint32_t)(s.row0 + s.rows)) return p;
  p.b = b;
  p.slot = (uint32_t)(s.len - s.rows) + (uint32_t)(p.row - s.row0);
  p.page = page_of(a, b, p.slot >> a.page_shift);
  p.on = p.page != kBadPage;
  if (!p.on) return p;
  p.t = p.slot & ((1u << a.page_shift) - 1);
  p.base = a.pages + ((uint64_t)p.page * a.n_heads + p.head) * a.page_bytes;
  return p;
}

// Reports sequences out of bounds: the last workgroup's job, as a bad one may
// have no row that finds it.
__device__ inline void report_bad(const Batch& a) {
  if (blockIdx.x != gridDim.x - 1 || !a.status) return;
  for (uint32_t b = threadIdx.x; b < a.n_seqs; b += kRowThreads) {
    const Seq s = seq_of(a, b);
    if (!s.ok || s.rows > s.len) corrupt(a.status);
  }
}

template <int D, int T>
__global__ __launch_bounds__(kRowThreads) void kv4_append_kernel(RowArgs r) {
  using L = Layout<D>;
  const Batch& a = r.a;
  report_bad(a);
  const Place p = place_of<D>(a, (uint64_t)blockIdx.x * kRowThreads + threadIdx.x);
  const bool on = p.on;
  float x[8] = {}, y[8] = {};
  if (on) {
    load8<T>(r.k, p.row * r.k_row + p.head * r.k_head + 8 * p.u, x);
    load8<T>(r.v, p.row * r.v_row + p.head * r.v_head + 8 * p.u, y);
  }
  uint32_t ks, vs;
  bool odd = false;
  // a lane that is off still lends its (empty) maximum to no other token's block: lanes of a block share the token
  const uint32_t kc = encode8(x, ks, odd), vc = encode8(y, vs, odd);
  if (!on) return;
  const uint32_t sh = a.page_shift;
  *reinterpret_cast<uint32_t*>(p.base + p.t * L::kCode + 4 * p.u) = kc;
  uint8_t* v = p.base + L::v_codes(sh);
  if constexpr (D == 64) {  // 8 channels are two pieces of 2 bytes
    *reinterpret_cast<uint16_t*>(v + L::v_piece(p.t, 2 * p.u)) = (uint16_t)vc;
    *reinterpret_cast<uint16_t*>(v + L::v_piece(p.t, 2 * p.u + 1)) = (uint16_t)(vc >> 16);
  } else if constexpr (D == 128) {
    *reinterpret_cast<uint32_t*>(v + L::v_piece(p.t, p.u)) = vc;
  } else {  // half a piece of 8 bytes
    *reinterpret_cast<uint32_t*>(v + L::v_piece(p.t, p.u >> 1) + 4 * (p.u & 1)) = vc;
  }
  if ((p.u & 3) == 0) {
    p.base[L::k_scales(sh) + p.t * L::kScale + p.u / 4] = (uint8_t)ks;
    p.base[L::v_scales(sh) + L::v_scale(p.t, p.u / 4)] = (uint8_t)vs;
  }
  if (p.u == 0) {
    const uint64_t at = (((uint64_t)p.page * a.n_heads + p.head) << sh) + p.t;
    if (r.mass) r.mass[at] = 0.0f;
    if (r.pos) r.pos[at] = r.positions ? r.positions[p.row] : (int32_t)p.slot;
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

template <int D, int T>
__global__ __launch_bounds__(kRowThreads) void kv4_read_kernel(RowArgs r) {
  using L = Layout<D>;
  const Batch& a = r.a;
  report_bad(a);
  const Place p = place_of<D>(a, (uint64_t)blockIdx.x * kRowThreads + threadIdx.x);
  if (!p.on) return;
  const uint32_t sh = a.page_shift;
  const uint64_t at = (p.row * a.n_heads + p.head) * D + 8 * p.u;
  if (r.k_out) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(p.base + p.t * L::kCode + 4 * p.u);
    const uint32_t s = p.base[L::k_scales(sh) + p.t * L::kScale + p.u / 4];
    *reinterpret_cast<u32x4*>(r.k_out + 2 * at) = decode8<T>(c, s);
  }
  if (r.v_out) {
    const uint8_t* v = p.base + L::v_codes(sh);
    uint32_t c;
    if constexpr (D == 64) {
      c = *reinterpret_cast<const uint16_t*>(v + L::v_piece(p.t, 2 * p.u)) |
          (uint32_t) * reinterpret_cast<const uint16_t*>(v + L::v_piece(p.t, 2 * p.u + 1)) << 16;
    } else if constexpr (D == 128) {
      c = *reinterpret_cast<const uint32_t*>(v + L::v_piece(p.t, p.u));
    } else {
      c = *reinterpret_cast<const uint32_t*>(v + L::v_piece(p.t, p.u >> 1) + 4 * (p.u & 1));
    }
    const uint32_t s = p.base[L::v_scales(sh) + L::v_scale(p.t, p.u / 4)];
    *reinterpret_cast<u32x4*>(r.v_out + 2 * at) = decode8<T>(c, s);
  }
}

// Workgroups for all packed rows; 0 beyond 2^24.
inline uint32_t row_blocks(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b) {
  const uint64_t groups = ((uint64_t)b->n_rows + 3) / 4;
  const uint64_t n = up(groups * c->n_heads * (c->head_dim / 2), kRowThreads) / kRowThreads;
  return n < (1ull << 24) ? (uint32_t)n : 0;
}

template <template <int, int> class Launch>
int dispatch(uint32_t dim, int dtype, bool e5m2, const RowArgs& r, dim3 grid, hipStream_t stream) {
  if (dtype == SPLITZIP_BF16) {
    if (dim == 64) Launch<64, SPLITZIP_BF16>::go(r, grid, stream);
    else if (dim == 128) Launch<128, SPLITZIP_BF16>::go(r, grid, stream);
    else Launch<256, SPLITZIP_BF16>::go(r, grid, stream);
  } else if (dtype == SPLITZIP_KV4_FP16) {
    if (dim == 64) Launch<64, SPLITZIP_KV4_FP16>::go(r, grid, stream);
    else if (dim == 128) Launch<128, SPLITZIP_KV4_FP16>::go(r, grid, stream);
    else Launch<256, SPLITZIP_KV4_FP16>::go(r, grid, stream);
  } else if (e5m2) {
    if (dim == 64) Launch<64, SPLITZIP_FP8_E5M2>::go(r, grid, stream);
    else if (dim == 128) Launch<128, SPLITZIP_FP8_E5M2>::go(r, grid, stream);
    else Launch<256, SPLITZIP_FP8_E5M2>::go(r, grid, stream);
  }
  return hipGetLastError() == hipSuccess ? SPLITZIP_OK : SPLITZIP_E_HIP;
}

template <int D, int T>
struct Append {
  static void go(const RowArgs& r, dim3 grid, hipStream_t s) { kv4_append_kernel<D, T><<<grid, kRowThreads, 0, s>>>(r); }
};
template <int D, int T>
struct Read {
  static void go(const RowArgs& r, dim3 grid, hipStream_t s) {
    if constexpr (T != SPLITZIP_FP8_E5M2) kv4_read_kernel<D, T><<<grid, kRowThreads, 0, s>>>(r);
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
  const uint32_t x = row_blocks(cache, batch);
  if (x == 0) return SPLITZIP_E_INVALID;
  RowArgs r = {};
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
  return dispatch<Append>(cache->head_dim, dtype, true, r, dim3(x), stream);
}

int splitzip_kv4_read(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype, void* d_k,
                      void* d_v, int32_t* d_status, hipStream_t stream) {
  using namespace kv4;
  if (!cache_ok(cache) || !batch_ok(cache, batch, true)) return SPLITZIP_E_INVALID;
  if (dtype != SPLITZIP_BF16 && dtype != SPLITZIP_KV4_FP16) return SPLITZIP_E_INVALID;
  if (!al(d_k, 16) || !al(d_v, 16) || !al(d_status, 4)) return SPLITZIP_E_INVALID;
  if (batch->n_rows == 0 || batch->n_seqs == 0 || (!d_k && !d_v)) return SPLITZIP_OK;
  const uint32_t x = row_blocks(cache, batch);
  if (x == 0) return SPLITZIP_E_INVALID;
  RowArgs r = {};
  r.a = batch_of(cache, batch, d_status);
  r.k_out = static_cast<uint8_t*>(d_k);
  r.v_out = static_cast<uint8_t*>(d_v);
  return dispatch<Read>(cache->head_dim, dtype, false, r, dim3(x), stream);
}

}  // extern "C"

#endif
