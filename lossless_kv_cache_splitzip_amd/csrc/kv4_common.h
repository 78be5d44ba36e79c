// Shared by the kernels of the 4-bit KV cache: the page layout, the checks of
// a batch on the host and on the device, and the conversions between E2M1
// codes and wider types (gfx950 has them as instructions: two elements each,
// scaled by a power of two, round to nearest even).
#ifndef SPLITZIP_KV4_COMMON_H
#define SPLITZIP_KV4_COMMON_H

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "splitzip.h"

namespace kv4 {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// grids count sequences and 256s of slots in dimensions of up to 65535
constexpr uint32_t kMaxSeqs = 65535, kMaxHeads = 1024, kMaxLen = 1u << 23, kMaxRows = 1u << 30, kMaxGroup = 64;

inline uint64_t up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

inline bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool dim_ok(uint32_t d) { return d == 64 || d == 128 || d == 256; }
inline bool page_ok(uint32_t p) { return p >= 16 && p <= 256 && (p & (p - 1)) == 0; }

// The cache and the batch as the kernels take them.
struct Batch {
  uint8_t* pages;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int32_t* status;
  uint64_t table_stride;
  uint64_t page_bytes;  // of one head
  uint32_t n_pages, n_heads, n_seqs, max_len, max_new, n_rows;
  uint32_t page_shift;  // log2 page_tokens
};

inline bool cache_ok(const splitzip_kv4_cache* c) {
  return c && c->d_pages && al(c->d_pages, 16) && c->n_pages >= 1 && c->n_pages < (1u << 31) && c->n_heads >= 1 &&
         c->n_heads <= kMaxHeads && dim_ok(c->head_dim) && page_ok(c->page_tokens);
}

inline bool batch_ok(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, bool rows) {
  if (!b || b->n_seqs > kMaxSeqs || b->max_len > kMaxLen) return false;
  if (b->table_stride < up(b->max_len, c->page_tokens) / c->page_tokens || b->table_stride > (1ull << 40)) return false;
  if (!al(b->d_table, 4) || !al(b->d_lens, 4) || !al(b->d_cu, 4)) return false;
  if (b->n_seqs > 0 && (!b->d_lens || (b->max_len > 0 && !b->d_table))) return false;
  if (!rows) return true;
  if (b->n_rows > kMaxRows || b->max_new > b->n_rows || (b->n_rows > 0 && b->max_new == 0)) return false;
  return b->d_cu != nullptr || b->n_rows == b->n_seqs;
}

inline Batch batch_of(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, int32_t* status) {
  Batch a;
  a.pages = static_cast<uint8_t*>(c->d_pages);
  a.table = b->d_table;
  a.lens = b->d_lens;
  a.cu = b->d_cu;
  a.status = status;
  a.table_stride = b->table_stride;
  a.page_bytes = splitzip_kv4_page_bytes(c->head_dim, c->page_tokens);
  a.n_pages = c->n_pages;
  a.n_heads = c->n_heads;
  a.n_seqs = b->n_seqs;
  a.max_len = b->max_len;
  a.max_new = b->max_new;
  a.n_rows = b->n_rows;
  a.page_shift = (uint32_t)__builtin_ctz(c->page_tokens);
  return a;
}

__device__ inline void corrupt(int32_t* status) {
  if (status) __hip_atomic_store(status, SPLITZIP_E_CORRUPT, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A sequence's length and packed rows; ok: all inside the batch's bounds.
struct Seq {
  int32_t len, row0, rows;
  bool ok;
};

__device__ inline Seq seq_from(const Batch& a, int32_t len, int32_t row0, int32_t end) {
  Seq s;
  s.len = len;
  s.row0 = row0;
  s.ok = len >= 0 && len <= (int32_t)a.max_len && row0 >= 0 && end >= row0 && end <= (int32_t)a.n_rows &&
         (uint32_t)(end - row0) <= a.max_new;
  s.rows = s.ok ? end - row0 : 0;
  return s;
}

__device__ inline Seq seq_of(const Batch& a, uint32_t b) {
  return seq_from(a, a.lens[b], a.cu ? a.cu[b] : (int32_t)b, a.cu ? a.cu[b + 1] : (int32_t)b + 1);
}

// Inclusive sums over the 64 lanes, in registers (row shifts, then the last
// lane of 16 and of 32 to those behind).
__device__ inline uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);  // row_shr:2
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);  // row_shr:4
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);  // row_shr:8
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);  // row_bcast:15
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);  // row_bcast:31
  return v;
}

__device__ inline uint32_t wave_last(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }

// The page of table entry i of sequence b.  A number outside the pool is
// reported and becomes page 0 with kBadPage set: to be read in its place
// (results are unspecified then), never written.
constexpr uint32_t kBadPage = 1u << 31;

__device__ inline uint32_t page_of(const Batch& a, uint32_t b, uint32_t i) {
  const uint32_t p = (uint32_t)a.table[b * a.table_stride + i];
  if (p < a.n_pages) return p;
  corrupt(a.status);
  return kBadPage;
}

// Bytes inside one head's part of a page (P tokens, D channels).
template <int D>
struct Layout {
  static constexpr uint32_t kCode = D / 2;    // bytes of a token's codes
  static constexpr uint32_t kScale = D / 32;  // and of its scales
  static __device__ uint32_t v_codes(uint32_t shift) { return kCode << shift; }
  static __device__ uint32_t k_scales(uint32_t shift) { return (2 * kCode) << shift; }
  static __device__ uint32_t v_scales(uint32_t shift) { return (2 * kCode + kScale) << shift; }
  // piece u (D/16 channels, D/32 bytes) of token t's V codes
  static __device__ uint32_t v_piece(uint32_t t, uint32_t u) { return ((t >> 2) * 16 + u) * (D / 8) + (t & 3) * (D / 32); }
  static __device__ uint32_t v_scale(uint32_t t, uint32_t blk) { return ((t >> 2) * kScale + blk) * 4 + (t & 3); }
};

__device__ inline float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

}  // namespace kv4

#endif
