// Eviction from the 4-bit cache by accumulated attention weight
// (splitzip_kv4_evict).
//
// The kept slots are those of the `budget` largest keys: a slot's weight as an
// ordered 32-bit integer, protected slots above all others.  The key of rank
// `budget` is found digit by digit from counts of the digits' values (radix
// selection), equal keys are ranked by slot.  Only the holes that eviction
// leaves below the new length are filled, from the kept slots beyond it: the
// call reads 8 bytes per slot and moves as few tokens as can be.
#ifndef SPLITZIP_KV4_EVICT_H
#define SPLITZIP_KV4_EVICT_H

#include "kv4_common.h"

namespace kv4 {

constexpr uint32_t kEvThreads = 1024;
constexpr uint32_t kMoveThreads = 256;

struct EvArgs {
  Batch a;
  uint32_t budget, sinks, recent, max_moves;
  const int32_t* next_pos;
  const float* mass;
  const int32_t* pos;
  int32_t* lens_out;
  float* mass_out;
  int32_t* pos_out;
  uint32_t* n_moves;  // [seq][head]
  uint32_t* holes;    // [seq][head][max_moves]
  uint32_t* movers;
};

// Weights in ascending order as integers: NaN lowest, both zeros equal.
__device__ inline uint32_t key_of(float w, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the workgroup of the values before this thread's, and all of it.
__device__ inline uint32_t block_scan(uint32_t v, uint32_t* sh, uint32_t& all) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t y = __shfl_up(x, d, 64);
    if (lane >= (uint32_t)d) x += y;
  }
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
  for (uint32_t w = 0; w < kEvThreads / 64; ++w) {
    if (w < wave) before += sh[w];
    all += sh[w];
  }
  __syncthreads();
  return before + x - v;
}

// One workgroup per head of a sequence.
__global__ __launch_bounds__(kEvThreads) void kv4_select_kernel(EvArgs e) {
  __shared__ uint32_t hist[256], sh[kEvThreads / 64];
  __shared__ uint32_t digit, rest;
  const Batch& a = e.a;
  const uint32_t b = blockIdx.y, head = blockIdx.x, tid = threadIdx.x;
  const uint32_t unit = b * a.n_heads + head;
  const int32_t len_in = a.lens[b];
  if (len_in < 0 || len_in > (int32_t)a.max_len) {
    if (tid == 0) {
      corrupt(a.status);
      e.n_moves[unit] = 0;
    }
    return;
  }
  const uint32_t len = (uint32_t)len_in, left = min(len, e.budget);
  const uint32_t in_page = (1u << a.page_shift) - 1;
  const int64_t newest = (int64_t)e.next_pos[b] - e.recent;
  auto at_of = [&](uint32_t i) -> uint64_t {
    return (((uint64_t)page_of(a, b, i >> a.page_shift) * a.n_heads + head) << a.page_shift) + (i & in_page);
  };
  auto key_at = [&](uint32_t i) -> uint32_t {
    const uint64_t at = at_of(i);
    const int32_t p = e.pos[at];
    return key_of(e.mass[at], p < (int64_t)e.sinks || p >= newest);
  };
  // the key of rank `left`, and how many of its equals stay
  uint32_t key = 0, ties = 0;
  if (len > left) {
    uint32_t want = left;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (uint32_t i = tid; i < len; i += kEvThreads) {
        const uint32_t k = key_at(i);
        if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t sum = 0, d = 255;
        for (;; --d) {
          if (sum + hist[d] >= want || d == 0) break;
          sum += hist[d];
        }
        digit = d;
        rest = want - sum;
      }
      __syncthreads();
      key |= digit << shift;
      want = rest;
      __syncthreads();
    }
    ties = want;
  }
  // in slot order: which stay, the holes below the new length, the slots that fill them
  uint32_t equal = 0, n_hole = 0, n_mover = 0;
  for (uint32_t i0 = 0; i0 < len; i0 += kEvThreads) {
    const uint32_t i = i0 + tid;
    const bool in = i < len;
    const uint64_t at = in ? at_of(i) : 0;
    const float w = in ? e.mass[at] : 0.0f;
    const int32_t p = in ? e.pos[at] : 0;
    const uint32_t k = key_of(w, p < (int64_t)e.sinks || p >= newest);
    bool keep = in;
    uint32_t all;
    if (len > left) {
      const bool eq = in && k == key;
      const uint32_t rank = block_scan(eq, sh, all) + equal;
      equal += all;
      keep = in && (k > key || (eq && rank < ties));
      const bool hole = in && !keep && i < left, mover = keep && i >= left;
      const uint32_t h = block_scan(hole, sh, all) + n_hole;
      n_hole += all;
      const uint32_t m = block_scan(mover, sh, all) + n_mover;
      n_mover += all;
      if (hole) e.holes[(uint64_t)unit * e.max_moves + h] = i;
      if (mover) e.movers[(uint64_t)unit * e.max_moves + m] = i;
    }
    if (keep && i < left) {
      if (e.mass_out != e.mass) e.mass_out[at] = w;
      if (e.pos_out != e.pos) e.pos_out[at] = p;
    }
  }
  if (tid == 0) e.n_moves[unit] = n_mover;
}

template <int kBytes>
__device__ inline void copy_piece(uint8_t* to, const uint8_t* from) {
  if constexpr (kBytes == 2) *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(from);
  else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
  else *reinterpret_cast<u32x2*>(to) = *reinterpret_cast<const u32x2*>(from);
}

// Fills the holes: 16 lanes a token.  Holes lie below the new length and
// their fillers beyond it, so no move touches another's bytes.
template <int D>
__global__ __launch_bounds__(kMoveThreads) void kv4_move_kernel(EvArgs e) {
  using L = Layout<D>;
  constexpr int kPiece = D / 32;
  const Batch& a = e.a;
  const uint32_t head = blockIdx.y, b = blockIdx.z, unit = b * a.n_heads + head;
  if (head == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
    const int32_t len = a.lens[b];
    e.lens_out[b] = len > (int32_t)a.max_len || len < (int32_t)e.budget ? len : (int32_t)e.budget;
  }
  const uint32_t n = e.n_moves[unit], u = threadIdx.x & 15, sh = a.page_shift, in_page = (1u << sh) - 1;
  for (uint32_t i = blockIdx.x * (kMoveThreads / 16) + threadIdx.x / 16; i < n; i += gridDim.x * (kMoveThreads / 16)) {
    const uint32_t to = e.holes[(uint64_t)unit * e.max_moves + i], from = e.movers[(uint64_t)unit * e.max_moves + i];
    const uint32_t to_page = (uint32_t)a.table[b * a.table_stride + (to >> sh)];
    const uint32_t from_page = (uint32_t)a.table[b * a.table_stride + (from >> sh)];
    if (to_page >= a.n_pages || from_page >= a.n_pages) continue;  // reported by the selection
    const uint64_t th = (uint64_t)to_page * a.n_heads + head, fh = (uint64_t)from_page * a.n_heads + head;
    const uint32_t tt = to & in_page, ft = from & in_page;
    uint8_t* tp = a.pages + th * a.page_bytes;
    const uint8_t* fp = a.pages + fh * a.page_bytes;
    copy_piece<kPiece>(tp + tt * L::kCode + u * kPiece, fp + ft * L::kCode + u * kPiece);
    copy_piece<kPiece>(tp + L::v_codes(sh) + L::v_piece(tt, u), fp + L::v_codes(sh) + L::v_piece(ft, u));
    if (u < L::kScale) {
      tp[L::k_scales(sh) + tt * L::kScale + u] = fp[L::k_scales(sh) + ft * L::kScale + u];
      tp[L::v_scales(sh) + L::v_scale(tt, u)] = fp[L::v_scales(sh) + L::v_scale(ft, u)];
    }
    if (u == 8) e.mass_out[(th << sh) + tt] = e.mass[(fh << sh) + ft];
    if (u == 9) e.pos_out[(th << sh) + tt] = e.pos[(fh << sh) + ft];
  }
}

struct EvPlan {
  uint64_t holes, movers, bytes;
  uint32_t max_moves;
};

inline EvPlan ev_plan(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, uint32_t budget) {
  EvPlan p;
  const uint64_t units = (uint64_t)b->n_seqs * c->n_heads;
  const uint32_t over = b->max_len > budget ? b->max_len - budget : 0;
  p.max_moves = budget < over ? budget : over;  // holes below the new length, fillers beyond it
  p.holes = up(units * 4, 256);
  p.movers = p.holes + up(units * p.max_moves * 4, 256);
  p.bytes = p.movers + up(units * p.max_moves * 4, 256);
  if (p.bytes < 256) p.bytes = 256;
  return p;
}

}  // namespace kv4

extern "C" {

size_t splitzip_kv4_evict_work_bytes(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch,
                                     uint32_t budget) {
  using namespace kv4;
  if (!cache_ok(cache) || !batch_ok(cache, batch, false) || budget == 0) return 0;
  return ev_plan(cache, batch, budget).bytes;
}

int splitzip_kv4_evict(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, uint32_t budget,
                       uint32_t sinks, uint32_t recent, const int32_t* d_next_pos, const float* d_mass,
                       const int32_t* d_pos, int32_t* d_lens_out, float* d_mass_out, int32_t* d_pos_out, void* d_work,
                       size_t work_bytes, int32_t* d_status, hipStream_t stream) {
  using namespace kv4;
  if (!cache_ok(cache) || !batch_ok(cache, batch, false)) return SPLITZIP_E_INVALID;
  if (budget == 0 || (uint64_t)sinks + recent > budget) return SPLITZIP_E_INVALID;
  if (!al(d_next_pos, 4) || !al(d_mass, 4) || !al(d_pos, 4) || !al(d_lens_out, 4) || !al(d_mass_out, 4) ||
      !al(d_pos_out, 4) || !al(d_work, 256) || !al(d_status, 4))
    return SPLITZIP_E_INVALID;
  if (batch->n_seqs == 0) return SPLITZIP_OK;
  if (!d_next_pos || !d_mass || !d_pos || !d_lens_out || !d_mass_out || !d_pos_out || !d_work) return SPLITZIP_E_INVALID;
  const EvPlan p = ev_plan(cache, batch, budget);
  if (work_bytes < p.bytes) return SPLITZIP_E_CAPACITY;
  EvArgs e = {};
  e.a = batch_of(cache, batch, d_status);
  e.budget = budget;
  e.sinks = sinks;
  e.recent = recent;
  e.max_moves = p.max_moves;
  e.next_pos = d_next_pos;
  e.mass = d_mass;
  e.pos = d_pos;
  e.lens_out = d_lens_out;
  e.mass_out = d_mass_out;
  e.pos_out = d_pos_out;
  uint8_t* w = static_cast<uint8_t*>(d_work);
  e.n_moves = reinterpret_cast<uint32_t*>(w);
  e.holes = reinterpret_cast<uint32_t*>(w + p.holes);
  e.movers = reinterpret_cast<uint32_t*>(w + p.movers);
  kv4_select_kernel<<<dim3(cache->n_heads, batch->n_seqs), kEvThreads, 0, stream>>>(e);
  if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  uint64_t x = (p.max_moves + 63) / 64;  // about 4 moves for each 16 lanes
  x = x < 1 ? 1 : x > 256 ? 256 : x;
  const dim3 grid((uint32_t)x, cache->n_heads, batch->n_seqs);
  if (cache->head_dim == 64) kv4_move_kernel<64><<<grid, kMoveThreads, 0, stream>>>(e);
  else if (cache->head_dim == 128) kv4_move_kernel<128><<<grid, kMoveThreads, 0, stream>>>(e);
  else kv4_move_kernel<256><<<grid, kMoveThreads, 0, stream>>>(e);
  return hipGetLastError() == hipSuccess ? SPLITZIP_OK : SPLITZIP_E_HIP;
}

}  // extern "C"

#endif
