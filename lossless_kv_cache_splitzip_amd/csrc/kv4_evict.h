// Eviction from the 4-bit cache by accumulated attention weight
// (splitzip_kv4_evict).
//
// The kept slots are those of the `budget` largest keys: a slot's weight as an
// ordered 32-bit integer, protected slots above all others.  The key of rank
// `budget` is found digit by digit (11, 11 and 10 bits) from counts of the
// digits' values; equal keys are ranked by slot.  Only the holes that eviction
// leaves below the new length are filled, from the kept slots beyond it: the
// call reads 8 bytes a slot and moves as few tokens as can be.
//
// Up to 16384 slots a head is one workgroup's, which keeps the keys in
// registers (kv4_evict_short_kernel); beyond that a head's slots are shared by
// workgroups of 4096 each, in six launches that exchange counts.  A moved token
// costs more than its bytes: its V codes lie in 4-byte pieces between those of
// 3 neighbours, so whole sectors come and go, about 1.1 KB a token.
#ifndef SPLITZIP_KV4_EVICT_H
#define SPLITZIP_KV4_EVICT_H

#include <type_traits>

#include "kv4_common.h"

namespace kv4 {

constexpr uint32_t kMoveThreads = 256;
// One workgroup a head up to this length (16,384 slots, 8 heads: 23 us where the
// long form takes 34, 512 heads 103 and 133; 32 slots a thread at 24,000: 46 and
// 34.5, 295 and 165).
constexpr uint32_t kShortLen = 16384;
// Beyond: 8 consecutive slots a thread (3 x 131,072 slots, 8 heads: 1024 threads of
// 4 slots 111 us, 512 of 8 106, 256 of 16 120, 1024 of 8 117).
constexpr uint32_t kEvThreads = 512, kEvRun = 2;
constexpr uint32_t kChunk = 4 * kEvRun * kEvThreads;
constexpr uint32_t kBins = 2048;
constexpr uint32_t kListed = 1024;           // moves that the short form keeps in LDS and does itself

struct EvArgs {
  Batch a;
  uint32_t budget, sinks, recent, max_moves, chunks;
  const int32_t* next_pos;
  const float* mass;
  const int32_t* pos;
  int32_t* lens_out;
  float* mass_out;
  int32_t* pos_out;
  uint32_t* n_moves;  // [seq][head]
  uint32_t* holes;    // [seq][head][max_moves]
  uint32_t* movers;
  uint32_t* bins;     // [seq][head][3][kBins]
  u32x4* found;       // [seq][head][3]: what the digits up to each say: key, how many of its equals stay, equals
  uint32_t* counts;   // [seq][head][chunks][4]: keys above / equal to the last kept, below / beyond the new length
};

// Weights in ascending order as integers: NaN lowest, both zeros equal.
__device__ inline uint32_t key_of(float w, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sums over the workgroup, one barrier each: the two halves of sh take turns.
template <uint32_t kThreads>
struct Scan {
  uint32_t (*sh)[kThreads / 64];
  uint32_t turn;
  // the values before this thread's, and all of them
  __device__ uint32_t operator()(uint32_t v, uint32_t& all) {
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, x = wave_scan(v);
    uint32_t* to = sh[turn];
    turn ^= 1;
    if (lane == 63) to[wave] = x;
    __syncthreads();
    const uint32_t w = wave_scan(lane < kThreads / 64 ? to[lane] : 0);
    all = wave_last(w);
    return (wave ? (uint32_t)__builtin_amdgcn_readlane((int)w, (int)wave - 1) : 0) + x - v;
  }
};

// The head that a workgroup works for.
struct Unit {
  uint32_t b, head, at;  // at: index of the side arrays [seq][head]
  uint32_t len, left;    // slots before and after; equal: nothing to evict
  int64_t newest;        // positions from here on are protected
  bool ok;
};

__device__ inline Unit unit_of(const EvArgs& e, uint32_t head, uint32_t b) {
  Unit u;
  u.b = b;
  u.head = head;
  u.at = b * e.a.n_heads + head;
  const int32_t len = e.a.lens[b];
  u.ok = len >= 0 && len <= (int32_t)e.a.max_len;
  u.len = u.ok ? (uint32_t)len : 0;
  u.left = min(u.len, e.budget);
  u.newest = (int64_t)e.next_pos[b] - e.recent;
  return u;
}

// Keys of 4 consecutive slots; of those at or beyond the length: `in` unset.
struct Four {
  uint32_t key[4];
  f32x4 mass;
  u32x4 pos;
  uint64_t at;  // index of the side arrays, or kNowhere
  bool in[4];
};
constexpr uint64_t kNowhere = ~0ull;

__device__ inline void load_four(const EvArgs& e, const Unit& u, uint32_t slot, Four& f) {
  const Batch& a = e.a;
  f.at = kNowhere;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f.in[k] = slot + k < u.len;
    f.key[k] = 0;
  }
  f.mass = f32x4{0, 0, 0, 0};
  f.pos = u32x4{0, 0, 0, 0};
  if (!f.in[0]) return;
  const uint32_t page = page_of(a, u.b, slot >> a.page_shift);
  const uint64_t at = (((uint64_t)(page & ~kBadPage) * a.n_heads + u.head) << a.page_shift) + (slot & ((1u << a.page_shift) - 1));
  f.mass = *reinterpret_cast<const f32x4*>(e.mass + at);
  f.pos = *reinterpret_cast<const u32x4*>(e.pos + at);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (f.in[k]) f.key[k] = key_of(f.mass[k], (int32_t)f.pos[k] < (int64_t)e.sinks || (int32_t)f.pos[k] >= u.newest);
  if (page != kBadPage) f.at = at;
}

__device__ constexpr int shift_of(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }

// Counts the keys' digits; keys whose higher digits are not the chosen ones stay out.
__device__ inline void count_four(const Four& f, int pass, uint32_t key, uint32_t* hist) {
  const int shift = shift_of(pass), higher = pass == 0 ? 32 : shift_of(pass - 1);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool on = f.in[k] && (pass == 0 || (f.key[k] >> higher) == (key >> higher));
    const uint32_t d = (f.key[k] >> shift) & (pass == 2 ? 1023u : 2047u);
    if (on) atomicAdd(&hist[d], 1u);  // adding once for lanes that agree: 11.1 us where this takes 8.5
  }
}

struct Chosen {
  uint32_t digit, rest, equal;  // rest: how many of the digit's `equal` keys stay
};

// The digit of the key of rank `want` (1 is the largest) from all counts; out
// is another one for each digit.  kClear: a thread clears what it has read.
template <bool kClear, uint32_t kThreads>
__device__ inline Chosen choose(uint32_t* hist, uint32_t want, Scan<kThreads>& scan, Chosen* out) {
  constexpr uint32_t kMine = kBins / kThreads;
  const uint32_t lowest = kBins - kMine * (threadIdx.x + 1);  // of this thread's digits, the largest being thread 0's
  uint32_t c[kMine], sum = 0, all;
#pragma unroll
  for (uint32_t k = 0; k < kMine; ++k) {
    c[k] = hist[lowest + k];
    if constexpr (kClear) hist[lowest + k] = 0;
    sum += c[k];
  }
  uint32_t before = scan(sum, all);
  if (before < want && want <= before + sum) {
#pragma unroll
    for (int k = kMine - 1; k >= 0; --k) {
      if (before < want && want <= before + c[k]) *out = Chosen{lowest + k, want - before, c[k]};
      before += c[k];
    }
  }
  __syncthreads();
  return *out;
}

// In slot order: which of a thread's 4 kRun consecutive slots stay, given the
// equal keys before them; the holes and the slots that fill them go to their
// lists.
struct Ranks {
  uint32_t equal, hole, mover;  // before these slots
};

template <uint32_t kThreads, uint32_t kRun>
__device__ inline void place_run(const EvArgs& e, const Unit& u, const Four (&f)[kRun], uint32_t slot, uint32_t key,
                                 uint32_t ties, bool all_equal_stay, Ranks& r, uint32_t* holes, uint32_t* movers,
                                 Scan<kThreads>& scan) {
  uint32_t all, rank = 0;
  if (!all_equal_stay) {
    uint32_t n = 0;
#pragma unroll
    for (uint32_t c = 0; c < kRun; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) n += f[c].in[k] && f[c].key[k] == key;
    rank = r.equal + scan(n, all);
    r.equal += all;
  }
  uint32_t keep = 0, hole = 0, mover = 0;  // keep: a bit a slot
#pragma unroll
  for (uint32_t c = 0; c < kRun; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t at = slot + 4 * c + k;
      const bool eq = f[c].key[k] == key, on = f[c].in[k];
      const bool stays = on && (f[c].key[k] > key || (eq && (all_equal_stay || rank < ties)));
      rank += on && eq;
      hole += on && !stays && at < u.left;
      mover += stays && at >= u.left;
      keep |= (uint32_t)stays << (4 * c + k);
    }
  // both counts fit 16 bits: at most 16384 slots
  const uint32_t before = scan(hole | mover << 16, all);
  uint32_t h = r.hole + (before & 0xFFFFu), m = r.mover + (before >> 16);
  r.hole += all & 0xFFFFu;
  r.mover += all >> 16;
  if (hole | mover) {
#pragma unroll
    for (uint32_t c = 0; c < kRun; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t at = slot + 4 * c + k;
        const bool stays = keep >> (4 * c + k) & 1;
        if (f[c].in[k] && !stays && at < u.left) holes[h++] = at;
        if (stays && at >= u.left) movers[m++] = at;
      }
  }
  if (e.mass_out == e.mass && e.pos_out == e.pos) return;
#pragma unroll
  for (uint32_t c = 0; c < kRun; ++c) {
    if (f[c].at == kNowhere) continue;
    if ((keep >> (4 * c) & 15u) == 15u && slot + 4 * c + 4 <= u.left) {  // the usual case: whole words
      if (e.mass_out != e.mass) *reinterpret_cast<f32x4*>(e.mass_out + f[c].at) = f[c].mass;
      if (e.pos_out != e.pos) *reinterpret_cast<u32x4*>(e.pos_out + f[c].at) = f[c].pos;
      continue;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((keep >> (4 * c + k) & 1) && slot + 4 * c + k < u.left) {
        if (e.mass_out != e.mass) e.mass_out[f[c].at + k] = f[c].mass[k];
        if (e.pos_out != e.pos) e.pos_out[f[c].at + k] = (int32_t)f[c].pos[k];
      }
  }
}

// Fills holes i, i + 1, .. of at most kTogether: 16 lanes a token.  Holes lie below the
// new length and their fillers beyond it, so no move touches another's bytes,
// and the tokens' loads are under way together.
constexpr uint32_t kTogether = 4;

template <int D>
__device__ inline void move_some(const EvArgs& e, uint32_t b, uint32_t head, const uint32_t* holes,
                                 const uint32_t* movers, uint32_t i, uint32_t n, uint32_t u) {
  using L = Layout<D>;
  using Piece = std::conditional_t<D == 64, uint16_t, std::conditional_t<D == 128, uint32_t, u32x2>>;
  const Batch& a = e.a;
  const uint32_t sh = a.page_shift, in_page = (1u << sh) - 1;
  uint32_t to[kTogether], from[kTogether], to_page[kTogether], from_page[kTogether];
  bool on[kTogether];
#pragma unroll
  for (uint32_t k = 0; k < kTogether; ++k) {
    const uint32_t m = min(i + k, n - 1);
    to[k] = holes[m];
    from[k] = movers[m];
  }
#pragma unroll
  for (uint32_t k = 0; k < kTogether; ++k) {
    to_page[k] = page_of(a, b, to[k] >> sh);
    from_page[k] = page_of(a, b, from[k] >> sh);
    on[k] = i + k < n && !((to_page[k] | from_page[k]) & kBadPage);
  }
  Piece kc[kTogether], vc[kTogether];
  uint8_t ks[kTogether], vs[kTogether];
  uint32_t side[kTogether];
#pragma unroll
  for (uint32_t k = 0; k < kTogether; ++k) {
    const uint64_t at = (uint64_t)(from_page[k] & ~kBadPage) * a.n_heads + head;
    const uint8_t* p = a.pages + at * a.page_bytes;
    const uint32_t t = from[k] & in_page, blk = u & (L::kScale - 1);
    kc[k] = *reinterpret_cast<const Piece*>(p + t * L::kCode + u * sizeof(Piece));
    vc[k] = *reinterpret_cast<const Piece*>(p + L::v_codes(sh) + L::v_piece(t, u));
    ks[k] = p[L::k_scales(sh) + t * L::kScale + blk];
    vs[k] = p[L::v_scales(sh) + L::v_scale(t, blk)];
    const uint64_t s = (at << sh) + t;
    side[k] = u == 8 ? __float_as_uint(e.mass[s]) : (uint32_t)e.pos[s];
  }
#pragma unroll
  for (uint32_t k = 0; k < kTogether; ++k) {
    if (!on[k]) continue;
    const uint64_t at = (uint64_t)to_page[k] * a.n_heads + head;
    uint8_t* p = a.pages + at * a.page_bytes;
    const uint32_t t = to[k] & in_page;
    *reinterpret_cast<Piece*>(p + t * L::kCode + u * sizeof(Piece)) = kc[k];
    *reinterpret_cast<Piece*>(p + L::v_codes(sh) + L::v_piece(t, u)) = vc[k];
    if (u < L::kScale) {
      p[L::k_scales(sh) + t * L::kScale + u] = ks[k];
      p[L::v_scales(sh) + L::v_scale(t, u)] = vs[k];
    }
    const uint64_t s = (at << sh) + t;
    if (u == 8) e.mass_out[s] = __uint_as_float(side[k]);
    if (u == 9) e.pos_out[s] = (int32_t)side[k];
  }
}

// One workgroup a head, 4 kRun consecutive slots a thread, keys in registers.
// kFused: at most kListed moves, done here too.
template <int D, uint32_t kThreads, uint32_t kRun, bool kFused>
__global__ __launch_bounds__(kThreads) void kv4_evict_short_kernel(EvArgs e) {
  __shared__ uint32_t hist[kBins], sh[2][kThreads / 64];
  __shared__ uint32_t list[2][kFused ? kListed : 1];
  __shared__ Chosen chosen[3];
  const uint32_t tid = threadIdx.x;
  Scan<kThreads> scan = {sh, 0};
  const Unit u = unit_of(e, blockIdx.x, blockIdx.y);
  if (!u.ok && tid == 0) corrupt(e.a.status);
  if (kFused && e.lens_out != e.a.lens && u.head == 0 && tid == 0) e.lens_out[u.b] = u.ok ? (int32_t)u.left : e.a.lens[u.b];
#pragma unroll
  for (uint32_t k = 0; k < kBins; k += kThreads) hist[k + tid] = 0;
  Four f[kRun];
#pragma unroll
  for (uint32_t c = 0; c < kRun; ++c) load_four(e, u, 4 * (kRun * tid + c), f[c]);
  uint32_t key = 0, ties = 0, equal = 0;
  if (u.len > u.left) {
    uint32_t want = u.left;
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
#pragma unroll
      for (uint32_t c = 0; c < kRun; ++c) count_four(f[c], pass, key, hist);
      __syncthreads();
      const Chosen d = choose<true>(hist, want, scan, &chosen[pass]);
      key |= d.digit << shift_of(pass);
      want = d.rest;
      equal = d.equal;
    }
    ties = want;
  }  // else every key is above 0 or equal to it, and all stay
  uint32_t* holes = kFused ? list[0] : e.holes + (uint64_t)u.at * e.max_moves;
  uint32_t* movers = kFused ? list[1] : e.movers + (uint64_t)u.at * e.max_moves;
  Ranks r = {0, 0, 0};
  place_run(e, u, f, 4 * kRun * tid, key, ties, ties == equal, r, holes, movers, scan);
  if constexpr (kFused) {
    __syncthreads();
    for (uint32_t i = kTogether * (tid >> 4); i < r.mover; i += kTogether * (kThreads / 16))
      move_some<D>(e, u.b, u.head, list[0], list[1], i, r.mover, tid & 15);
  } else if (tid == 0) {
    e.n_moves[u.at] = r.mover;
  }
}

__global__ __launch_bounds__(256) void kv4_evict_zero_kernel(u32x4* p, uint64_t n) {
  const uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = u32x4{0, 0, 0, 0};
}

// The key that the passes before `pass` (1, 2, 3) found: what an earlier launch
// wrote down and the last pass's counts.
__device__ inline Chosen key_before(const EvArgs& e, const Unit& u, int pass, Scan<kEvThreads>& scan, Chosen* out) {
  u32x4* found = e.found + (uint64_t)u.at * 3;
  const u32x4 old = pass == 1 ? u32x4{0, u.left, 0, 0} : found[pass - 2];
  const Chosen d = choose<false>(e.bins + ((uint64_t)u.at * 3 + pass - 1) * kBins, old[1], scan, out);
  const uint32_t key = old[0] | d.digit << shift_of(pass - 1);
  if (blockIdx.x == 0 && threadIdx.x == 0) found[pass - 1] = u32x4{key, d.rest, d.equal, 0};
  return Chosen{key, d.rest, d.equal};
}

// Long heads, pass 0, 1, 2: a chunk's digits into the head's counts.  Pass 3:
// the chunk's keys above the last kept one and equal to it.
template <int kPass>
__global__ __launch_bounds__(kEvThreads) void kv4_evict_count_kernel(EvArgs e) {
  __shared__ uint32_t hist[kBins], sh[2][kEvThreads / 64];
  __shared__ Chosen chosen;
  Scan<kEvThreads> scan = {sh, 0};
  const uint32_t tid = threadIdx.x, slot = blockIdx.x * kChunk + 4 * kEvRun * tid;
  const Unit u = unit_of(e, blockIdx.y, blockIdx.z);
  if (kPass == 0 && !u.ok && tid == 0) corrupt(e.a.status);
  if (u.len <= u.left || blockIdx.x * kChunk >= u.len) return;
  Four f[kEvRun];
#pragma unroll
  for (uint32_t c = 0; c < kEvRun; ++c) load_four(e, u, slot + 4 * c, f[c]);
  uint32_t key = 0;
  if constexpr (kPass > 0) key = key_before(e, u, kPass, scan, &chosen).digit;
  if constexpr (kPass < 3) {
#pragma unroll
    for (uint32_t n = 0; n < kBins; n += kEvThreads) hist[n + tid] = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t c = 0; c < kEvRun; ++c) count_four(f[c], kPass, key, hist);
    __syncthreads();
    uint32_t* to = e.bins + ((uint64_t)u.at * 3 + kPass) * kBins;
#pragma unroll
    for (uint32_t k = 0; k < kBins; k += kEvThreads) {
      const uint32_t n = hist[tid + k];
      if (n) __hip_atomic_fetch_add(&to[tid + k], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  } else {
    uint32_t low = 0, high = 0, all_low, all_high;  // above | equal << 16
#pragma unroll
    for (uint32_t c = 0; c < kEvRun; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t n = f[c].in[k] ? (f[c].key[k] > key ? 1u : f[c].key[k] == key ? 1u << 16 : 0u) : 0u;
        if (slot + 4 * c + k < u.left) low += n;
        else high += n;
      }
    scan(low, all_low);
    scan(high, all_high);
    if (tid == 0)
      *reinterpret_cast<u32x4*>(e.counts + ((uint64_t)u.at * e.chunks + blockIdx.x) * 4) =
          u32x4{all_low & 0xFFFFu, all_low >> 16, all_high & 0xFFFFu, all_high >> 16};
  }
}

// Long heads: a chunk's holes and movers into the head's lists, ranked by the
// counts of the chunks before it.
__global__ __launch_bounds__(kEvThreads) void kv4_evict_list_kernel(EvArgs e) {
  __shared__ uint32_t sh[2][kEvThreads / 64];
  Scan<kEvThreads> scan = {sh, 0};
  const uint32_t tid = threadIdx.x, chunk = blockIdx.x, slot = chunk * kChunk + 4 * kEvRun * tid;
  const Unit u = unit_of(e, blockIdx.y, blockIdx.z);
  if (chunk == 0 && tid == 0 && u.len <= u.left) e.n_moves[u.at] = 0;
  if (chunk * kChunk >= u.len) return;
  Four f[kEvRun];
#pragma unroll
  for (uint32_t c = 0; c < kEvRun; ++c) load_four(e, u, slot + 4 * c, f[c]);
  uint32_t key = 0, ties = 0;
  bool all_stay = true;  // all of the last kept key's equals
  Ranks r = {0, 0, 0};
  if (u.len > u.left) {
    const u32x4 found = e.found[(uint64_t)u.at * 3 + 2];
    key = found[0];
    ties = found[1];
    all_stay = ties == found[2];
    const u32x4* counts = reinterpret_cast<const u32x4*>(e.counts + (uint64_t)u.at * e.chunks * 4);
    // equal keys before each earlier chunk decide how many of its own stay: scanned a chunk a thread at a time
    for (uint32_t c0 = 0; c0 < chunk; c0 += kEvThreads) {
      const uint32_t c = c0 + tid;
      const u32x4 n = c < chunk ? counts[c] : u32x4{0, 0, 0, 0};
      uint32_t all;
      const uint32_t before = r.equal + scan(n[1] + n[3], all);
      const uint32_t stay = before >= ties ? 0 : min(ties - before, n[1] + n[3]), stay_low = min(stay, n[1]);
      const uint32_t lows = c < chunk ? min(u.left - min(u.left, c * kChunk), kChunk) : 0;  // slots below the new length
      r.equal += all;
      scan(lows - (n[0] + stay_low), all);
      r.hole += all;
      scan(n[2] + (stay - stay_low), all);
      r.mover += all;
    }
  }
  place_run(e, u, f, slot, key, ties, all_stay, r, e.holes + (uint64_t)u.at * e.max_moves,
             e.movers + (uint64_t)u.at * e.max_moves, scan);
  // the last chunk knows how many there are
  if (u.len > u.left && (chunk + 1) * kChunk >= u.len && tid == 0) e.n_moves[u.at] = r.mover;
}

__device__ inline void write_len(const EvArgs& e, uint32_t b) {
  const int32_t len = e.a.lens[b];
  e.lens_out[b] = len > (int32_t)e.a.max_len || len < 0 || (uint32_t)len <= e.budget ? len : (int32_t)e.budget;
}

// The moves that the lists name, and the new lengths: nothing here reads the old ones.
template <int D>
__global__ __launch_bounds__(kMoveThreads) void kv4_move_kernel(EvArgs e) {
  const uint32_t head = blockIdx.y, b = blockIdx.z, unit = b * e.a.n_heads + head;
  if (blockIdx.x == 0 && head == 0 && threadIdx.x == 0) write_len(e, b);
  const uint32_t n = e.n_moves[unit], step = kTogether * (kMoveThreads / 16);
  for (uint32_t i = blockIdx.x * step + kTogether * (threadIdx.x / 16); i < n; i += gridDim.x * step)
    move_some<D>(e, b, head, e.holes + (uint64_t)unit * e.max_moves, e.movers + (uint64_t)unit * e.max_moves, i, n,
                 threadIdx.x & 15);
}

// New lengths, after every workgroup that reads the old ones has run.
__global__ __launch_bounds__(256) void kv4_lens_kernel(EvArgs e) {
  const uint32_t b = blockIdx.x * 256 + threadIdx.x;
  if (b >= e.a.n_seqs) return;
  write_len(e, b);
}

struct EvPlan {
  uint64_t holes, movers, bins, counts, found, bytes;
  uint32_t max_moves, chunks;
};

inline EvPlan ev_plan(const splitzip_kv4_cache* c, const splitzip_kv4_batch* b, uint32_t budget) {
  EvPlan p;
  const uint64_t units = (uint64_t)b->n_seqs * c->n_heads;
  const uint32_t over = b->max_len > budget ? b->max_len - budget : 0;
  p.max_moves = budget < over ? budget : over;  // holes below the new length, fillers beyond it
  p.chunks = b->max_len > kShortLen ? (b->max_len + kChunk - 1) / kChunk : 0;
  p.holes = up(units * 4, 256);
  p.movers = p.holes + up(units * p.max_moves * 4, 256);
  p.bins = p.movers + up(units * p.max_moves * 4, 256);
  p.counts = p.bins + (p.chunks ? units * 3 * kBins * 4 : 0);
  p.found = p.counts + up(units * p.chunks * 16, 256);
  p.bytes = p.found + (p.chunks ? units * 48 : 0);
  if (p.bytes < 256) p.bytes = 256;
  return p;
}

template <int D, bool kFused>
void evict_short(const EvArgs& e, dim3 heads, hipStream_t stream) {
  const uint32_t n = e.a.max_len;
  // 512 heads of 2049 slots: 18.9 us with 256 threads and 16 slots each, 14.2 with 512 and 8, 13.9 with 1024 and 4
  if (n <= 2048) kv4_evict_short_kernel<D, 512, 1, kFused><<<heads, 512, 0, stream>>>(e);
  else if (n <= 4096) kv4_evict_short_kernel<D, 512, 2, kFused><<<heads, 512, 0, stream>>>(e);
  else if (n <= 8192) kv4_evict_short_kernel<D, 1024, 2, kFused><<<heads, 1024, 0, stream>>>(e);
  else kv4_evict_short_kernel<D, 1024, 4, kFused><<<heads, 1024, 0, stream>>>(e);
}

template <int D>
int evict(const EvArgs& e, const EvPlan& p, hipStream_t stream) {
  const dim3 heads(e.a.n_heads, e.a.n_seqs);
  const bool fused = p.chunks == 0 && p.max_moves <= kListed;
  if (p.chunks == 0) {
    if (fused) evict_short<D, true>(e, heads, stream);
    else evict_short<D, false>(e, heads, stream);
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  } else {
    const uint64_t zeros = (uint64_t)e.a.n_seqs * e.a.n_heads * 3 * kBins / 4;
    kv4_evict_zero_kernel<<<(uint32_t)((zeros + 255) / 256), 256, 0, stream>>>(reinterpret_cast<u32x4*>(e.bins), zeros);
    const dim3 grid(p.chunks, e.a.n_heads, e.a.n_seqs);
    kv4_evict_count_kernel<0><<<grid, kEvThreads, 0, stream>>>(e);
    kv4_evict_count_kernel<1><<<grid, kEvThreads, 0, stream>>>(e);
    kv4_evict_count_kernel<2><<<grid, kEvThreads, 0, stream>>>(e);
    kv4_evict_count_kernel<3><<<grid, kEvThreads, 0, stream>>>(e);
    kv4_evict_list_kernel<<<grid, kEvThreads, 0, stream>>>(e);
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  }
  if (!fused) {
    const uint32_t x = p.max_moves / (kTogether * (kMoveThreads / 16)) + 1;  // a workgroup's moves, once through
    kv4_move_kernel<D><<<dim3(x > 1024 ? 1024 : x, e.a.n_heads, e.a.n_seqs), kMoveThreads, 0, stream>>>(e);
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  } else if (e.lens_out == e.a.lens) {
    kv4_lens_kernel<<<(e.a.n_seqs + 255) / 256, 256, 0, stream>>>(e);
    if (hipGetLastError() != hipSuccess) return SPLITZIP_E_HIP;
  }
  return SPLITZIP_OK;
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
  if (!al(d_next_pos, 4) || !al(d_mass, 16) || !al(d_pos, 16) || !al(d_lens_out, 4) || !al(d_mass_out, 16) ||
      !al(d_pos_out, 16) || !al(d_work, 256) || !al(d_status, 4))
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
  e.chunks = p.chunks;
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
  e.bins = reinterpret_cast<uint32_t*>(w + p.bins);
  e.counts = reinterpret_cast<uint32_t*>(w + p.counts);
  e.found = reinterpret_cast<u32x4*>(w + p.found);
  if (cache->head_dim == 64) return evict<64>(e, p, stream);
  return cache->head_dim == 128 ? evict<128>(e, p, stream) : evict<256>(e, p, stream);
}

}  // extern "C"

#endif
