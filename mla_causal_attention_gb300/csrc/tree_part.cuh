// tree_part.cuh -- how the work of the tree attention is shared out between the CTA pairs, for the
// kernel that makes the partition and those that walk through it.
#pragma once
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mla {
namespace tree {

constexpr int kTile = 128;  // keys per tile
constexpr int kRows = 128;  // query rows per unit, 64 per CTA
// What the end of a unit costs -- its mix read out and written, the next one's rows fetched -- in
// tiles: 0, 2, 3, 4, 8 of them give 446, 437, 427, 430, 436 us for ragged batches of trees, 64.7,
// 62.0, 61.8, 61.6, 66.3 for a ragged decode.
constexpr int kEndTiles = 3;

// ---- the partition -----------------------------------------------------------------------
// Sequence b has n_b H rows in M_b units and K_b key tiles.  Units are numbered, and their tiles
// laid end to end, in the order (sequence, unit, key).  Pair c does units c, c + P, c + 2 P, ..
// whole for the first n_w waves of P units: in a wave the pairs walk through the keys of the
// same few sequences at the same time, and find them in L2 (64-token trees on 32768 keys: 1.20 ms;
// all tiles cut into equal ranges, where every pair is at another key, 1.61, and in five rounds
// of such ranges 1.30).  The tiles of the remaining units
// are cut into one contiguous range per pair, each as long as brings the pair's work, with
// kEndTiles for every unit's end, to the common level; n_w is the largest number of waves that leaves every pair at or below it.  A
// range's tiles of one unit are a segment: a unit within one segment is finished there, the
// others leave partial mixes, range c's first segment in slot 2 c, its last, if another, in slot
// 2 c + 1.
struct TreeSeq {
  int q0, n, kv, ctx;
  bool bad;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b) {
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], k = a.kv_len[b];
  TreeSeq s;
  s.q0 = min(max(c0, 0), a.T);
  s.n = min(max(c1, s.q0), a.T) - s.q0;
  s.kv = (int)min((int64_t)max(k, 0), (int64_t)a.max_pages << a.page_shift);
  s.ctx = max(s.kv - s.n, 0);
  s.bad = s.q0 != c0 || s.q0 + s.n != c1 || s.kv != k || s.kv < s.n;
  return s;
}
__device__ __forceinline__ int seq_tiles(const TreeSeq& s) { return (s.kv + kTile - 1) / kTile; }
// Units of a sequence; without keys (a bad length) it has none, and clear_keyless zeroes its rows.
__device__ __forceinline__ int seq_units(const TreeArgs& a, const TreeSeq& s) {
  return s.kv > 0 ? (s.n * a.H + kRows - 1) / kRows : 0;
}

// The last of n ascending values that is <= x (the first is).
template <typename T>
__device__ __forceinline__ int find_last(const T* v, int n, T x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}
// The same by a whole warp, 32 probes at a time.
template <typename T>
__device__ __forceinline__ int find_warp(const T* v, int n, T x, int lane) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at < hi && v[at] <= x);
    lo += (31 - __clz(le | 1u)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// One segment: rows 128 m .. of sequence b's rows, key tiles [k0, k1).
struct Seg {
  int b, m, k0, k1;
  TreeSeq s;
  int slot;  // partial slot, or -1: the unit is finished here
};

// By one block of 256 threads: prefix sums of units and tiles, the waves, the ranges.  Every
// step is a chain of loads, so the searches run in shared memory, several waves at a time (4096
// sequences of one token, 16 heads: 42 us for the launch, 279 with a walk through the sequences in
// the workspace).
// room: shared memory for the sums and tiles of up to kNear sequences; more are read back from
// the workspace.
constexpr int kNear = 8192;
constexpr int kPartSmem = (kNear + 1) * 20;
static __device__ __noinline__ void tree_partition(const TreeArgs& a, uint8_t* room) {
  constexpr int kBatch = 4;  // waves per search
  const bool near = a.B <= kNear;
  int64_t* tile0 = near ? reinterpret_cast<int64_t*>(room) : a.tile0;
  int64_t* unit0 = near ? tile0 + a.B + 1 : a.unit0;
  int* tiles = reinterpret_cast<int*>(unit0 + a.B + 1);  // of a sequence's units, if near
  __shared__ int64_t s_w[8], s_u[8], s_x;
  __shared__ int s_nw;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t W = 0, U = 0;
  int keyless = 0;  // a sequence has new tokens and no keys
  for (int b0 = 0; b0 < a.B; b0 += 256) {
    const int b = b0 + tid;
    int64_t w = 0, u = 0;
    int K = 0;
    bool none = false;
    if (b < a.B) {
      const TreeSeq s = tree_seq(a, b);
      if (s.bad) set_status(a.status, MLA_ERR_KVLEN);
      if (a.draft_mask && s.n > 64) set_status(a.status, MLA_ERR_TREE);
      none = s.n > 0 && s.kv == 0;
      u = seq_units(a, s);
      K = seq_tiles(s);
      w = u * K;
    }
    int64_t inc_w = w, inc_u = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc_w, o);
      const int64_t y = __shfl_up_sync(0xffffffffu, inc_u, o);
      if (lane >= o) {
        inc_w += x;
        inc_u += y;
      }
    }
    if (lane == 31) {
      s_w[warp] = inc_w;
      s_u[warp] = inc_u;
    }
    keyless |= __syncthreads_or(none);
    int64_t before_w = W, before_u = U;
    for (int k = 0; k < 8; ++k) {
      if (k < warp) {
        before_w += s_w[k];
        before_u += s_u[k];
      }
      W += s_w[k];
      U += s_u[k];
    }
    if (b < a.B) {
      a.tile0[b] = before_w + inc_w - w;
      a.unit0[b] = before_u + inc_u - u;
      if (near) {
        tile0[b] = before_w + inc_w - w;
        unit0[b] = before_u + inc_u - u;
        tiles[b] = K;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    tile0[a.B] = a.tile0[a.B] = W;
    unit0[a.B] = a.unit0[a.B] = U;
    s_nw = (int)min(U / a.pairs, (int64_t)0x7fffffff);
  }
  __syncthreads();  // the block reads these back
  // Thread c: how many whole units leave pair c at or below the level; the fewest of all pairs are
  // done.
  const int P = a.pairs;  // at most 256
  const int64_t cost = W + kEndTiles * U, level = (cost + P - 1) / P;
  int top = 1;
  while (top < a.B) top <<= 1;
  const auto tiles_of = [&](int b) { return near ? tiles[b] : seq_tiles(tree_seq(a, b)); };
  // What units i P + c cost for kBatch waves from i on, before `end`.
  const auto wave_costs = [&](int64_t i, int64_t end, int64_t (&c)[kBatch]) {
    int at[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) at[e] = 0;
    for (int step = top >> 1; step > 0; step >>= 1)  // the last sequence that begins at or before
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int q = at[e] + step;
        if (q < a.B && unit0[q] <= (i + e) * P + tid) at[e] = q;
      }
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      c[e] = i + e < end ? tiles_of(at[e]) + kEndTiles : 0;
  };
  int64_t load = 0;
  int nw = tid < P ? s_nw : 0;
  if (tid < P) {
    const int most = nw;
    int64_t c[kBatch];
    bool full = false;
    for (int64_t i = 0; i < most && !full; i += kBatch) {
      wave_costs(i, most, c);
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (!full && load + c[e] > level) {
          full = true;
          nw = (int)min(i + e, (int64_t)most);
        }
        if (!full) load += c[e];
      }
    }
  }
  __syncthreads();  // every thread has read s_nw
  if (tid < P) atomicMin(&s_nw, nw);
  __syncthreads();
  for (int64_t i = s_nw; i < nw; i += kBatch) {
    int64_t c[kBatch];
    wave_costs(i, nw, c);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) load -= c[e];
  }
  nw = s_nw;
  // Ranges, from the first tile behind the whole units on.
  const int64_t need = tid < P ? level - load : 0;
  int64_t inc = need;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_w[warp] = inc;
  if (tid == 0) {  // the cost of the whole units
    const int64_t u = (int64_t)nw * P;
    s_x = cost;
    if (u < U) {
      const int b = find_last(unit0, a.B, u);
      s_x = tile0[b] + (u - unit0[b]) * tiles_of(b) + kEndTiles * u;
    }
  }
  __syncthreads();
  for (int k = 0; k < warp; ++k) inc += s_w[k];
  // The tile at which a running cost is reached.
  const auto tile_at = [&](int64_t x) {
    if (x >= cost) return W;
    int lo = 0, hi = a.B;  // the last sequence whose cost begins at or before x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile0[mid] + kEndTiles * unit0[mid] <= x) lo = mid; else hi = mid;
    }
    const int64_t off = x - (tile0[lo] + kEndTiles * unit0[lo]);
    const int K = tiles_of(lo);
    const int64_t m = off / (K + kEndTiles);
    return tile0[lo] + m * K + min(off - m * (K + kEndTiles), (int64_t)K);
  };
  if (tid == 0) {
    a.range0[P] = W;
    a.range0[P + 1] = nw;
    a.range0[P + 2] = keyless;
  }
  // Each pair's first segment, spelled out: every role of the split kernel starts with one load
  // instead of a search.
  if (tid < P) {
    const int64_t x = tile_at(s_x + inc - need), x1 = tile_at(s_x + inc);
    a.range0[tid] = x;
    Seg g = {};
    g.b = -1;
    if (nw > 0) {
      g.b = find_last(unit0, a.B, (int64_t)tid);
      g.s = tree_seq(a, g.b);
      g.m = (int)(tid - unit0[g.b]);
      g.k1 = seq_tiles(g.s);
      g.slot = -1;
    } else if (x < x1) {
      g.b = find_last(tile0, a.B, x);
      g.s = tree_seq(a, g.b);
      const int K = seq_tiles(g.s);
      const int64_t off = x - tile0[g.b];
      g.m = (int)(off / K);
      g.k0 = (int)(off - (int64_t)g.m * K);
      g.k1 = (int)min((int64_t)K, g.k0 + (x1 - x));
      g.slot = g.k0 == 0 && g.k1 == K ? -1 : 2 * tid;
    }
    int4* rec = a.first + 3 * tid;
    rec[0] = make_int4(g.b, g.m, g.k0, g.k1);
    rec[1] = make_int4(g.s.q0, g.s.n, g.s.kv, g.s.ctx);
    rec[2] = make_int4(g.slot, 0, 0, 0);
  }
}

// ---- the key weights' share ---------------------------------------------------------------
// Key tiles of 256 rows against tiles of 128 query rows: sequence b has P_b R_b steps, in the order
// (sequence, key tile, row tile), and pair c of the P = min(pairs, W) that are used does steps
// [W c / P, W (c + 1) / P).
constexpr int kKeyTile = 256;
__device__ __forceinline__ int key_tiles(const TreeSeq& s) {
  return s.n > 0 ? (s.kv + kKeyTile - 1) / kKeyTile : 0;
}
__device__ __forceinline__ int row_tiles(const TreeArgs& a, const TreeSeq& s) {
  return (s.n * a.H + kRows - 1) / kRows;
}

// Floats that a sequence's scores take if they are kept: rows x whole tiles of 128 keys.  Those of many
// rows are computed again.  Kept and computed again, us: 64 sequences of 4000 keys and 64 rows 88,
// 148; 128 rows 124, 149; 256 rows 210, 230; 16 of 512 rows 121, 119, 8 of 512 rows on 1000 keys 37,
// 47; 4 of 1024 rows 73, 72; one of 4096 rows 119, 72.
__device__ __forceinline__ int64_t store_size(const TreeArgs& a, const TreeSeq& s) {
  const int64_t rows = (int64_t)s.n * a.H;
  return rows <= kKeptRows ? rows * seq_tiles(s) * kTile : 0;
}

// By one block of 256 threads: which sequences' scores are kept; the tiles and steps in front of each
// sequence; the counters cleared.  The store is given out in the order of the sequences.  One that asks for
// more than is left gets nothing and takes nothing from those behind it (63 requests of one token on
// 4000 keys behind one of 8 tokens on 140000: 336 us if it did, 291; in front of it 292).
static __device__ __noinline__ void key_steps(const TreeArgs& a, const KeySteps& k) {
  __shared__ int64_t s_sum[3][8], s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 2 * a.pairs; i += 256) k.count[i] = 0;
  // The sum of x over the threads before this one; all is the block's.
  const auto scan = [&](int64_t x, int which, int64_t& all) {
    int64_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_sum[which][warp] = inc;
    __syncthreads();
    all = 0;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) inc += s_sum[which][i];
      all += s_sum[which][i];
    }
    return inc - x;
  };
  int64_t size = 0, tiles = 0, steps = 0;  // of the sequences before
  for (int b0 = 0; b0 < a.B; b0 += 256) {
    const int b = b0 + tid;
    TreeSeq s = {};
    if (b < a.B) s = tree_seq(a, b);
    const int64_t own = store_size(a, s);
    int64_t all, from;
    bool keep = own > 0;
    for (;;) {
      from = size + scan(keep ? own : 0, 0, all);
      const bool over = keep && from + own > k.room;  // the first that does not fit, and all behind it
      if (over && from <= k.room) s_left = k.room - from;  // the first
      if (!__syncthreads_or(over)) break;
      keep = keep && !(over && own > s_left);  // that one, and whatever is larger than what it found
    }
    size += all;
    const int64_t t = keep ? seq_tiles(s) : 0;
    const int64_t w = keep ? 0 : (int64_t)key_tiles(s) * row_tiles(a, s);
    const int64_t t0 = tiles + scan(t, 1, all);
    tiles += all;
    const int64_t w0 = steps + scan(w, 2, all);
    steps += all;
    if (b < a.B) {
      k.store0[b] = keep ? from : -1;
      k.read0[b] = t0;
      k.step0[b] = w0;
    }
    __syncthreads();
  }
  if (tid == 0) {
    k.read0[a.B] = tiles;
    k.step0[a.B] = steps;
  }
}

// Zeroes the mixes of sequences that have new tokens and no keys: no unit writes them, and the folded
// queries in their place would be taken for mixes.  By `threads` threads of each pair's CTAs.
__device__ __forceinline__ void clear_keyless(const TreeArgs& a, int pair, int thread, int threads) {
  if (a.range0[a.pairs + 2] == 0) return;
  for (int b = pair; b < a.B; b += a.pairs) {
    const TreeSeq s = tree_seq(a, b);
    if (s.kv > 0) continue;
    uint4* rows = reinterpret_cast<uint4*>(a.q_lat + (size_t)s.q0 * a.H * 512);
    for (int64_t i = thread; i < (int64_t)s.n * a.H * 64; i += threads)
      rows[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Walks a pair's segments: its whole units, then its range.  Warp-uniform; every role has its own
// and looks the next segment up while it works on one, since that takes a chain of loads.
struct SegWalk {
  int64_t wave, waves, x, x1, base, next_base;
  int pair, b, K, lane, slot;
  TreeSeq s;
  // The pair's first segment; false if it has none.
  __device__ __forceinline__ bool start(const TreeArgs& a, int pair_id, int lane_id, Seg& g) {
    const int4* rec = a.first + 3 * pair_id;
    const int4 r0 = rec[0], r1 = rec[1], r2 = rec[2];
    pair = pair_id;
    lane = lane_id;
    waves = a.range0[a.pairs + 1];
    x = a.range0[pair];
    x1 = a.range0[pair + 1];
    b = -1;
    g.b = r0.x;
    g.m = r0.y;
    g.k0 = r0.z;
    g.k1 = r0.w;
    g.s.q0 = r1.x;
    g.s.n = r1.y;
    g.s.kv = r1.z;
    g.s.ctx = r1.w;
    g.slot = r2.x;
    wave = 1;
    slot = 2 * pair;
    if (waves == 0) {
      x += g.k1 - g.k0;
      slot = 2 * pair + 1;
    }
    return g.b >= 0;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, Seg& g) {
    if (wave < waves) {
      const int64_t u = wave * a.pairs + pair;
      ++wave;
      g.b = find_warp(a.unit0, a.B, u, lane);
      g.m = (int)(u - a.unit0[g.b]);
      g.s = tree_seq(a, g.b);
      g.k0 = 0;
      g.k1 = seq_tiles(g.s);
      g.slot = -1;
      return true;
    }
    if (x >= x1) return false;
    if (b < 0 || x >= next_base) enter(a, find_warp(a.tile0, a.B, x, lane));
    const int64_t off = x - base;
    g.b = b;
    g.m = (int)(off / K);
    g.k0 = (int)(off - (int64_t)g.m * K);
    g.k1 = (int)min((int64_t)K, g.k0 + (x1 - x));
    g.s = s;
    g.slot = g.k0 == 0 && g.k1 == K ? -1 : slot;
    slot = 2 * pair + 1;
    x += g.k1 - g.k0;
    return true;
  }
  __device__ __forceinline__ void enter(const TreeArgs& a, int seq) {
    b = seq;
    base = a.tile0[b];
    next_base = a.tile0[b + 1];
    s = tree_seq(a, b);
    K = seq_tiles(s);
  }
};

}  // namespace tree
}  // namespace mla
