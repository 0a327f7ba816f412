// key_weights.cu -- the attention weight that each cached key receives, on CTA pairs.
//
// For the new tokens i of a sequence and all heads h, with the scores of the tree attention
//   s_ihj = scale * (q_lat[i,h] . c_j + q_pe[i,h] . k_pe_j)     over the keys j that token i sees,
//   w_j   = sum_{i,h} exp(s_ihj - L_ih),    L_ih = log sum_j exp(s_ihj)
// is added to what the key's slot holds.  Each row's L has to be known before the sum over the rows
// can begin.  Sequence by sequence the scores are kept for it, as long as a store of up to 256 MB has
// room (most of it stays in L2), and computed again for the others: written and read again, 8 bytes per
// row and key take as long as their 2176 operations on the tensor cores, but with few rows it is
// the keys, 1152 bytes each, that are not read twice.
//
// Kernels, each a programmatic dependent launch of the one before:
//   tree_proj_kernel<fold, two>  the queries folded into the latent space (tree_proj.cu), in two bf16
//                                parts: weights are summed in fp32, and 8 bits of mantissa in the
//                                queries would be off by 1e-3 in each weight, two parts are by 1e-5
//   row_stats_kernel             each row's maximum and sum, flash style, by the tree attention's
//                                partition (128 rows against tiles of 128 keys)
//   row_lse_kernel               L of the rows whose keys several pairs shared
//   key_read_kernel              w_j from the scores that were kept
//   key_sum_kernel               w_j of the other sequences: tiles of 256 keys against tiles of 128 rows
//
// What bounds it: 2 * 2 * 1088 operations per row and key (the latent columns twice, once for each
// part), or 1152 bytes per key where a sequence has few rows (decode batch: 374 MB in 68 to 70 of 99 us).
//
// row_stats: the tree attention's scores without its mix.  A pair holds 64 rows of queries in each
//   CTA, 136 KB in the two parts, and streams the keys, 64 per CTA; S = Q K^T, M128 N128, every key
//   sub-tile against both parts.  A sequence of up to 64 rows has 32 in each CTA, 68 KB, which leaves
//   room for 120 KB of keys in flight instead of 72.  Thread = (row, half of the keys), running
//   maximum and sum in registers.
// key_sum: the other way round.  A pair holds 256 keys, 128 per CTA (144 KB), and streams the rows;
//   S^T = K Q^T, M256 N128 (N64 for up to 64 rows), so that a thread has one key and adds up the
//   weights of the tile's rows: no sum crosses threads.  M256 halves what is streamed per
//   operation: each CTA stages only half of the rows, 32 bytes a cycle.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "kernels.h"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tree_part.cuh"

namespace mla {
namespace {

using namespace tree;

constexpr int kLD = 512;         // latent width (kv_lora_rank)
constexpr int kThreads = 256;
constexpr int kSub64 = 64 * 128;    // 64 rows x 64 columns, bf16, 128-byte swizzled
constexpr int kSub128 = 128 * 128;  // 128 rows

struct KeyParams {
  CUtensorMap tm_q64, tm_q32;    // q_lat {1024, T*H}, boxes {64, 64} and {64, 32}
  CUtensorMap tm_qr64, tm_qr32;  // q_pe  {64,  T*H}
  CUtensorMap tm_c;              // c_pages  {512, slots}, boxes {64, min(page, 64)}
  CUtensorMap tm_kr;             // pe_pages {64,  slots}
  KeyWeightsArgs a;
};

// The pool row that holds a key, or the pool's end (read as zeros) where the table holds no page.
__device__ __forceinline__ int key_row(const TreeArgs& a, int b, int kv, int key) {
  if (key >= kv) return 0;  // not loaded
  const int page = a.block_table[(int64_t)b * a.max_pages + (key >> a.page_shift)];
  if (page < 0 || page >= a.num_pages) {
    set_status(a.status, MLA_ERR_PAGE);
    return a.num_pages << a.page_shift;
  }
  return (page << a.page_shift) + (key & ((1 << a.page_shift) - 1));
}
// Boxes of `box` keys that hold one of the first min(left, most) keys.
__device__ __forceinline__ int boxes_of(int left, int most, int box) {
  return (min(max(left, 0), most) + box - 1) / box;
}

// Which of the 64 keys from `key` on a row sees: the bits of the new tokens' mask (or, without
// one, the tokens up to its own), every cached key, none from kv on.
__device__ __forceinline__ uint64_t seen_bits(int key, int ctx, int kv, bool masked, uint64_t mask,
                                              int i) {
  const int left = kv - key;  // keys that exist
  const uint64_t exist = left >= 64 ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1;
  const int off = key - ctx;  // index of the first key among the new tokens
  uint64_t w;
  if (masked) {
    if (off >= 0)
      w = off < 64 ? mask >> off : 0ull;
    else
      w = off <= -64 ? ~0ull : (mask << -off) | ((1ull << -off) - 1);
  } else {
    const int cnt = i + 1 - off;
    w = cnt >= 64 ? ~0ull : cnt <= 0 ? 0ull : (1ull << cnt) - 1;
  }
  return w & exist;
}

// Barrier over the four warps that read the scores; ANDs a predicate across them, so that they leave
// the loops together when one of them gave up waiting.
__device__ __forceinline__ bool readers_and(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n"
      " bar.red.and.pred po, 1, 128, pi;\n selp.u32 %0, 1, 0, po;\n}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]),
                 "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Eight words w[at ..] to p, in one store with an L2 policy if p is aligned.
template <int N>
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[N], int at, bool wide,
                                        uint64_t policy) {
  if (wide) {
    asm volatile(
        "st.global.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(p),
        "r"(w[at]), "r"(w[at + 1]), "r"(w[at + 2]), "r"(w[at + 3]), "r"(w[at + 4]),
        "r"(w[at + 5]), "r"(w[at + 6]), "r"(w[at + 7]), "l"(policy)
        : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[at], w[at + 1], w[at + 2], w[at + 3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[at + 4], w[at + 5], w[at + 6], w[at + 7]);
  }
}

// Whether rows of the store begin with a line of L2.
__device__ __forceinline__ bool kept_lines(const KeyWeightsArgs& a) {
  return (reinterpret_cast<uintptr_t>(a.store) & 127u) == 0;
}

// A CTA leaves once neither it nor its peer has anything in flight into its shared memory.  In the
// regular course every copy and MMA has been waited for by now.  After a wait gave up, copies may
// still be landing: they take microseconds.
__device__ __forceinline__ void leave(volatile int* abort_flag, int warp, uint32_t tbase,
                                      uint32_t cols) {
  __syncwarp();
  if (*abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::pair::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::pair::tmem_dealloc(tbase, cols);
  }
}

// Test build only: a warp of the first pair withholds the arrival that frees its first score tile.  The MMA
// warp's bounded wait for it then gives up, which exercises the timeout report and the unwinding of
// both CTAs.
__device__ __forceinline__ bool withheld(uint32_t t) {
#ifdef MLA_TEST_DROP_S_FREE
  return blockIdx.x == 0 && threadIdx.x == 128 && t == 0;
#else
  return false;
#endif
}

// log2 of a row's sum of weights 2^(s - m), plus m; infinite for a row that sees nothing.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f ? m + log2f(l) : l == 0.f ? INFINITY : l;
}

// ---- each row's maximum and sum ---------------------------------------------------------
namespace stats {

constexpr int kAhead = 1;        // tiles between a tile's L2 prefetch and its loads (2: trees 105 us, 1: 102)
constexpr int kOnceRows = 96;    // up to so many rows a sequence's keys are soon dropped from L2
constexpr int kOffQ = 0;                       // 17 sub-tiles: q_lat's two parts, q_pe
constexpr int kOffK = kOffQ + 17 * kSub64;     // 9 sub-tiles: latent columns, rotary key
constexpr int kGroup = 3 * kSub64;             // what a barrier stands for
constexpr int kMorePlaces = 5;                 // of such groups, two of them behind 32 rows of queries
constexpr int kOffMore = kOffK - 2 * kGroup;
static_assert(kOffMore >= kOffQ + 18 * kSub64 / 2, "64 rows are read at the last 32");
constexpr int kOffRed = kOffK + 9 * kSub64;    // [64 rows] (maximum, sum) of the upper keys
constexpr int kOffBar = kOffRed + 512;
constexpr int kSmem = kOffBar + 256 + 1024;    // + barriers + alignment slack
static_assert(kSmem <= 232448, "shared memory per block");
constexpr uint32_t kTmemCols = 128;            // two score tiles, 64 columns each

// Barriers.  "even": used in the even CTA only (both CTAs arrive there).
struct Bars {
  uint64_t q_full;      // even: the segment's queries landed in both CTAs
  uint64_t q_empty;     // the segment's last score MMA has read them
  uint64_t k_full[kMorePlaces];   // even: three sub-tiles of keys landed in both CTAs
  uint64_t k_empty[kMorePlaces];
  uint64_t s_full[2];   // scores of a tile in TMEM
  uint64_t s_free[2];   // even: the scores have been read (8 warps)
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Rows of a unit in the even CTA, as in the tree attention.
__device__ __forceinline__ int rows_first(const TreeArgs& a, const Seg& g) {
  return g.s.n * a.H - g.m * kRows <= 64 ? 32 : 64;
}

// Places of key groups.  More are of use where HBM is the bound: rows of one unit that fill half of
// it (decode batch 112.5 us -> 109.5).  A half unit next to full ones would run ahead of them,
// who read the same keys (B = 64, 192 rows, 4000 keys: 192 us with three places, 198 with five).
__device__ __forceinline__ int places(const TreeArgs& a, const Seg& g) {
  return g.s.n * a.H <= 64 ? kMorePlaces : 3;
}
__device__ __forceinline__ int place_at(int at) {
  return at < 3 ? kOffK + at * kGroup : kOffMore + (at - 3) * kGroup;
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    row_stats_kernel(const __grid_constant__ KeyParams p) {
  namespace tp = tc::pair;
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sQ = smem + kOffQ;
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort_flag = &bars->abort_flag;
  const TreeArgs& a = p.a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tp::cta_rank();
  const int pair_id = blockIdx.x >> 1;
  int* status = a.status;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 2);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < kMorePlaces; ++i) {
      mbar_init(&bars->k_full[i], 2);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 8);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tp::tmem_alloc(&bars->tmem_base, kTmemCols);
    tp::tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&p.tm_q64);
    prefetch_tmap(&p.tm_qr64);
    prefetch_tmap(&p.tm_c);
    prefetch_tmap(&p.tm_kr);
  }
  tc::fence_before_sync();
  __syncthreads();
  tp::cluster_sync();  // both CTAs' barriers are ready before either signals the other's
  tc::fence_after_sync();
  const uint32_t tbase = bars->tmem_base;
  grid_dep_wait();  // the partition and the folded queries
  SegWalk walk;
  Seg g, after;
  bool more = walk.start(a, pair_id, lane, g);
  const int box = min(1 << a.page_shift, 64);  // keys per TMA box
  const int boxes = 64 / box;                  // boxes per 64 keys
  const int pool = a.num_pages << a.page_shift;

  if (warp == 0) {
    // ================= keys and queries =================
    const uint32_t q_full = tp::even_addr(&bars->q_full);
    const uint32_t k_full = tp::even_addr(&bars->k_full[0]);
    uint32_t phase = 0;  // bit per place
    int ns = 0;          // segments
    bool ok = true;
    for (; ok && more; g = after) {
      const auto look = [&](int tile) {  // lane q: the row of box q of this CTA's half
        return lane < boxes
                   ? key_row(a, g.b, g.s.kv, tile * kTile + 64 * rank + lane * box) : 0;
      };
      int rows_next = look(g.k0);
      // Keys that few units read come from HBM, and are asked into L2 ahead of their loads.  With
      // rows so few that HBM is the bound they are better read once and soon dropped, so
      // that the scores stay (64 sequences of 4000 keys, 16 rows: 81 us -> 72; 64 rows on U[512, 8192]
      // keys: 109 -> 102; 80 rows on 4000: 104.4 -> 101.4; 96: 108.6 -> 107.9; 112: 112.5 -> 113.5; 128
      // rows, bound by their MMAs: 117 -> 118.  With 16 sequences of 8000 keys 112 rows gain too, 65 -> 59).
      const bool once = g.s.n * a.H <= kOnceRows;
      const bool ask = !once && g.s.n * a.H <= kKeptRows;
      const uint64_t policy = once ? l2_policy_evict_first() : l2_policy_evict_normal();
      int ahead = ask && g.k0 + kAhead < g.k1 ? look(g.k0 + kAhead) : 0;
      if (ns > 0) ok = mbar_wait(&bars->q_empty, (ns - 1) & 1, status, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int q_row = g.s.q0 * a.H + g.m * kRows + rows_first(a, g) * rank;
      const int ring = places(a, g);
      const int sub_q = ring == 3 ? kSub64 : kSub64 / 2;
      if (tc::elect_one()) {
        const CUtensorMap* ql = ring == 3 ? &p.tm_q64 : &p.tm_q32;
        tp::arrive_expect_tx(q_full, 17 * sub_q);
#pragma unroll 1
        for (int s = 0; s < 16; ++s) tp::tma_load_3d(sQ + s * sub_q, ql, q_full, 64 * s, q_row, 0);
        tp::tma_load_3d(sQ + 16 * sub_q, ring == 3 ? &p.tm_qr64 : &p.tm_qr32, q_full, 0, q_row, 0);
      }
      __syncwarp();
      ++ns;
      int at = 0;  // place
      for (int k = g.k0; k < g.k1 && ok; ++k) {
        const int rows = rows_next;
        if (k + 1 < g.k1) rows_next = look(k + 1);
        if (k == g.k0) more = walk.next(a, after);
        const int nb = boxes_of(g.s.kv - k * kTile - 64 * rank, 64, box);
        int row[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) row[q] = __shfl_sync(0xffffffffu, rows, q);
#pragma unroll 1
        for (int grp = 0; grp < 3; ++grp) {
          ok = mbar_wait(&bars->k_empty[at], ~(phase >> at) & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (tc::elect_one()) {
            const uint32_t bar = k_full + 8 * at;
            uint8_t* dst = smem + place_at(at);
            const CUtensorMap* last = grp < 2 ? &p.tm_c : &p.tm_kr;
            const int col = 192 * grp;
            tp::arrive_expect_tx(bar, 3 * nb * box * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q < nb) {
                uint8_t* to = dst + q * box * 128;
                tp::tma_load_3d_hint(to, &p.tm_c, bar, col, row[q], 0, policy);
                tp::tma_load_3d_hint(to + kSub64, &p.tm_c, bar, col + 64, row[q], 0, policy);
                tp::tma_load_3d_hint(to + 2 * kSub64, last, bar, grp < 2 ? col + 128 : 0, row[q], 0,
                                     policy);
              }
          }
          __syncwarp();
          phase ^= 1u << at;
          at = at + 1 < ring ? at + 1 : 0;
        }
        if (ask && k + kAhead < g.k1) {
          if (lane < boxes_of(g.s.kv - (k + kAhead) * kTile - 64 * rank, 64, box) && ahead < pool) {
            bulk_prefetch_l2(a.c_pages + (size_t)ahead * kLD, box * kLD * 2);
            bulk_prefetch_l2(a.pe_pages + (size_t)ahead * 64, box * 128);
          }
          if (k + 1 + kAhead < g.k1) ahead = look(k + 1 + kAhead);
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ================= score MMAs =================
    constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, 128, false);
    const uint64_t d_k = tc::smem_desc_sw128(0, 16, 1024);  // K-major
    const uint32_t q_lo = smem_u32(sQ) >> 4;
    uint32_t t = 0;      // tiles over the run
    uint32_t phase = 0;  // bit per place
    int ns = 0;          // segments
    bool ok = true;
    for (; ok && more; g = after) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full, ns & 1, status, abort_flag));
      const int ring = places(a, g);
      const uint32_t sub_q = (ring == 3 ? kSub64 : kSub64 / 2) >> 4;
      int at = 0;
      for (int k = g.k0; k < g.k1 && ok; ++k, ++t) {
        // The score tile to be overwritten, that of tile t - 2, has been read.
        if (t > 1) ok = mbar_wait(&bars->s_free[t & 1], ((t >> 1) - 1) & 1, status, abort_flag);
        const uint32_t d = tbase + (t & 1) * 64;
        const bool last = k + 1 == g.k1;
#pragma unroll 1
        for (int grp = 0; grp < 3; ++grp) {
          ok = ok && mbar_wait(&bars->k_full[at], (phase >> at) & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t k_lo = smem_u32(smem + place_at(at)) >> 4;
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 12; ++kk) {
              const int sub = 3 * grp + (kk >> 2);
              const uint64_t kd = d_k | (uint64_t)(k_lo + (kk >> 2) * (kSub64 >> 4) + (kk & 3) * 2);
              // latent columns against both parts; the rotary key, the ninth, against q_pe
              const uint32_t q_at = q_lo + (sub < 8 ? sub : 16) * sub_q + (kk & 3) * 2;
              tp::mma_ss(d, d_k | (uint64_t)q_at, kd, kIdS, (grp | kk) != 0 ? 1u : 0u);
              if (sub < 8)
                tp::mma_ss(d, d_k | (uint64_t)(q_at + 8 * sub_q), kd, kIdS, 1u);
            }
            tp::commit_both(&bars->k_empty[at]);
            if (grp == 2) {
              if (last) tp::commit_both(&bars->q_empty);
              tp::commit_both(&bars->s_full[t & 1]);
            }
          }
          __syncwarp();
          phase ^= 1u << at;
          at = at + 1 < ring ? at + 1 : 0;
        }
        if (k == g.k0) more = walk.next(a, after);
      }
      ++ns;
    }
    // The releases that no one has waited for have arrived before this CTA leaves.
    if (ok && t > 0) {
      for (int at = 0; at < kMorePlaces; ++at)
        mbar_wait(&bars->k_empty[at], ~(phase >> at) & 1, status, abort_flag);
      mbar_wait(&bars->q_empty, (ns - 1) & 1, status, abort_flag);
    }
  } else if (warp >= 4) {
    // ================= maxima and sums =================
    const int q4 = warp & 3;
    const int half = q4 >> 1;                 // keys 64 half .. of a tile
    const int r = (q4 & 1) * 32 + lane;       // row of this CTA's 64
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    float2* red = reinterpret_cast<float2*>(smem + kOffRed);
    const uint32_t s_free = tp::even_addr(&bars->s_free[0]);
    const float sl2 = a.scale_log2;
    // Scores stay in L2 until they are read; key_read_kernel lifts it again, line by line, so that
    // nothing of it is left behind the call (decode batch 108 us without, 103 with).
    const uint64_t stay = l2_policy_evict_last();
    const bool wide = kept_lines(p.a);
    // What a slot holds, for the merge: first row, rows, whether it is its unit's first segment
    // and its last.  One thread clears the pair's two notes and fills in those of its segments.
    const bool notes = rank == 0 && threadIdx.x == 128;
    if (notes) {
      a.part_note[2 * pair_id] = make_int4(0, 0, 0, 0);
      a.part_note[2 * pair_id + 1] = make_int4(0, 0, 0, 0);
    }
    uint32_t t = 0;
    bool ok = true;
    for (; more; g = after) {
      const int first = rows_first(a, g);
      const int row = g.m * kRows + first * rank + r;  // row of the sequence
      const bool real = r < first && row < g.s.n * a.H;
      const int i = row / a.H;                      // new token
      const bool masked = a.draft_mask != nullptr;
      const uint64_t mask = masked && real ? (uint64_t)a.draft_mask[g.s.q0 + i] : 0ull;
      // Where this thread's scores are kept: [unit][key tile][its rows][128 keys].
      const int64_t kept = real ? p.a.steps.store0[g.b] : -1;
      const int unit_rows = min(kRows, g.s.n * a.H - g.m * kRows);
      float* keep = p.a.store + kept +
                    ((int64_t)g.m * kRows * seq_tiles(g.s) + row - g.m * kRows) * kTile + 64 * half;
      float m = -INFINITY, l = 0.f;
      for (int k = g.k0; k < g.k1; ++k, ++t) {
        ok = ok && mbar_wait(&bars->s_full[t & 1], (t >> 1) & 1, status, abort_flag);
        __syncwarp();
        tc::fence_after_sync();
        uint32_t x[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tc::tmem_ld32(tbase + lane_off + (t & 1) * 64 + c * 32, x[c]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c) pin<32>(x[c]);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0 && !withheld(t)) tp::arrive(s_free + 8 * (t & 1));
        const int key = k * kTile + 64 * half;
        if ((k + 1) * kTile > g.s.ctx) {  // the tile holds new tokens or ends behind the last
          const uint64_t seen = seen_bits(key, g.s.ctx, g.s.kv, masked, mask, i);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t w = (uint32_t)(seen >> (32 * c));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((w >> e) & 1u)) x[c][e] = __float_as_uint(-INFINITY);
          }
        }
        if (kept >= 0) {
          float* to = keep + (int64_t)k * unit_rows * kTile;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(to + 32 * c + e, x[c], e, wide, stay);
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], __uint_as_float(x[c][e]),
                                     __uint_as_float(x[c][e + 1]));
        const float top = fmaxf(m, fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sl2);
        const float mb = top == -INFINITY ? 0.f : top;  // nothing seen yet: weights are 2^-inf = 0
        l *= ex2_approx(m - mb);
        m = top;
        const uint64_t sl2_2 = f2_pack(sl2, sl2), neg_2 = f2_pack(-mb, -mb);
        uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            f2_unpack(ffma2(f2_pack(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), sl2_2,
                            neg_2),
                      p0, p1);
            sum2[(e >> 1) & 3] = fadd2(sum2[(e >> 1) & 3], f2_pack(ex2_approx(p0), ex2_approx(p1)));
          }
        float sa, sb;
        f2_unpack(fadd2(fadd2(sum2[0], sum2[1]), fadd2(sum2[2], sum2[3])), sa, sb);
        l += sa + sb;
      }
      more = walk.next(a, after);
      // The two halves of the keys together.
      if (half) red[r] = make_float2(m, l);
      if (!readers_and(ok)) break;
      if (!half) {
        const float2 o = red[r];
        const float top = fmaxf(m, o.x), mb = top == -INFINITY ? 0.f : top;
        l = l * ex2_approx(m - mb) + o.y * ex2_approx(o.x - mb);
        m = top;
        if (g.slot < 0) {
          if (real) p.a.lse[(size_t)g.s.q0 * a.H + row] = row_lse(m, l);
        } else if (r < first) {
          const size_t at = (size_t)g.slot * kRows + first * rank + r;
          reinterpret_cast<float2*>(a.part_ml)[at] = make_float2(m, l);
        }
      }
      if (g.slot >= 0 && notes)
        a.part_note[g.slot] = make_int4(g.s.q0 * a.H + g.m * kRows,
                                        min(kRows, g.s.n * a.H - g.m * kRows), g.k0 == 0,
                                        g.k1 == seq_tiles(g.s));
      readers_and(true);  // the sums have been read before the next segment's
    }
  }
  leave(abort_flag, warp, tbase, kTmemCols);
}

// L of the rows of units that several pairs shared: a block per slot, a thread per row; blocks of
// slots that no unit begins in end at once.  A unit's segments lie in the slots of successive pairs:
// from the one marked first, each next pair's first slot (pairs without work have empty ones) to the
// one marked last.
__global__ void __launch_bounds__(kRows) row_lse_kernel(const KeyWeightsArgs a) {
  grid_dep_launch();
  __shared__ int4 note[512];
  grid_dep_wait();
  const int slots = 2 * a.t.pairs, s0 = blockIdx.x, r = threadIdx.x;
  const int4 n0 = a.t.part_note[s0];
  if (n0.z == 0) return;
  for (int i = s0 + r; i < slots; i += kRows) note[i] = a.t.part_note[i];
  __syncthreads();
  if (r >= n0.y) return;
  float m = -INFINITY, l = 0.f;
  bool last = false;
  for (int s = s0; !last && s < slots; s = (s | 1) + 1) {
    if (note[s].y == 0) continue;
    last = note[s].w != 0;
    const float2 o = reinterpret_cast<const float2*>(a.t.part_ml)[(size_t)s * kRows + r];
    const float top = fmaxf(m, o.x), mb = top == -INFINITY ? 0.f : top;
    l = l * ex2_approx(m - mb) + o.y * ex2_approx(o.x - mb);
    m = top;
  }
  a.lse[(size_t)n0.x + r] = row_lse(m, l);
}

// The slots of the unit whose rows begin with `row`, in the order of its keys, by a warp; their number,
// 0 if it was not shared.
__device__ __forceinline__ int unit_slots(const KeyWeightsArgs& a, int row, int lane, int16_t* list) {
  const int slots = 2 * a.t.pairs;
  int s0 = -1;
  for (int i = lane; i < slots; i += 32) {
    const int4 n = a.t.part_note[i];
    if (n.z != 0 && n.x == row) s0 = i;
  }
  s0 = __reduce_max_sync(0xffffffffu, s0);
  if (s0 < 0) return 0;
  if (lane == 0) list[0] = (int16_t)s0;
  int n = 1;
  bool last = false;
  for (int s = (s0 | 1) + 1; s < slots && !last; s += 64) {
    const int at = s + 2 * lane;
    const int4 x = at < slots ? a.t.part_note[at] : make_int4(0, 0, 0, 0);
    const uint32_t ends = __ballot_sync(0xffffffffu, x.y != 0 && x.w != 0);
    const uint32_t upto = ends ? (2u << (__ffs(ends) - 1)) - 1 : 0xffffffffu;
    const uint32_t some = __ballot_sync(0xffffffffu, x.y != 0) & upto;
    if ((some >> lane) & 1u) list[n + __popc(some & ((1u << lane) - 1))] = (int16_t)at;
    n += __popc(some);
    last = ends != 0;
  }
  return n;
}

}  // namespace stats

// ---- the sum over the rows, of scores that were kept ------------------------------------
// A block takes tiles of 128 keys; its eight warps share the rows, a lane has four keys.  Bound by
// reading the scores, 4 bytes per row and key, mostly from L2.  kMerge: the blocks work out the L of
// their rows themselves, which saves a kernel between two others; where all rows of a call are no
// more than a sequence's may be (one token on 1000 keys: 19.1 -> 15.5 us on the GPU).
namespace kept {

constexpr int kReadThreads = 256;
constexpr int kDeep = 8;  // rows in flight per warp

template <bool kMerge>
__global__ void __launch_bounds__(kReadThreads) key_read_kernel(const KeyWeightsArgs a) {
  __shared__ float part[8][kTile];
  __shared__ float own_lse[kMerge ? kKeptRows : 1];
  __shared__ int16_t list[kMerge ? kKeptRows / kRows : 1][256];  // slots of the sequence's units
  __shared__ int parts[kMerge ? kKeptRows / kRows : 1];
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  const int64_t tiles = a.steps.read0[a.t.B];
  const float sl2 = a.t.scale_log2;
  const bool lines = kept_lines(a);
  // An equal run of tiles for every block, mostly of one sequence, which it looks up once.
  const int64_t x0 = tiles * blockIdx.x / gridDim.x, x1 = tiles * (blockIdx.x + 1) / gridDim.x;
  int64_t base = 0, next = -1;
  int b = 0, rows = 0, K = 0;
  TreeSeq s = {};
  const float* lse = nullptr;
  const float* store = nullptr;
  for (int64_t x = x0; x < x1; ++x) {
    if (x >= next) {
      b = find_warp(a.steps.read0, a.t.B, x, lane);
      base = a.steps.read0[b];
      next = a.steps.read0[b + 1];
      s = tree_seq(a.t, b);
      rows = s.n * a.t.H;
      K = seq_tiles(s);
      lse = a.lse + (size_t)s.q0 * a.t.H;
      store = a.store + a.steps.store0[b];
      if constexpr (kMerge) {
        __syncthreads();  // the rows' L of the sequence before have been read
        if (warp * kRows < rows) {
          const int n = stats::unit_slots(a, s.q0 * a.t.H + warp * kRows, lane, list[warp]);
          if (lane == 0) parts[warp] = n;
        }
        __syncthreads();
        for (int r = threadIdx.x; r < rows; r += kReadThreads) {
          const int u = r / kRows, n = parts[u];
          const float2* ml = reinterpret_cast<const float2*>(a.t.part_ml) + r % kRows;
          float m = -INFINITY, l = 0.f;
          for (int i = 0; i < n; i += 8) {  // eight partials in flight
            float2 o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[e] = i + e < n ? ml[(size_t)list[u][i + e] * kRows] : make_float2(-INFINITY, 0.f);
            float top = m;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, o[e].x);
            const float mb = top == -INFINITY ? 0.f : top;
            l *= ex2_approx(m - mb);
#pragma unroll
            for (int e = 0; e < 8; ++e) l += o[e].y * ex2_approx(o[e].x - mb);
            m = top;
          }
          own_lse[r] = n > 0 ? row_lse(m, l) : lse[r];
        }
        __syncthreads();
        lse = own_lse;
      }
    }
    const int k = (int)(x - base);
    const int key = k * kTile + (int)threadIdx.x;
    const bool some_hidden = (k + 1) * kTile > s.ctx;  // the tile holds new tokens
    const bool mine = threadIdx.x < kTile && key < s.kv;
    const int slot = mine ? key_row(a.t, b, s.kv, key) : 0;
    const bool writes = mine && slot < a.t.num_pages << a.t.page_shift;
    const float held = writes && key < s.ctx && a.decay != 0.f ? a.weights[slot] : 0.f;
    // Sums in two parts (see key_sum_kernel).
    float total[4] = {}, dropped[4] = {};
    for (int r0 = warp; r0 < rows; r0 += 8 * kDeep) {
      // The 64 rows of a round are in one unit, whose rows of a tile lie together.
      const int m = r0 / kRows, unit_rows = min(kRows, rows - m * kRows);
      const float* from =
          store + ((int64_t)m * kRows * K + (int64_t)k * unit_rows + (r0 - m * kRows)) * kTile +
          4 * lane;
      const float* of = lse + r0;
      float4 v[kDeep];
      float L[kDeep];
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        L[e] = INFINITY;
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + 8 * e < rows) {
          v[e] = __ldcs(reinterpret_cast<const float4*>(from + 8 * e * kTile));
          if (lines && lane % 8 == 0) l2_evict_normal(from + 8 * e * kTile);
          L[e] = of[8 * e];
        }
      }
      // A row that is not there, or that sees nothing (L infinite, its scores -inf), adds 2^-inf = 0.
      float got[4] = {};
#pragma unroll
      for (int e = 0; e < kDeep; ++e) {
        got[0] += ex2_approx(fmaf(v[e].x, sl2, -L[e]));
        got[1] += ex2_approx(fmaf(v[e].y, sl2, -L[e]));
        got[2] += ex2_approx(fmaf(v[e].z, sl2, -L[e]));
        got[3] += ex2_approx(fmaf(v[e].w, sl2, -L[e]));
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float y = got[c] - dropped[c], sum = total[c] + y;
        dropped[c] = (sum - total[c]) - y;
        total[c] = sum;
      }
    }
    if (some_hidden && !(total[0] + total[1] + total[2] + total[3] < INFINITY)) {
      // A row that sees a key that is no number has no L, and 2^(-inf - L) is none either where it hides
      // one of these keys: once more, by the masks.
#pragma unroll
      for (int c = 0; c < 4; ++c) total[c] = dropped[c] = 0.f;
      const bool masked = a.t.draft_mask != nullptr;
#pragma unroll 1
      for (int r = warp; r < rows; r += 8) {
        const int m = r / kRows, unit_rows = min(kRows, rows - m * kRows);
        const float4 v = *reinterpret_cast<const float4*>(
            store + ((int64_t)m * kRows * K + (int64_t)k * unit_rows + (r - m * kRows)) * kTile +
            4 * lane);
        const float x[4] = {v.x, v.y, v.z, v.w};
        const int i = r / a.t.H;  // new token
        const uint64_t mask = masked ? (uint64_t)a.t.draft_mask[s.q0 + i] : 0ull;
        const uint64_t seen = seen_bits(k * kTile + 4 * lane, s.ctx, s.kv, masked, mask, i);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float got = (seen >> c) & 1u ? ex2_approx(fmaf(x[c], sl2, -lse[r])) : 0.f;
          const float y = got - dropped[c], sum = total[c] + y;
          dropped[c] = (sum - total[c]) - y;
          total[c] = sum;
        }
      }
    }
    *reinterpret_cast<float4*>(&part[warp][4 * lane]) =
        make_float4(total[0], total[1], total[2], total[3]);
    __syncthreads();
    if (writes) {
      float got = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) got += part[w][threadIdx.x];
      a.weights[slot] = fmaf(held, a.decay, got);
    }
    __syncthreads();
  }
}

}  // namespace kept

// ---- the sum over the rows --------------------------------------------------------------
namespace sum {

constexpr int kStages = 4;                     // of the rows: a latent sub-tile's two parts
constexpr int kStage = 2 * kSub64;
constexpr int kOffK = 0;                       // 9 sub-tiles of 128 keys
constexpr int kOffQ = kOffK + 9 * kSub128;
constexpr int kOffRow = kOffQ + kStages * kStage;  // [2 step parities][128 rows] RowNote
constexpr int kOffKey = kOffRow + 2 * 128 * 16;    // [2 step parities][128 keys] KeyNote
constexpr int kOffBar = kOffKey + 2 * 128 * 8;
constexpr int kSmem = kOffBar + 256 + 1024;
static_assert(kSmem <= 232448, "shared memory per block");
constexpr uint32_t kTmemCols = 256;            // two score tiles, 128 columns each

struct Bars {
  uint64_t k_full[3];   // even: sub-tiles 3 g .. 3 g + 2 of the segment's keys landed in both CTAs
  uint64_t k_empty[3];  // the segment's last MMA on them is done
  uint64_t q_full[kStages];   // even
  uint64_t q_empty[kStages];
  uint64_t s_full[2];   // scores of a step in TMEM
  uint64_t s_free[2];   // even: the scores have been read (8 warps)
  uint64_t n_full[2];   // a step's notes are written (by warp 3)
  uint64_t n_free[2];   // they have been read (4 warps)
  uint32_t tmem_base;
  int abort_flag;
  int last;             // this CTA's segment was the last of its key tile's
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// What a step's scores are read with, brought by a warp of its own: behind each of them lies a chain
// of loads, and the warps that sum would wait for it (7 of 20 thousand cycles for a segment of one
// step).  One per row (those behind the last count as seeing nothing), and one per key: its slot, or
// -1 where there is nothing to write, and what that goes on from.
struct RowNote {
  float lse;
  int token;
  uint64_t mask;
};
struct KeyNote {
  int slot;
  float held;
};

// Row tiles [r0, r1) of sequence b against its keys 256 k ..
struct KeySeg {
  int b, k, r0, r1, rows, tiles;  // rows of the sequence, tiles of them
  TreeSeq s;
  int64_t x;                      // its first step
};
struct KeyWalk {
  int64_t x, x1, base, next_base;
  int64_t W, P;  // steps in all, and the pairs that have some
  int b, lane;
  TreeSeq s;
  __device__ __forceinline__ void start(const KeyWeightsArgs& a, int pair, int lane_id) {
    W = a.steps.step0[a.t.B];
    P = min((int64_t)a.t.pairs, W);
    x = pair < P ? W * pair / P : W;
    x1 = pair < P ? W * (pair + 1) / P : W;
    next_base = -1;
    lane = lane_id;
  }
  // The pair that does step x.
  __device__ __forceinline__ int pair_of(int64_t step) const {
    int64_t c = step * P / W;
    while (W * (c + 1) / P <= step) ++c;
    while (W * c / P > step) --c;
    return (int)c;
  }
  __device__ __forceinline__ bool next(const KeyWeightsArgs& a, KeySeg& g) {
    if (x >= x1) return false;
    if (x >= next_base) {
      b = find_warp(a.steps.step0, a.t.B, x, lane);
      base = a.steps.step0[b];
      next_base = a.steps.step0[b + 1];
      s = tree_seq(a.t, b);
    }
    g.b = b;
    g.s = s;
    g.rows = s.n * a.t.H;
    g.tiles = row_tiles(a.t, s);
    const int64_t off = x - base;
    g.k = (int)(off / g.tiles);
    g.r0 = (int)(off - (int64_t)g.k * g.tiles);
    g.r1 = (int)min((int64_t)g.tiles, g.r0 + (x1 - x));
    g.x = x;
    x += g.r1 - g.r0;
    return true;
  }
};
// Columns of a row tile's scores: 128, or 64 for up to 64 rows.
__device__ __forceinline__ int columns(const KeySeg& g, int r) {
  return g.rows - r * kRows > 64 ? 128 : 64;
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    key_sum_kernel(const __grid_constant__ KeyParams p) {
  namespace tp = tc::pair;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sK = smem + kOffK;
  uint8_t* sQ = smem + kOffQ;
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int* abort_flag = &bars->abort_flag;
  const TreeArgs& a = p.a.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tp::cta_rank();
  const int pair_id = blockIdx.x >> 1;
  int* status = a.status;
  grid_dep_wait();  // the rows' sums, and with them the partition and the folded queries
  if (p.a.steps.step0[a.B] == 0) return;  // everything was kept

  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bars->k_full[i], 2);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars->q_full[i], 2);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 8);
      mbar_init(&bars->n_full[i], 1);
      mbar_init(&bars->n_free[i], 4);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tp::tmem_alloc(&bars->tmem_base, kTmemCols);
    tp::tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&p.tm_q64);
    prefetch_tmap(&p.tm_qr64);
    prefetch_tmap(&p.tm_q32);
    prefetch_tmap(&p.tm_qr32);
    prefetch_tmap(&p.tm_c);
    prefetch_tmap(&p.tm_kr);
  }
  tc::fence_before_sync();
  __syncthreads();
  tp::cluster_sync();  // both CTAs' barriers are ready before either signals the other's
  tc::fence_after_sync();
  const uint32_t tbase = bars->tmem_base;
  // Every role looks its next segment up while it works on one: that takes a chain of loads.
  KeyWalk walk;
  walk.start(p.a, pair_id, lane);
  KeySeg g, after;
  bool more = walk.next(p.a, g);

  if (warp == 0) {
    // ================= keys =================
    const uint32_t k_full = tp::even_addr(&bars->k_full[0]);
    const int box = min(1 << a.page_shift, 64);  // keys per TMA box
    const int boxes = 128 / box;                 // boxes of this CTA's keys, at most 8
    const auto look = [&](const KeySeg& s) {  // lane q: the row of box q of this CTA's keys
      return lane < boxes
                 ? key_row(a, s.b, s.s.kv, s.k * kKeyTile + 128 * rank + lane * box) : 0;
    };
    int ns = 0, steps = 0;  // of the segment before, for all of which its keys are in use
    bool ok = true;
    int next = more ? look(g) : 0;
    for (; ok && more; ++ns, g = after) {
      const uint64_t patience = kWaitLimitNs + (uint64_t)steps * 20000;  // a step takes 2 to 3 us
      steps = g.r1 - g.r0;
      const int nb = boxes_of(g.s.kv - (g.k * kKeyTile + 128 * rank), 128, box);
      int row[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) row[q] = __shfl_sync(0xffffffffu, next, q);
      more = walk.next(p.a, after);
      if (more) next = look(after);
#pragma unroll 1
      for (int grp = 0; grp < 3; ++grp) {
        if (ns > 0) ok = mbar_wait(&bars->k_empty[grp], (ns - 1) & 1, status, abort_flag, patience);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (tc::elect_one()) {
          const uint32_t bar = k_full + 8 * grp;
          uint8_t* dst = sK + 3 * grp * kSub128;
          const CUtensorMap* last = grp < 2 ? &p.tm_c : &p.tm_kr;
          const int col = 192 * grp;
          tp::arrive_expect_tx(bar, 3 * nb * box * 128);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < nb) {
              uint8_t* to = dst + q * box * 128;
              tp::tma_load_3d(to, &p.tm_c, bar, col, row[q], 0);
              tp::tma_load_3d(to + kSub128, &p.tm_c, bar, col + 64, row[q], 0);
              tp::tma_load_3d(to + 2 * kSub128, last, bar, grp < 2 ? col + 128 : 0, row[q], 0);
            }
        }
        __syncwarp();
      }
    }
  } else if (warp == 2) {
    // ================= rows =================
    const uint32_t q_full = tp::even_addr(&bars->q_full[0]);
    uint32_t u = 0;  // stages over the run
    bool ok = true;
    for (; ok && more; g = after) {
      bool then = false;
      for (int r = g.r0; r < g.r1 && ok; ++r) {
        const int half = columns(g, r) / 2;  // rows of this CTA
        const CUtensorMap* tq = half == 64 ? &p.tm_q64 : &p.tm_q32;
        const CUtensorMap* tr = half == 64 ? &p.tm_qr64 : &p.tm_qr32;
        const int row = g.s.q0 * a.H + r * kRows + half * rank;
#pragma unroll 1
        for (int c = 0; c < 9; ++c, ++u) {
          const uint32_t st = u % kStages, n = u / kStages;
          if (n > 0) ok = mbar_wait(&bars->q_empty[st], (n - 1) & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (tc::elect_one()) {
            uint8_t* dst = sQ + st * kStage;
            const uint32_t bar = q_full + 8 * st;
            tp::arrive_expect_tx(bar, (c < 8 ? 2 : 1) * half * 128);
            if (c < 8) {
              tp::tma_load_3d(dst, tq, bar, 64 * c, row, 0);
              tp::tma_load_3d(dst + kSub64, tq, bar, 512 + 64 * c, row, 0);
            } else {
              tp::tma_load_3d(dst, tr, bar, 0, row, 0);
            }
          }
          __syncwarp();
          if (r == g.r0 && c == 0) then = walk.next(p.a, after);
        }
      }
      more = then;
    }
  } else if (warp == 1 && rank == 0) {
    // ================= MMAs =================
    const uint64_t d_k = tc::smem_desc_sw128(0, 16, 1024);  // K-major
    const uint32_t q_lo = smem_u32(sQ) >> 4, k_lo = smem_u32(sK) >> 4;
    uint32_t t = 0, u = 0;  // steps, stages over the run
    int ns = 0;
    bool ok = true;
    for (; ok && more; ++ns, g = after) {
      bool then = false;
      for (int r = g.r0; r < g.r1 && ok; ++r, ++t) {
        // The scores to be overwritten, those of step t - 2, have been read.
        if (t > 1) ok = mbar_wait(&bars->s_free[t & 1], ((t >> 1) - 1) & 1, status, abort_flag);
        const uint32_t d = tbase + (t & 1) * 128;
        const uint32_t idesc = columns(g, r) == 128 ? tc::idesc_bf16_f32(256, 128, false)
                                                    : tc::idesc_bf16_f32(256, 64, false);
#pragma unroll
        for (int c = 0; c < 9; ++c, ++u) {
          const uint32_t st = u % kStages;
          if (r == g.r0 && c % 3 == 0)
            ok = ok && mbar_wait(&bars->k_full[c / 3], ns & 1, status, abort_flag);
          ok = ok && mbar_wait(&bars->q_full[st], (u / kStages) & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint32_t k_at = k_lo + c * (kSub128 >> 4), q_at = q_lo + st * (kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t kd = d_k | (uint64_t)(k_at + 2 * kk);
              tp::mma_ss(d, kd, d_k | (uint64_t)(q_at + 2 * kk), idesc, (c | kk) != 0 ? 1u : 0u);
              if (c < 8)
                tp::mma_ss(d, kd, d_k | (uint64_t)(q_at + (kSub64 >> 4) + 2 * kk), idesc, 1u);
            }
            tp::commit_both(&bars->q_empty[st]);
            if (r + 1 == g.r1 && c % 3 == 2) tp::commit_both(&bars->k_empty[c / 3]);
            if (c == 8) tp::commit_both(&bars->s_full[t & 1]);
          }
          __syncwarp();
        }
        if (r == g.r0) then = walk.next(p.a, after);
      }
      more = then;
    }
    // The releases that no one has waited for have arrived before this CTA leaves.
    if (ok && ns > 0) {
      for (int grp = 0; grp < 3; ++grp)
        mbar_wait(&bars->k_empty[grp], (ns - 1) & 1, status, abort_flag);
      for (uint32_t k = u - kStages; k < u; ++k)
        mbar_wait(&bars->q_empty[k % kStages], (k / kStages) & 1, status, abort_flag);
    }
  } else if (warp == 3) {
    // ================= notes =================
    const bool masked = a.draft_mask != nullptr;
    uint32_t t = 0;
    bool ok = true;
    for (; ok && more; more = walk.next(p.a, g)) {
      for (int r = g.r0; r < g.r1 && ok; ++r, ++t) {
        RowNote row[4];
        KeyNote key[4];
        const bool last = r + 1 == g.r1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = r * kRows + 32 * k + lane;
          row[k] = {INFINITY, 0, 0ull};
          if (at < g.rows) {
            row[k].lse = p.a.lse[(size_t)g.s.q0 * a.H + at];
            row[k].token = at / a.H;
            if (masked) row[k].mask = (uint64_t)a.draft_mask[g.s.q0 + row[k].token];
          }
          if (last) {
            const int j = g.k * kKeyTile + 128 * rank + 32 * k + lane;
            const int slot = j < g.s.kv ? key_row(a, g.b, g.s.kv, j) : -1;
            key[k].slot = slot < a.num_pages << a.page_shift ? slot : -1;
            key[k].held = 0.f;
            if (key[k].slot >= 0 && j < g.s.ctx && p.a.decay != 0.f)
              key[k].held = p.a.weights[key[k].slot];
          }
        }
        if (t > 1) ok = mbar_wait(&bars->n_free[t & 1], ((t >> 1) - 1) & 1, status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        RowNote* rows = reinterpret_cast<RowNote*>(smem + kOffRow) + (t & 1) * 128;
        KeyNote* keys = reinterpret_cast<KeyNote*>(smem + kOffKey) + (t & 1) * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rows[32 * k + lane] = row[k];
          if (last) keys[32 * k + lane] = key[k];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->n_full[t & 1]);
      }
    }
  } else if (warp >= 4) {
    // ================= weights and their sums =================
    const int q4 = warp & 3, tid = threadIdx.x - 128;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t s_free = tp::even_addr(&bars->s_free[0]);
    const float sl2 = a.scale_log2;
    const bool masked = a.draft_mask != nullptr;
    uint32_t t = 0;
    bool ok = true;
    for (; more; g = after) {
      const int off = g.k * kKeyTile + 128 * rank + tid - g.s.ctx;  // index among the new tokens, or < 0
      const bool all_see = __all_sync(0xffffffffu, off < 0);
      const uint32_t bit = off >= 0 && off < 64 ? 1u << (off & 31) : 0u;  // of a mask's upper or lower word
      // Sums in two parts, the running total and what its roundings have dropped: a key's sum goes
      // over up to millions of rows.
      float total = 0.f, dropped = 0.f;
      KeyNote key = {};
      bool then = false;
      for (int r = g.r0; r < g.r1 && ok; ++r, ++t) {
        if (r == g.r0) then = walk.next(p.a, after);
        ok = ok && mbar_wait(&bars->n_full[t & 1], (t >> 1) & 1, status, abort_flag);
        ok = ok && mbar_wait(&bars->s_full[t & 1], (t >> 1) & 1, status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        const RowNote* note = reinterpret_cast<const RowNote*>(smem + kOffRow) + (t & 1) * 128;
        const int cols = columns(g, r);
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t x[32];
          tc::tmem_ld32(tbase + lane_off + (t & 1) * 128 + c, x);
          tc::tmem_wait_ld();
          pin<32>(x);
          if (c + 32 >= cols) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0 && !withheld(t)) tp::arrive(s_free + 8 * (t & 1));
          }
          if (all_see) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float lse = note[c + e].lse;
              const float w = ex2_approx(fmaf(__uint_as_float(x[e]), sl2, -lse));
              part[e & 3] += lse != INFINITY ? w : 0.f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const RowNote row = note[c + e];
              const uint32_t word = off >= 32 ? (uint32_t)(row.mask >> 32) : (uint32_t)row.mask;
              const bool sees = off < 0 || (masked ? (word & bit) != 0 : off <= row.token);
              const float w = ex2_approx(fmaf(__uint_as_float(x[e]), sl2, -row.lse));
              part[e & 3] += sees && row.lse != INFINITY ? w : 0.f;
            }
          }
        }
        if (r + 1 == g.r1) key = (reinterpret_cast<const KeyNote*>(smem + kOffKey) + (t & 1) * 128)[tid];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->n_free[t & 1]);
        const float y = (part[0] + part[1]) + (part[2] + part[3]) - dropped;
        const float sum = total + y;
        dropped = (sum - total) - y;
        total = sum;
      }
      ok = readers_and(ok);  // the four warps leave together: below are barriers between them
      if (!ok) break;
      float got = total;
      bool mine = true;
      if (g.r1 - g.r0 < g.tiles) {
        // The key tile is shared by pairs c0 .. c1: each leaves its sums in a slot, the first that of
        // its last segment (unless it begins with the tile), the others that of their first; the
        // last to come adds them up in order.
        const int64_t x0 = g.x - g.r0;
        const int c0 = walk.pair_of(x0), c1 = walk.pair_of(x0 + g.tiles - 1);
        const int slot0 = walk.W * c0 / walk.P == x0 ? 2 * c0 : 2 * c0 + 1;
        const int at = rank * 128 + tid;
        p.a.part_sum[(size_t)(pair_id == c0 ? slot0 : 2 * pair_id) * kKeyTile + at] = total;
        __threadfence();
        readers_and(true);
        if (tid == 0) bars->last = atomicAdd(p.a.steps.count + 2 * c0 + rank, 1) == c1 - c0;
        readers_and(true);
        mine = bars->last != 0;
        if (mine) {
          __threadfence();
          got = 0.f;
          for (int c = c0; c <= c1; ++c)
            got += __ldcg(p.a.part_sum + (size_t)(c == c0 ? slot0 : 2 * c) * kKeyTile + at);
        }
      }
      if (mine && key.slot >= 0) p.a.weights[key.slot] = fmaf(key.held, p.a.decay, got);
      more = then;
    }
  }
  leave(abort_flag, warp, tbase, kTmemCols);
}

}  // namespace sum

// Tensor maps, cached by pointers and sizes (see tree.cu).
struct MapKey {
  const void* ptr[4];
  int T, H, num_pages, page_shift;
  bool operator==(const MapKey& o) const {
    for (int i = 0; i < 4; ++i)
      if (ptr[i] != o.ptr[i]) return false;
    return T == o.T && H == o.H && num_pages == o.num_pages && page_shift == o.page_shift;
  }
};
struct MapEntry {
  MapKey key;
  CUtensorMap maps[6];
  bool valid;
};
std::mutex g_mu;
MapEntry g_maps[16];
int g_next = 0;

bool key_maps(const TreeArgs& a, KeyParams* p) {
  CUtensorMap* maps[6] = {&p->tm_q64, &p->tm_q32, &p->tm_qr64, &p->tm_qr32, &p->tm_c, &p->tm_kr};
  const MapKey key = {{a.q_lat, a.q_pe, a.c_pages, a.pe_pages}, a.T, a.H, a.num_pages, a.page_shift};
  std::lock_guard<std::mutex> lk(g_mu);
  for (const MapEntry& e : g_maps) {
    if (e.valid && e.key == key) {
      for (int i = 0; i < 6; ++i) *maps[i] = e.maps[i];
      return true;
    }
  }
  const uint64_t rows = (uint64_t)a.T * a.H, slots = (uint64_t)a.num_pages << a.page_shift;
  const uint32_t box = std::min(1 << a.page_shift, 64);
  if (!encode_bf16_3d(&p->tm_q64, a.q_lat, 2 * kLD, rows, 1, rows, 64) ||
      !encode_bf16_3d(&p->tm_q32, a.q_lat, 2 * kLD, rows, 1, rows, 32) ||
      !encode_bf16_3d(&p->tm_qr64, a.q_pe, 64, rows, 1, rows, 64) ||
      !encode_bf16_3d(&p->tm_qr32, a.q_pe, 64, rows, 1, rows, 32) ||
      !encode_bf16_3d(&p->tm_c, a.c_pages, kLD, slots, 1, slots, box) ||
      !encode_bf16_3d(&p->tm_kr, a.pe_pages, 64, slots, 1, slots, box))
    return false;
  MapEntry& e = g_maps[g_next];
  g_next = (g_next + 1) % 16;
  e.key = key;
  for (int i = 0; i < 6; ++i) e.maps[i] = *maps[i];
  e.valid = true;
  return true;
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsArgs& a, cudaStream_t stream) {
  KeyParams p;
  if (!key_maps(a.t, &p)) return cudaErrorInvalidValue;
  p.a = a;
  static std::atomic<uint64_t> attr_done{0};  // bit per device: smem attributes set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(stats::row_stats_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             stats::kSmem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(sum::key_sum_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sum::kSmem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_release);
  }
  e = launch_tree_fold_two(a.t, a.steps, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2 * a.t.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = stats::kSmem;
  e = cudaLaunchKernelEx(&cfg, stats::row_stats_kernel, p);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  if (!a.all_kept) {
    cfg.blockDim = dim3(kRows);
    e = cudaLaunchKernelEx(&cfg, stats::row_lse_kernel, a);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles =  // at most
      (int64_t)a.t.B * ((((int64_t)a.t.max_pages << a.t.page_shift) + kTile - 1) / kTile);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(2 * a.t.pairs * 12, tiles));
  cfg.blockDim = dim3(kept::kReadThreads);
  e = a.all_kept ? cudaLaunchKernelEx(&cfg, kept::key_read_kernel<true>, a)
                 : cudaLaunchKernelEx(&cfg, kept::key_read_kernel<false>, a);
  if (e != cudaSuccess || a.all_kept) return e;
  cfg.gridDim = dim3(2 * a.t.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sum::kSmem;
  return cudaLaunchKernelEx(&cfg, sum::key_sum_kernel, p);
}

}  // namespace mla
