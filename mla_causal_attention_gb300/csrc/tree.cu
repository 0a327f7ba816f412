// tree.cu -- attention of packed new tokens over the paged latent cache, on CTA pairs.
//
// For new token t of sequence b and head h, over the keys j the token sees,
//   s_j = scale * (q_lat[t,h] . c_j + q_pe[t,h] . k_pe_j),   q_lat = W_K[h]^T q_nope
//   out = W_V[h] (sum_j softmax(s)_j c_j)
// (the up-projection kv_b_proj folded into the query and applied once to the mix).  All tokens
// and heads of a sequence read the same latent rows, so its n * H rows of queries form one
// matrix, cut into units of 128 rows, against tiles of 128 keys.
//
// Kernels, each a programmatic dependent launch of the one before:
//   tree_proj_kernel<fold>  q_lat, and the partition of the work (tree_proj.cu)
//   tree_split_kernel       the attention over the latent rows, flash style
//   tree_merge_kernel       partial mixes of the units that several pairs shared (tree_proj.cu)
//   tree_proj_kernel<up>    out = W_V mix (tree_proj.cu)
//
// What bounds it: per row and key 2 * (576 + 512) operations against 1152 bytes per key, read
// once for all rows of a sequence: one token per sequence (64 rows) is bound by HBM, from about
// four tokens on the tensor cores are.  Each unit's mix is 128 rows x 512 columns of fp32, all
// of an SM's TMEM; a pair of CTAs holds 64 rows each instead (256 of the 512 TMEM columns,
// tcgen05 cta_group::2 with M = 128), which leaves room for two score tiles, and each CTA
// stages only its half of the keys (scores) and of the latent columns (mix): 72 KB + 64 KB in
// shared memory beside the queries' 72 KB.  So the next tile's scores run on the tensor cores
// while this tile's softmax is computed.
//
// Rounded to bf16, the type of the MMAs' operands: the folded queries, the softmax weights (their sum
// is taken before), each row's mix, the output.  Scores, maxima, sums and partial mixes are fp32.
//
// Per tile of 128 keys:  S = Q K^T   M128 N128 K576: CTA r stages keys 64 r .. 64 r + 63
//                        O += P C    M128 N256 K128, twice: CTA r stages latent columns
//                                    256 n + 128 r .. + 127 of all 128 keys
// Warps: 0 keys' and queries' TMA, 2 latent columns' TMA, 1 and 3 (even CTA) the MMAs of scores
// and mixes, 4-7 softmax.
// TMEM: S tiles at columns 0 and 64, O blocks n at 128 and 256.  Softmax thread (row r, half g)
// = lane 64 g + r holds the scores of keys 64 g .. 64 g + 63 of its row, and the mix columns
// 256 n + 128 g + c.
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

constexpr int kSubQ = 64 * 128;  // 64 rows x 64 columns, bf16, 128-byte swizzled
constexpr int kSubV = 128 * 128; // 128 keys x 64 columns
constexpr int kThreads = 256;
constexpr int kOffQ = 0;                     // 9 sub-tiles: q_lat columns 0-511, q_pe
constexpr int kOffK = kOffQ + 9 * kSubQ;     // 9 sub-tiles: latent columns 0-511, rotary key
constexpr int kOffV = kOffK + 9 * kSubQ;     // 4 sub-tiles: columns 256 n + 128 r + 64 s
constexpr int kOffP = kOffV + 4 * kSubV;     // weights: 2 sub-tiles of 64 keys
constexpr int kOffRed = kOffP + 2 * kSubQ;   // [2 tile parities][2 halves][64 rows] floats
constexpr int kOffBar = kOffRed + 1024;
constexpr int kSmem = kOffBar + 256 + 1024;  // + barriers + alignment slack
static_assert(kSmem <= 232448, "shared memory per block");
constexpr int kAhead = 2;        // tiles between a tile's L2 prefetch and its loads
constexpr uint32_t kColO = 128;
constexpr float kRescale = 8.0f;  // log2 units: the mix is rescaled when the maximum grows by more

struct TreeParams {
  CUtensorMap tm_q;   // q_lat {512, T*H}, boxes {64, 64}
  CUtensorMap tm_qr;  // q_pe  {64,  T*H}
  CUtensorMap tm_c;   // c_pages  {512, slots}, boxes {64, min(page, 64)}
  CUtensorMap tm_kr;  // pe_pages {64,  slots}
  TreeArgs a;
};

// Barriers.  "even": used in the even CTA only (both CTAs arrive there).
struct TBars {
  uint64_t q_full;      // even: the segment's queries landed in both CTAs
  uint64_t q_empty;     // the segment's last score MMA has read them
  uint64_t k_full[3];   // even: sub-tiles 3 g .. 3 g + 2 of the keys landed in both CTAs
  uint64_t k_empty[3];
  uint64_t v_full[2];   // even: latent columns of block n landed in both CTAs
  uint64_t v_empty;     // block 0's columns read (block 1's: mix_done)
  uint64_t v_tail;      // this CTA's columns of a tile that ends inside, before the zeroing
  uint64_t s_full[2];   // scores of a tile in TMEM
  uint64_t s_free[2];   // even: the scores have been read (8 warps)
  uint64_t p_ready;     // even: weights of a tile written (8 warps)
  uint64_t mix_done;    // the tile's mix added: weights and columns read, O up to date
  uint64_t o_free;      // even: O of the segment read out (8 warps)
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(TBars) <= 256, "barrier block");

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

// Rows of a unit in the even CTA: half of those of a unit that has at most 64 (a sequence with
// one token), so that both CTAs share the writing of its mix, else 64.
__device__ __forceinline__ int rows_first(const TreeArgs& a, const Seg& g) {
  return g.s.n * a.H - g.m * kRows <= 64 ? 32 : 64;
}

// Boxes of `box` keys that hold one of the first min(left, 64) keys.
__device__ __forceinline__ int boxes_of(int left, int box) {
  return (min(max(left, 0), 64) + box - 1) / box;
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

// Barrier over the four softmax warps that ANDs a predicate across them: they leave the loops
// together when one of them gave up waiting.
__device__ __forceinline__ bool softmax_and(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred pi, po;\n setp.ne.u32 pi, %1, 0;\n"
      " bar.red.and.pred po, 1, 128, pi;\n selp.u32 %0, 1, 0, po;\n}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Eight words w[at ..] to p, in one store if the workspace is 32-byte aligned.
template <int N>
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[N], int at, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[at]),
                 "r"(w[at + 1]), "r"(w[at + 2]), "r"(w[at + 3]), "r"(w[at + 4]), "r"(w[at + 5]),
                 "r"(w[at + 6]), "r"(w[at + 7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[at], w[at + 1], w[at + 2], w[at + 3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[at + 4], w[at + 5], w[at + 6], w[at + 7]);
  }
}

template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]),
                 "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    tree_split_kernel(const __grid_constant__ TreeParams p) {
  namespace tp = tc::pair;
  grid_dep_launch();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* sQ = smem + kOffQ;
  uint8_t* sK = smem + kOffK;
  uint8_t* sV = smem + kOffV;
  uint8_t* sP = smem + kOffP;
  TBars* bars = reinterpret_cast<TBars*>(smem + kOffBar);
  volatile int* abort_flag = &bars->abort_flag;
  const TreeArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tp::cta_rank();
  const int pair_id = blockIdx.x >> 1;
  int* status = a.status;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 2);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&bars->k_full[i], 2);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->v_full[i], 2);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 8);
    }
    mbar_init(&bars->v_empty, 1);
    mbar_init(&bars->v_tail, 1);
    mbar_init(&bars->p_ready, 8);
    mbar_init(&bars->mix_done, 1);
    mbar_init(&bars->o_free, 8);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tp::tmem_alloc(&bars->tmem_base, 512);
    tp::tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&p.tm_q);
    prefetch_tmap(&p.tm_qr);
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
    uint32_t t = 0;  // tiles over the run
    int ns = 0;      // segments
    bool ok = true;
    for (; ok && more; g = after) {
      const auto look = [&](int tile) {  // lane q: the row of box q of this CTA's half
        return lane < boxes
                   ? key_row(a, g.b, g.s.kv, tile * kTile + 64 * rank + lane * box) : 0;
      };
      int rows_next = look(g.k0);
      // Where a sequence is a single unit its keys come from HBM, and are asked into L2 two tiles
      // before their loads (ragged decode batch 69.5 -> 65.7 us; 4 tiles 73, 8 tiles 83).  Where
      // several units share them most loads hit L2 anyway, and asking costs more than it
      // brings (64-token trees 1.20 -> 1.30 ms), even if only one of the units asks.
      const bool alone = g.s.n * a.H <= kRows;
      int ahead = alone && g.k0 + kAhead < g.k1 ? look(g.k0 + kAhead) : 0;
      if (ns > 0) ok = mbar_wait(&bars->q_empty, (ns - 1) & 1, status, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int q_row = g.s.q0 * a.H + g.m * kRows + rows_first(a, g) * rank;
      if (tc::elect_one()) {
        tp::arrive_expect_tx(q_full, 9 * kSubQ);
#pragma unroll 1
        for (int s = 0; s < 8; ++s)
          tp::tma_load_3d(sQ + s * kSubQ, &p.tm_q, q_full, 64 * s, q_row, 0);
        tp::tma_load_3d(sQ + 8 * kSubQ, &p.tm_qr, q_full, 0, q_row, 0);
      }
      __syncwarp();
      ++ns;
      for (int k = g.k0; k < g.k1 && ok; ++k, ++t) {
        const int rows = rows_next;
        if (k + 1 < g.k1) rows_next = look(k + 1);
        if (k == g.k0) more = walk.next(a, after);
        const int nb = boxes_of(g.s.kv - k * kTile - 64 * rank, box);
        int row[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) row[q] = __shfl_sync(0xffffffffu, rows, q);
#pragma unroll 1
        for (int grp = 0; grp < 3; ++grp) {
          if (t > 0) ok = mbar_wait(&bars->k_empty[grp], (t - 1) & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (tc::elect_one()) {
            const uint32_t bar = k_full + 8 * grp;
            uint8_t* dst = sK + 3 * grp * kSubQ;
            const CUtensorMap* last = grp < 2 ? &p.tm_c : &p.tm_kr;
            const int col = 192 * grp;
            tp::arrive_expect_tx(bar, 3 * nb * box * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q < nb) {
                uint8_t* to = dst + q * box * 128;
                tp::tma_load_3d(to, &p.tm_c, bar, col, row[q], 0);
                tp::tma_load_3d(to + kSubQ, &p.tm_c, bar, col + 64, row[q], 0);
                tp::tma_load_3d(to + 2 * kSubQ, last, bar, grp < 2 ? col + 128 : 0, row[q], 0);
              }
          }
          __syncwarp();
        }
        if (alone && k + kAhead < g.k1) {
          if (lane < boxes_of(g.s.kv - (k + kAhead) * kTile - 64 * rank, box) && ahead < pool) {
            bulk_prefetch_l2(a.c_pages + (size_t)ahead * kLD, box * kLD * 2);
            bulk_prefetch_l2(a.pe_pages + (size_t)ahead * 64, box * 128);
          }
          if (k + 1 + kAhead < g.k1) ahead = look(k + 1 + kAhead);
        }
      }
    }
  } else if (warp == 2) {
    // ================= latent columns of the mix =================
    const uint32_t v_full = tp::even_addr(&bars->v_full[0]);
    const uint32_t v_tail = smem_u32(&bars->v_tail);
    uint32_t t = 0, tails = 0;
    bool ok = true;
    for (; ok && more; g = after) {
      const auto look = [&](int tile) {  // lane q: the row of box q of the tile
        return lane < 2 * boxes ? key_row(a, g.b, g.s.kv, tile * kTile + lane * box) : 0;
      };
      int rows_next = look(g.k0);
      for (int k = g.k0; k < g.k1; ++k, ++t) {
        const int rows = rows_next;
        if (k + 1 < g.k1) rows_next = look(k + 1);
        if (k == g.k0) more = walk.next(a, after);
        const int left = min(g.s.kv - k * kTile, kTile);  // > 0
        const bool tail = left < kTile;
        if (tail && lane == 0)
          mbar_arrive_expect_tx(&bars->v_tail, 4 * ((left + box - 1) / box) * box * 128);
        int row[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) row[q] = __shfl_sync(0xffffffffu, rows, q);
        const int nb = (left + box - 1) / box;
#pragma unroll 1
        for (int n = 0; n < 2; ++n) {
          if (t > 0)
            ok = mbar_wait(n ? &bars->mix_done : &bars->v_empty, (t - 1) & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (tc::elect_one()) {
            const uint32_t bar = tail ? v_tail : v_full + 8 * n;
            uint8_t* dst = sV + 2 * n * kSubV;
            const int col = 256 * n + 128 * rank;
            if (!tail) tp::arrive_expect_tx(bar, 2 * kSubV);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < nb) {
                tp::tma_load_3d(dst + q * box * 128, &p.tm_c, bar, col, row[q], 0);
                tp::tma_load_3d(dst + kSubV + q * box * 128, &p.tm_c, bar, col + 64, row[q], 0);
              }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (tail) {
          // Rows behind the last key hold whatever the page or an earlier tile held there: their
          // weight is zero, but zero times an infinity is not, so they are cleared.
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->v_tail, tails & 1, status, abort_flag));
          if (!ok) break;
          ++tails;
          for (int i = left * 8 + lane; i < kTile * 8; i += 32)
#pragma unroll
            for (int s = 0; s < 4; ++s)
              *reinterpret_cast<uint4*>(sV + s * kSubV + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tp::arrive(v_full);
            tp::arrive(v_full + 8);
          }
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ================= score MMAs =================
    // Scores and mixes are issued by two warps: waiting for a barrier takes about 170 cycles and
    // issuing an MMA 24, so one warp for both was the slowest part (3600 cycles per tile; the
    // MMAs themselves take 36 x 33.8 + 16 x 64.2 = 2244).
    constexpr uint32_t kIdS = tc::idesc_bf16_f32(128, 128, false);
    const uint64_t d_k = tc::smem_desc_sw128(0, 16, 1024);  // K-major
    const uint32_t q_lo = smem_u32(sQ) >> 4, k_lo = smem_u32(sK) >> 4;
    uint32_t t = 0;  // tiles over the run
    int ns = 0;      // segments
    bool ok = true;
    for (; ok && more; g = after) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full, ns & 1, status, abort_flag));
      for (int k = g.k0; k < g.k1 && ok; ++k, ++t) {
        // The score tile to be overwritten, that of tile t - 2, has been read.
        if (t > 1) ok = mbar_wait(&bars->s_free[t & 1], ((t >> 1) - 1) & 1, status, abort_flag);
        const uint32_t d = tbase + (t & 1) * 64;
        const bool last = k + 1 == g.k1;
#pragma unroll 1
        for (int grp = 0; grp < 3; ++grp) {
          ok = ok && mbar_wait(&bars->k_full[grp], t & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t at = 3 * grp * (kSubQ >> 4);
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 12; ++kk) {
              const uint32_t off = at + (kk >> 2) * (kSubQ >> 4) + (kk & 3) * 2;
              tp::mma_ss(d, d_k | (uint64_t)(q_lo + off), d_k | (uint64_t)(k_lo + off), kIdS,
                         (grp | kk) != 0 ? 1u : 0u);
            }
            tp::commit_both(&bars->k_empty[grp]);
            if (grp == 2) {
              tp::commit_both(&bars->s_full[t & 1]);
              if (last) tp::commit_both(&bars->q_empty);
            }
          }
          __syncwarp();
        }
        if (k == g.k0) more = walk.next(a, after);
      }
      ++ns;
    }
  } else if (warp == 3 && rank == 0) {
    // ================= mix MMAs =================
    // In two batches.  Four, so that scores queue behind less of a mix, took 1.36 instead of 1.21
    // ms for the 64-token trees, and 1.64 with a batch held back until the one before the last had
    // finished; one batch of 16 took 1.25.
    constexpr uint32_t kIdO = tc::idesc_bf16_f32(128, 256, true);
    const uint64_t d_p = tc::smem_desc_sw128(0, 16, 1024);     // K-major
    const uint64_t d_v = tc::smem_desc_sw128(0, kSubV, 1024);  // MN-major: 64-column halves
    const uint32_t v_lo = smem_u32(sV) >> 4, p_lo = smem_u32(sP) >> 4;
    uint32_t t = 0;
    int ns = 0;
    bool ok = true;
    for (; ok && more; g = after) {
      for (int k = g.k0; k < g.k1 && ok; ++k, ++t) {
        ok = mbar_wait(&bars->p_ready, t & 1, status, abort_flag);
        if (ok && k == g.k0 && ns > 0)  // the segment before has read its mix out
          ok = mbar_wait(&bars->o_free, (ns - 1) & 1, status, abort_flag);
#pragma unroll 1
        for (int n = 0; n < 2; ++n) {
          ok = ok && mbar_wait(&bars->v_full[n], t & 1, status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t d = tbase + kColO + 128 * n, v_at = v_lo + 2 * n * (kSubV >> 4);
          const uint32_t acc = k > g.k0 ? 1u : 0u;
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tp::mma_ss(d, d_p | (uint64_t)(p_lo + (kk >> 2) * (kSubQ >> 4) + (kk & 3) * 2),
                         d_v | (uint64_t)(v_at + kk * (2048 >> 4)), kIdO, kk > 0 ? 1u : acc);
            tp::commit_both(n ? &bars->mix_done : &bars->v_empty);
          }
          __syncwarp();
        }
        if (k == g.k0) more = walk.next(a, after);
      }
      ++ns;
    }
  } else if (warp >= 4) {
    // ================= softmax =================
    const int q4 = warp & 3;
    const int half = q4 >> 1;                 // keys 64 half .. of a tile
    const int r = (q4 & 1) * 32 + lane;       // row of this CTA's 64
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    float* red = reinterpret_cast<float*>(smem + kOffRed);  // [parity][half][64]
    const uint32_t s_free = tp::even_addr(&bars->s_free[0]);
    const uint32_t p_ready = tp::even_addr(&bars->p_ready);
    const uint32_t o_free = tp::even_addr(&bars->o_free);
    const float sl2 = a.scale_log2;
    const bool wide = (reinterpret_cast<uintptr_t>(a.q_lat) & 31u) == 0;  // part_acc alike
    // What a slot holds, for the merge: first row, rows, whether it is its unit's first segment
    // and its last.  One thread clears the pair's two notes and fills in those of its segments.
    const bool notes = rank == 0 && threadIdx.x == 128;
    if (notes) {
      a.part_note[2 * pair_id] = make_int4(0, 0, 0, 0);
      a.part_note[2 * pair_id + 1] = make_int4(0, 0, 0, 0);
    }
    clear_keyless(a, pair_id, rank * 128 + threadIdx.x - 128, 256);
    uint32_t t = 0;
    bool ok = true, gone = false;  // a wait of this thread's gave up; all four warps leave
    for (; more; g = after) {
      const int first = rows_first(a, g);
      const int row = g.m * kRows + first * rank + r;  // row of the sequence
      const bool real = r < first && row < g.s.n * a.H;
      const int i = row / a.H;                      // new token
      const bool masked = a.draft_mask != nullptr;
      const uint64_t mask = masked && real ? (uint64_t)a.draft_mask[g.s.q0 + i] : 0ull;
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
        if (lane == 0) tp::arrive(s_free + 8 * (t & 1));
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
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e >> 1) & 3] = fmax3(mx[(e >> 1) & 3], __uint_as_float(x[c][e]),
                                     __uint_as_float(x[c][e + 1]));
        const float own = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        float* rd = red + (t & 1) * 128;
        rd[half * 64 + r] = own;
        gone = !softmax_and(ok);
        if (gone) break;
        const float top = fmaxf(own, rd[(half ^ 1) * 64 + r]) * sl2;
        // Both threads of a row take the same decisions from the same maxima.
        const bool need = top > m + kRescale || (m == -INFINITY && top > -INFINITY);
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m - top);
          m = top;
          l *= alpha;
        }
        const float mb = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights are 2^-inf = 0
        const uint64_t sl2_2 = f2_pack(sl2, sl2), neg_2 = f2_pack(-mb, -mb);
        uint64_t sum2[2] = {0ull, 0ull};
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            f2_unpack(ffma2(f2_pack(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])), sl2_2,
                            neg_2),
                      p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum2[(e >> 1) & 1] = fadd2(sum2[(e >> 1) & 1], f2_pack(p0, p1));
            pk[c * 16 + (e >> 1)] = pack_bf16x2(p0, p1);
          }
        float sa, sb;
        f2_unpack(fadd2(sum2[0], sum2[1]), sa, sb);
        l += sa + sb;
        // The weights' buffer and O are free once the tile before has been mixed in.
        if (t > 0) ok = mbar_wait(&bars->mix_done, (t - 1) & 1, status, abort_flag);
        __syncwarp();
        if (k > g.k0 && __any_sync(0xffffffffu, need)) {
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < 16; ++c) {
            uint32_t o[16];
            tc::tmem_ld16(tbase + lane_off + kColO + c * 16, o);
            tc::tmem_wait_ld();
            pin<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::tmem_st16(tbase + lane_off + kColO + c * 16, o);
          }
          tc::tmem_wait_st();
        }
        // Weights [64 rows x 64 keys] of this half, 128-byte swizzled like a TMA tile.
        uint8_t* dst = sP + half * kSubQ + r * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(dst + ((c ^ (r & 7)) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc::fence_before_sync();
        __syncwarp();
#ifdef MLA_TEST_DROP_P_READY
        // Test build only: a softmax warp of the first pair withholds the arrival for its second
        // tile.  The mix warp's bounded wait for it then gives up, which exercises the timeout
        // report and the unwinding of both CTAs.
        const bool withhold = blockIdx.x == 0 && warp == 4 && t == 1;
#else
        constexpr bool withhold = false;
#endif
        if (lane == 0 && !withhold) tp::arrive(p_ready);
      }
      if (gone) break;
      more = walk.next(a, after);
      // The segment's mix, once its last tile has been added.
      ok = ok && mbar_wait(&bars->mix_done, (t - 1) & 1, status, abort_flag);
      __syncwarp();
      tc::fence_after_sync();
      float* rl = red + (t & 1) * 128;  // this parity's maxima are behind a barrier
      rl[half * 64 + r] = l;
      gone = !softmax_and(ok);
      if (gone) break;
      l += rl[(half ^ 1) * 64 + r];
      const bool whole = g.slot < 0;
      const float f = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
      if (!whole && notes)
        a.part_note[g.slot] = make_int4(g.s.q0 * a.H + g.m * kRows,
                                        min(kRows, g.s.n * a.H - g.m * kRows), g.k0 == 0,
                                        g.k1 == seq_tiles(g.s));
      const size_t slot_row = (size_t)(whole ? 0 : g.slot) * kRows + first * rank;
      if (!whole && half == 0 && r < first)
        *reinterpret_cast<float2*>(a.part_ml + (slot_row + r) * 2) = make_float2(m, l);
      // Each lane writes its own row, 64 columns at a time, in 32-byte stores, a whole sector each:
      // a store instruction takes a cycle per row, so a segment's 64 KB per warp take about 4100
      // cycles (9000 with 16-byte stores, 6400 through shared memory and tensor stores, whose
      // only free buffer is one stage).  The TMEM loads are waited for where they are issued:
      // a register that is still being loaded must not be carried around the loop, the compiler
      // may move it.
      uint16_t* fin = a.q_lat + ((size_t)g.s.q0 * a.H + row) * kLD;
      float* part = a.part_acc + (slot_row + r) * kLD;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[2][32];
        tc::tmem_ld32(tbase + lane_off + kColO + c * 64, o[0]);
        tc::tmem_ld32(tbase + lane_off + kColO + c * 64 + 32, o[1]);
        tc::tmem_wait_ld();
        pin<32>(o[0]);
        pin<32>(o[1]);
        if (c == 3) {  // the mix is out of TMEM: the next segment's may be written
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tp::arrive(o_free);
        }
        if (!real) continue;
        const int col = 256 * (c >> 1) + 128 * half + 64 * (c & 1);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (whole) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              w[k] = pack_bf16x2(__uint_as_float(o[q][2 * k]) * f,
                                 __uint_as_float(o[q][2 * k + 1]) * f);
            store32(fin + col + 32 * q, w, 0, wide);
            store32(fin + col + 32 * q + 16, w, 8, wide);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(part + col + 32 * q + e, o[q], e, wide);
          }
        }
      }
      softmax_and(true);  // the sums have been read before the next tile's maxima
    }
  }

  // A CTA leaves once neither it nor its peer has anything in flight into its shared memory.
  // In the regular course every copy and MMA has been waited for by now.  After a wait gave
  // up, copies may still be landing: they take microseconds.
  __syncwarp();
  if (*abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tp::cluster_sync();
  if (warp == 1) {
    tc::fence_after_sync();
    tp::tmem_dealloc(tbase, 512);
  }
}

// Tensor maps, cached by pointers and sizes.  Calls that go round more sets than there are entries (a
// model's layers, each with its pages and weight) encode all ten of a call, 0.8 us of its 17 on the
// host.
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
  CUtensorMap maps[4];
  bool valid;
};
std::mutex g_mu;
MapEntry g_maps[16];
int g_next = 0;

bool tree_maps(const TreeArgs& a, TreeParams* p) {
  const MapKey key = {{a.q_lat, a.q_pe, a.c_pages, a.pe_pages}, a.T, a.H, a.num_pages, a.page_shift};
  std::lock_guard<std::mutex> lk(g_mu);
  for (const MapEntry& e : g_maps) {
    if (e.valid && e.key == key) {
      p->tm_q = e.maps[0];
      p->tm_qr = e.maps[1];
      p->tm_c = e.maps[2];
      p->tm_kr = e.maps[3];
      return true;
    }
  }
  const uint64_t rows = (uint64_t)a.T * a.H, slots = (uint64_t)a.num_pages << a.page_shift;
  const uint32_t box = std::min(1 << a.page_shift, 64);
  if (!encode_bf16_3d(&p->tm_q, a.q_lat, kLD, rows, 1, rows, 64) ||
      !encode_bf16_3d(&p->tm_qr, a.q_pe, 64, rows, 1, rows, 64) ||
      !encode_bf16_3d(&p->tm_c, a.c_pages, kLD, slots, 1, slots, box) ||
      !encode_bf16_3d(&p->tm_kr, a.pe_pages, 64, slots, 1, slots, box))
    return false;
  MapEntry& e = g_maps[g_next];
  g_next = (g_next + 1) % 16;
  e.key = key;
  e.maps[0] = p->tm_q;
  e.maps[1] = p->tm_qr;
  e.maps[2] = p->tm_c;
  e.maps[3] = p->tm_kr;
  e.valid = true;
  return true;
}

}  // namespace

cudaError_t launch_latent_tree(const TreeArgs& a, cudaStream_t stream) {
  TreeParams p;
  if (!tree_maps(a, &p)) return cudaErrorInvalidValue;
  p.a = a;
  static std::atomic<uint64_t> attr_done{0};  // bit per device: smem attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(tree_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_release);
  }
  e = launch_tree_fold(a, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2 * a.pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  e = cudaLaunchKernelEx(&cfg, tree_split_kernel, p);
  if (e != cudaSuccess) return e;
  return launch_tree_up(a, stream);
}

}  // namespace mla
