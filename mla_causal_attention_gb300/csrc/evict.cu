// evict.cu -- which rows of a paged cache stay within a budget, and moving them together.
//
//   paged_evict_kernel     the rows that each sequence keeps, and the pages that come free
//   compact_chunks_kernel, latent_compact_kernel
//                          the kept rows to the front of their sequence's pages, in place
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace mla {
namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// One or two words of CTA `rank`'s shared memory, at the place of this CTA's p.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ int2 peer_load2(const int* p, uint32_t rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(peer_addr(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ int peer_load(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}

// ---- choice -----------------------------------------------------------------------------
// Sequence b of len rows keeps k = min(len, budget): its first s = min(sinks, k), its last
// r = min(recent, k - s), and the m = k - s - r heaviest of those between, of equal ones the lower
// rows.  The m-th heaviest is found by its digits, four of 8 bits of a whole number that orders
// as the weights do: a histogram of the digit over the rows that agree with the digits found so
// far, and the bin in which the m-th lies.  Then the rows above it, and as many of those equal to
// it as are missing, are listed by a prefix sum over ballots.
//
// A cluster of CTAs per sequence, each with an equal run of the rows between and each warp with an
// equal run of those; the histograms are added up through distributed shared memory.  The numbers
// stay in registers for all passes, or, with more than 8 to a thread, in shared memory, and what that
// does not hold is read again.  The work is 4
// bytes per row: what bounds it is latency, of the loads through the block table and of the barriers
// between the passes.
constexpr int kEvPer = 8;        // rows of a thread at a time
constexpr int kPasses = 4, kBins = 256;  // (three of 2048: every CTA reads all histograms, 10 us a pass)

template <int kEvWarps>
struct EvictSmem {
  alignas(16) int hist[kPasses][kBins];
  alignas(16) int sum[2][kBins];  // all CTAs' histograms, by the parity of the pass
  int part[kEvWarps];             // of a block-wide scan
  int above[kEvWarps], ties[kEvWarps];  // rows of each warp's run
  alignas(8) int cta[2];          // rows above, ties of this CTA
};

struct EvictSeq {
  int len, k, s, r, m;
  bool bad;
};
__device__ __forceinline__ EvictSeq evict_seq(const PagedEvictArgs& a, int b) {
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  const int n = a.kv_len[b], want = a.budget[b];
  EvictSeq q;
  q.len = (int)min((int64_t)max(n, 0), cap);
  const int most = min(q.len, max(want, 0));
  q.k = min(most, a.K);
  q.s = min(a.sinks, q.k);
  q.r = min(a.recent, q.k - q.s);
  q.m = q.k < q.len ? q.k - q.s - q.r : 0;
  q.bad = q.len != n || want < 0 || most > a.K;
  return q;
}
__device__ __forceinline__ int pages_for(const PagedEvictArgs& a, int rows) {
  return (int)(((int64_t)rows + (1 << a.page_shift) - 1) >> a.page_shift);
}

// A whole number that orders as the weights do; NaN is the lowest, minus zero is zero.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum over the block's threads; *total is the sum.  One barrier; `part` is not to be
// used again before another.
template <int kWarps>
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  const int p = lane < kWarps ? part[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, p);
  return inc - v + __reduce_add_sync(0xffffffffu, lane < warp ? p : 0);
}

// kEvThreads: 512, two CTAs on an SM, or 1024 where a CTA's rows are more than the registers of 512 hold.
constexpr int kFewThreads = 512, kManyThreads = 1024;
template <int kEvThreads>
__global__ void __launch_bounds__(kEvThreads, 1024 / kEvThreads)
    paged_evict_kernel(const PagedEvictArgs a) {
  constexpr int kEvWarps = kEvThreads / 32;
  constexpr bool kRounds = kEvThreads == kManyThreads;  // a thread may have more rows than registers
  extern __shared__ uint32_t keys[];  // numbers of each warp's first a.held rounds of rows
  __shared__ EvictSmem<kEvWarps> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int b = blockIdx.x / C;
  const EvictSeq q = evict_seq(a, b);
  const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
  int32_t* kept = a.kept + (int64_t)b * a.K;
  const int share = rank * kEvThreads + tid, shares = C * kEvThreads;
  // Pages past the kept rows, behind those of the sequences before, which every cluster counts for itself:
  // 512 sequences of 100 rows take 19 us with the list and 18 without, 4096 of them 119 and 106, 65535
  // 3.1 ms and 1.6.  What is loaded for that is on its way together with the weights.
  const int gone0 = pages_for(a, q.k), gone = pages_for(a, q.len) - gone0;
  int before = 0, page0 = 0;
  if (a.freed) {
    for (int i = tid; i < b; i += kEvThreads) {
      const EvictSeq o = evict_seq(a, i);
      before += pages_for(a, o.len) - pages_for(a, o.k);
    }
    if (share < gone) page0 = table[gone0 + share];
  }
  const auto all_ctas = [&] {  // a barrier over the cluster
    if (C > 1) cluster_barrier(); else __syncthreads();
  };

  if (q.m > 0) {
    // This CTA's run of the rows between the ends, and this warp's of those.
    const int mid = q.len - q.s - q.r;  // > m
    const int per = (mid + C - 1) / C;
    const int i0 = min(rank * per, mid), n = min(per, mid - i0);
    const int run = (((n + kEvWarps - 1) / kEvWarps) + 31) & ~31;
    const int w0 = min(warp * run, n), w1 = min(w0 + run, n);
    const int rounds = kRounds ? (run + 32 * kEvPer - 1) / (32 * kEvPer) : 1;
    bool bad = false;
    // Rows w0 + lane + 32 (kEvPer round + e) of this thread, from the pool: the loads of a round at once.
    uint32_t v[kEvPer];
    const auto weigh = [&](int round) {
      const int first = w0 + 32 * kEvPer * round + lane;
      int page[kEvPer];
#pragma unroll
      for (int e = 0; e < kEvPer; ++e)
        page[e] = first + 32 * e < w1 ? table[(q.s + i0 + first + 32 * e) >> a.page_shift] : 0;
#pragma unroll
      for (int e = 0; e < kEvPer; ++e) {
        const int row = q.s + i0 + first + 32 * e;
        const bool held = page[e] >= 0 && page[e] < a.num_pages;
        float w = __uint_as_float(0x7fc00000u);  // counts as lowest
        if (first + 32 * e < w1 && held)
          w = a.weights[((int64_t)page[e] << a.page_shift) + (row & ((1 << a.page_shift) - 1))];
        v[e] = __float_as_uint(w);
        bad |= !held;
      }
#pragma unroll
      for (int e = 0; e < kEvPer; ++e) v[e] = order_of(__uint_as_float(v[e]));
    };
    uint32_t* mine = keys + (size_t)warp * a.held * 32 * kEvPer + lane;  // 32 kEvPer to a round
    const auto fetch = [&](int round) {
      if (rounds == 1) return;  // they are in the registers
      if (round >= a.held) return weigh(round);
#pragma unroll
      for (int e = 0; e < kEvPer; ++e) v[e] = mine[32 * (kEvPer * round + e)];
    };
    weigh(0);
    for (int i = tid; i < kPasses * kBins; i += kEvThreads) (&sm.hist[0][0])[i] = 0;
    if (rounds > 1)
      for (int r = 0; r < min(rounds, a.held); ++r) {
        if (r > 0) weigh(r);
#pragma unroll
        for (int e = 0; e < kEvPer; ++e) mine[32 * (kEvPer * r + e)] = v[e];
      }
    __syncthreads();

    uint32_t found = 0;  // the digits of the m-th heaviest so far, from the top
    int left = q.m;      // its rank among the rows that agree with them
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
      const int shift = 24 - 8 * pass;
      const uint32_t agree = pass == 0 ? 0u : ~0u << (shift + 8);
      for (int r = 0; r < rounds; ++r) {
        fetch(r);
        const int first = w0 + 32 * kEvPer * r + lane;
#pragma unroll
        for (int e = 0; e < kEvPer; ++e)
          if (first + 32 * e < w1 && (v[e] & agree) == found)
            atomicAdd(&sm.hist[pass][(v[e] >> shift) & 255], 1);
      }
      all_ctas();
      const int* sum = sm.hist[pass];
      if (C > 1) {
        if (tid < kBins) {
          int at = 0;
          for (int c0 = 0; c0 < C; c0 += 8) {
            int x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = peer_load(&sm.hist[pass][tid], min(c0 + e, C - 1));
#pragma unroll
            for (int e = 0; e < 8; ++e) at += c0 + e < C ? x[e] : 0;
          }
          sm.sum[pass & 1][tid] = at;
        }
        __syncthreads();
        sum = sm.sum[pass & 1];
      }
      // Every warp finds the bin for itself: lane l has bins 8 (31 - l) .. + 7, so that a prefix sum
      // counts from the top.
      const int lo = 8 * (31 - lane);
      const int4 x = *reinterpret_cast<const int4*>(sum + lo), y = *reinterpret_cast<const int4*>(sum + lo + 4);
      const int d[8] = {y.w, y.z, y.y, y.x, x.w, x.z, x.y, x.x};
      int all = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) all += d[e];
      int upto = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += z;
      }
      const uint32_t reach = __ballot_sync(0xffffffffu, upto >= left);
      const int at = __ffs(reach) - 1;  // the first lane by which the m-th is counted
      int bin = lo + 7, rest = left - (upto - all);
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (rest > d[e] && bin == lo + 7 - e) {
          rest -= d[e];
          --bin;
        }
      found |= (uint32_t)__shfl_sync(0xffffffffu, bin, at) << shift;
      left = __shfl_sync(0xffffffffu, rest, at);
    }

    // `left` of the rows equal to `found` are kept, the lowest ones.
    int above = 0, ties = 0;
    for (int r = 0; r < rounds; ++r) {
      fetch(r);
#pragma unroll
      for (int e = 0; e < kEvPer; ++e) {
        const bool real = w0 + 32 * (kEvPer * r + e) + lane < w1;
        above += real && v[e] > found;
        ties += real && v[e] == found;
      }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
      sm.above[warp] = above;
      sm.ties[warp] = ties;
    }
    __syncthreads();
    above = lane < kEvWarps ? sm.above[lane] : 0;
    ties = lane < kEvWarps ? sm.ties[lane] : 0;
    if (C > 1) {
      if (warp == 0) {
        const int x = __reduce_add_sync(0xffffffffu, above), y = __reduce_add_sync(0xffffffffu, ties);
        if (lane == 0) {
          sm.cta[0] = x;
          sm.cta[1] = y;
        }
      }
      cluster_barrier();
    }
    if (lane >= warp) above = ties = 0;
    if (lane < rank) {  // at most 16 CTAs
      const int2 o = peer_load2(sm.cta, lane);
      above += o.x;
      ties += o.y;
    }
    above = __reduce_add_sync(0xffffffffu, above);  // before this warp's run
    ties = __reduce_add_sync(0xffffffffu, ties);
    const uint32_t below = (1u << lane) - 1;
    for (int r = 0; r < rounds; ++r) {
      fetch(r);
#pragma unroll
      for (int e = 0; e < kEvPer; ++e) {
        const int row = w0 + 32 * (kEvPer * r + e) + lane;
        const bool up = row < w1 && v[e] > found, tie = row < w1 && v[e] == found;
        const uint32_t ups = __ballot_sync(0xffffffffu, up), eqs = __ballot_sync(0xffffffffu, tie);
        const int my_ties = ties + __popc(eqs & below);
        const int at = above + __popc(ups & below) + min(my_ties, left);
        // (the bounds hold unless someone writes the weights meanwhile)
        if ((up || (tie && my_ties < left)) && at >= 0 && at < q.m) kept[q.s + at] = q.s + i0 + row;
        above += __popc(ups);
        ties += __popc(eqs);
      }
    }
    if (bad) set_status(a.status, MLA_ERR_PAGE);
  }

  // What needs no choice: the ends, or everything; the rest of the row.
  const int head = q.k < q.len ? q.s : q.k;
  for (int i = share; i < head; i += shares) kept[i] = i;
  for (int i = share; i < a.K - q.k; i += shares) kept[q.k + i] = -1;
  if (q.k < q.len)
    for (int i = share; i < q.r; i += shares) kept[q.k - q.r + i] = q.len - q.r + i;
  if (share == 0) {
    a.kept_len[b] = q.k;
    if (q.bad) set_status(a.status, MLA_ERR_KVLEN);
  }
  if (a.freed) {
    int at;
    block_scan<kEvWarps>(before, sm.part, &at);
    for (int i = share; i < gone; i += shares) {
      const int page = i == share ? page0 : table[gone0 + i];
      if (page < 0 || page >= a.num_pages) set_status(a.status, MLA_ERR_PAGE);
      a.freed[at + i] = page;
    }
    if (b == a.B - 1 && share == 0) a.n_freed[0] = at + gone;
  }
  if (q.m > 0 && C > 1) cluster_barrier();  // no CTA leaves while another may read its counts
}

// ---- compaction -------------------------------------------------------------------------
// Row kept[i] of a sequence becomes its row i, for rising lists, so kept[i] >= i.  Chunks of 32 rows
// go to warps in order, as they come free.  A warp reads its chunk's rows into shared memory, says
// so, waits until every row that lies where it is going to write has been read by the chunk it belongs to,
// and writes.  Those are the rows kept[k] in [32 c, 32 c + 32), which belong to chunks up to
// c: all of them have been handed out before, and reading waits for nothing, so every wait ends.
// Where half of the rows go, the chunks waited for are half as far down and long since read; where
// few go, they are the two or three before, which are being read at the same time.
//
// 2 * 1156 bytes per row that moves; six warps per SM with 36 KB each keep 33 MB in flight.  What bounds
// it is the chain of a warp's chunk, its list and table, reads and writes one after the other: 64
// sequences' 113000 rows take 55 us, 54 where they go to other memory and wait for nothing, so that being in
// place costs next to nothing; 34 with reads alone, 36 with writes alone, 19 with neither.  (A CTA per
// sequence and slice of the columns, which reads and writes runs of rows in turn, took 107 us for 64
// sequences and 460 for 65536 rows of one.)
constexpr int kCpRows = 32;                      // of a chunk, a lane each
constexpr int kCpWarps = 6;
constexpr int kCpSlot = kCpRows * (1024 + 128);  // a chunk's latent rows, then its rotary keys
constexpr int kCpSmem = kCpWarps * kCpSlot + 64;
static_assert(kCpSmem <= 232448, "shared memory per block");

__device__ __forceinline__ int64_t kept_rows(const LatentCompactArgs& a, int b) {
  return min((int64_t)min(max(a.kept_len[b], 0), a.K), (int64_t)a.max_pages << a.page_shift);
}

// By one block: the chunks in front of each sequence, no chunk taken, none read (65535 sequences of 50 kept
// rows take 1.5 ms in all, 512 of them 18 us).
constexpr int kListThreads = 1024;
__global__ void __launch_bounds__(kListThreads) compact_chunks_kernel(const LatentCompactArgs a) {
  grid_dep_launch();
  __shared__ int part[kListThreads / 32];
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kListThreads) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.B) {
      const int64_t k = kept_rows(a, b);
      if (k != a.kept_len[b]) set_status(a.status, MLA_ERR_KVLEN);
      n = (int)((k + kCpRows - 1) / kCpRows);
    }
    int total;
    const int own = block_scan<kListThreads / 32>(n, part, &total);
    if (b < a.B) a.chunk0[b] = before + own;
    before += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    a.chunk0[a.B] = before;
    a.chunk0[a.B + 1] = 0;  // the next chunk to hand out
  }
  for (int64_t i = threadIdx.x; i < before; i += kListThreads) a.read[i] = 0;
}

// The first of n rising values that is >= x, by a warp.
__device__ __forceinline__ int first_at_least(const int32_t* v, int n, int x, int lane) {
  int lo = 0, hi = n;  // every value before lo is below x, hi's is not (or is the end)
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step - 1;
    const uint32_t below = __ballot_sync(0xffffffffu, at < hi && v[at] < x);
    const int k = __popc(below);  // whole steps below x
    lo += k * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// The slot of position p, or -1 where the table holds no page.
__device__ __forceinline__ int64_t slot_of(const LatentCompactArgs& a, const int32_t* table, int p) {
  const int page = table[p >> a.page_shift];
  if (page < 0 || page >= a.num_pages) {
    set_status(a.status, MLA_ERR_PAGE);
    return -1;
  }
  return ((int64_t)page << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}

__global__ void __launch_bounds__(32 * kCpWarps) latent_compact_kernel(const LatentCompactArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + kCpWarps * kCpSlot) + warp;
  uint8_t* c_row = smem + warp * kCpSlot + lane * 1024;
  uint8_t* pe_row = smem + warp * kCpSlot + kCpRows * 1024 + lane * 128;
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_dep_wait();
  const int64_t chunks = a.chunk0[a.B];
  const uint64_t policy = l2_policy_evict_first();
  uint32_t loads = 0;
  // The chunk that a warp moves next: its number, its sequence, this lane's row; its source and
  // target, none where it stays, or the list is no such list.
  int64_t g, first, from, to;
  int b, i, k;
  const auto take = [&] {
    g = 0;
    if (lane == 0)
      g = (int64_t)atomicAdd(reinterpret_cast<unsigned long long*>(a.chunk0 + a.B + 1), 1ull);
    g = __shfl_sync(0xffffffffu, g, 0);
    if (g >= chunks) return;
    b = 0;  // the last sequence whose chunks begin at or before g
    for (int hi = a.B; hi - b > 1;) {
      const int step = (hi - b + 31) / 32, at = b + lane * step;
      const uint32_t le = __ballot_sync(0xffffffffu, at < hi && a.chunk0[at] <= g);
      b += (31 - __clz(le | 1u)) * step;
      hi = min(hi, b + step);
    }
    first = a.chunk0[b];
    i = (int)(g - first) * kCpRows + lane;
    k = (int)kept_rows(a, b);
    from = to = -1;
    if (i < k) {
      const int p = a.kept[(int64_t)b * a.K + i];
      const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
      if (p < i || p >= (int64_t)a.max_pages << a.page_shift) {
        set_status(a.status, MLA_ERR_KVLEN);
      } else if (p != i) {
        from = slot_of(a, table, p);
        to = slot_of(a, table, i);
      }
    }
  };
  take();
  while (g < chunks) {
    const bool moves = from >= 0 && to >= 0;
    const int n = __popc(__ballot_sync(0xffffffffu, moves));
    float w = 0.f;
    // The next chunk is taken once this one's rows are on their way out; with their loads in flight
    // would be sooner, but then other warps wait longer for what it reads (compact batch 62.9 us, 55.4).
    const int64_t g_now = g, first_now = first, put = to;
    if (n == 0) {
      if (lane == 0) atomicExch(a.read + g_now, 1);  // nothing of it is read
      take();
    } else {
      if (lane == 0) mbar_arrive_expect_tx(bar, n * (1024 + 128));
      __syncwarp();
      if (moves) {
        bulk_g2s(c_row, a.c_pages + from * 512, 1024, bar, policy);
        bulk_g2s(pe_row, a.pe_pages + from * 64, 128, bar, policy);
        if (a.weights) w = a.weights[from];
      }
      // Meanwhile: the chunks that this one's targets are read by.
      const int32_t* kept = a.kept + (int64_t)b * a.K;
      const int c = (i - lane) / kCpRows, end = min(i - lane + kCpRows, k);
      const int k0 = first_at_least(kept, k, i - lane, lane), k1 = first_at_least(kept, k, end, lane);
      bool ok = true;
      const uint32_t addr = smem_u32(bar);
      const uint64_t t0 = globaltimer_ns();
      while (ok && !mbar_try_wait(addr, loads & 1)) ok = globaltimer_ns() - t0 <= kWaitLimitNs;
      ++loads;
      asm volatile("" ::"f"(w) : "memory");  // the weight is here
      __threadfence();
      __syncwarp();
#ifdef MLA_TEST_DROP_READ
      // Test build only: the first chunk does not say that it has been read.  The bounded waits for
      // it then give up.
      const bool says = g_now != 0;
#else
      constexpr bool says = true;
#endif
      if (lane == 0 && says) atomicExch(a.read + g_now, 1);
      for (int q = k0 / kCpRows + lane; ok && q < c && q * kCpRows < k1; q += 32) {
        const int* flag = a.read + first_now + q;
        int seen;
        do {
          asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(flag) : "memory");
          ok = seen != 0 || globaltimer_ns() - t0 <= kWaitLimitNs;
        } while (ok && seen == 0);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) set_status(a.status, MLA_ERR_TIMEOUT);
        // Rows may still be landing, which takes microseconds; the block ends behind them.
        for (const uint64_t t1 = globaltimer_ns(); globaltimer_ns() - t1 < 2000000ull;) {
        }
        break;
      }
      asm volatile("fence.proxy.async;" ::: "memory");
      if (moves) {
        bulk_s2g(a.c_pages + put * 512, c_row, 1024);
        bulk_s2g(a.pe_pages + put * 64, pe_row, 128);
        if (a.weights) a.weights[put] = w;
      }
      bulk_commit_group();
      take();
      bulk_wait_read_all();
      __syncwarp();
    }
  }
}

}  // namespace

namespace {

// Numbers that a CTA keeps in shared memory at most; in rounds of its threads' registers.
constexpr int kMostRows = 49152;
template <int kEvThreads>
constexpr int kMostHeld = kEvThreads == kManyThreads ? kMostRows / (kEvThreads * kEvPer) : 0;

// A launch of B clusters of C CTAs; the attributes that it needs are set once per device.
template <int kEvThreads>
cudaError_t evict_config(int B, int C, int held, int dev, cudaLaunchAttribute* attr,
                         cudaLaunchConfig_t* cfg) {
  constexpr int kRound = kEvThreads * kEvPer;
  static std::atomic<uint64_t> attr_done{0};  // bit per device: attributes set
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    cudaError_t e = cudaSuccess;
    if (kMostHeld<kEvThreads> > 0)
      e = cudaFuncSetAttribute(paged_evict_kernel<kEvThreads>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kMostHeld<kEvThreads> * kRound * 4);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(paged_evict_kernel<kEvThreads>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_release);
  }
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = C;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  *cfg = {};
  cfg->gridDim = dim3((unsigned)(B * C));
  cfg->blockDim = dim3(kEvThreads);
  cfg->dynamicSmemBytes = (size_t)held * kRound * 4;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
  return cudaSuccess;
}

// Clusters of 2^log_c CTAs that the device holds at once, or 0 if it does not say.
template <int kEvThreads>
int clusters_at_once(int log_c, int dev) {
  static std::atomic<int> known[64][5] = {};
  std::atomic<int>& k = known[dev & 63][log_c];
  int n = k.load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg;
  if (evict_config<kEvThreads>(1, 1 << log_c, kMostHeld<kEvThreads>, dev, attr, &cfg) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, paged_evict_kernel<kEvThreads>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  k.store(n, std::memory_order_relaxed);
  return n;
}

template <int kEvThreads>
cudaError_t launch_evict(PagedEvictArgs a, int C, int64_t per, int dev, cudaStream_t stream) {
  // Rounds of a warp's rows whose numbers are kept in shared memory: none where there is but one.
  constexpr int kRound = kEvThreads * kEvPer;
  const int64_t rounds = (per + kRound - 1) / kRound + 1;  // a warp's run is a multiple of 32 rows
  a.held = per <= kRound ? 0 : (int)std::min<int64_t>(rounds, kMostHeld<kEvThreads>);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg;
  const cudaError_t e = evict_config<kEvThreads>(a.B, C, a.held, dev, attr, &cfg);
  if (e != cudaSuccess) return e;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, paged_evict_kernel<kEvThreads>, a);
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t stream) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)a.max_pages << a.page_shift;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  // CTAs of a sequence: one for 4096 rows that the table allows, up to 8, or 16 for up to three sequences
  // (eight or more of them would come in waves; four to seven of 524288 rows take 62 us with 8, 31 with
  // 16, and with 65536 rows each 14.8, 12.6; shorter ones in such tables 14.2, 15.9).
  // CTAs of 512 threads, two on an SM, hold that many rows in registers; for more they have 1024.  A
  // barrier over a cluster takes 0.6 us and there are six: 64 sequences of up to 8192 rows take 13.8 us
  // with a CTA for 2048 rows, 10.3 for 4096, 10.9 for 8192.
  int C = 1;
  while (C < (a.B <= 3 ? 16 : 8) && (int64_t)a.B * 2 * C <= 2 * sms && most > (int64_t)4096 * C) C *= 2;
  // No more than the device holds at once, where fewer still have their rows' numbers in shared memory
  // (what does not is read six times: 37 sequences of 262144 rows take 86 us with 8 CTAs each, three
  // waves, 149 with 2 in one).  A cluster lies within a GPC, so of large ones there is less room
  // than the SMs have: 152, 74, 36, 14 of 2, 4, 8, 16 CTAs of 512 threads, 76, 36, 15, 7 of 1024.  A
  // second wave: 16 sequences of 65536 rows take 28 us with 8 CTAs each, 21 with 4; 70 of 32768 rows 30
  // with 4, 20 with 2; 100 of 16384 rows 28 with 2, 17 with one.
  const auto rows_of = [&](int c) { return (most + c - 1) / c; };
  const auto at_once = [&](int c) {
    int log_c = 0;
    while ((1 << log_c) < c) ++log_c;
    return rows_of(c) > kFewThreads * kEvPer ? clusters_at_once<kManyThreads>(log_c, dev)
                                             : clusters_at_once<kFewThreads>(log_c, dev);
  };
  while (C > 1 && rows_of(C / 2) <= kMostRows && a.B > at_once(C)) C /= 2;
  // All by the table's width, since the lengths are on the device: 64 sequences of 8192 rows take 10.8 us
  // in a table that wide and 29 in one of 131072 rows.
  const int64_t per = rows_of(C);
  return per > kFewThreads * kEvPer ? launch_evict<kManyThreads>(a, C, per, dev, stream)
                                    : launch_evict<kFewThreads>(a, C, per, dev, stream);
}

cudaError_t launch_latent_compact(const LatentCompactArgs& a, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};  // bit per device: smem attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(latent_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kCpSmem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_release);
  }
  compact_chunks_kernel<<<1, kListThreads, 0, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const int64_t chunks = (int64_t)a.B * ((a.K + kCpRows - 1) / kCpRows);  // at most
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, chunks));
  cfg.blockDim = dim3(32 * kCpWarps);
  cfg.dynamicSmemBytes = kCpSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_compact_kernel, a);
}

}  // namespace mla
