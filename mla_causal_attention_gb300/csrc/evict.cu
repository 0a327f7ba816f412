// evict.cu -- which rows of a paged cache stay within a budget, and moving them together.
//
//   paged_evict_kernel     the rows that each sequence keeps, and the pages that come free
//   latent_compact_kernel  the kept rows to the front of their sequence's pages, in place
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
// A word of CTA `rank`'s shared memory, at the place of this CTA's p.
__device__ __forceinline__ int peer_load(const int* p, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// ---- choice -----------------------------------------------------------------------------
// Sequence b of len rows keeps k = min(len, budget): its first s = min(sinks, k), its last
// r = min(recent, k - s), and the m = k - s - r heaviest of those between, of equal ones the lower
// rows.  The m-th heaviest is found by its digits, 11, 11 and 10 bits of a whole number that orders
// as the weights do: a histogram of the digit over the rows that agree with the digits found so
// far, and the bin in which the m-th lies.  Then the rows above it, and as many of those equal to
// it as are missing, are listed by a prefix sum over ballots.
//
// A cluster of CTAs per sequence, each with an equal run of the rows between, whose numbers it
// keeps in shared memory for the passes; the histograms are added up through distributed shared
// memory.  The work is 4 bytes per row: what bounds it is latency, of the loads through the block
// table and of the barriers between the passes.
constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kBins = 2048;

struct EvictSmem {
  int hist[3][kBins];
  int part[kEvWarps];             // of a block-wide scan
  int above[kEvWarps], ties[kEvWarps];  // rows of each warp's run
  int cta[2];                     // rows above, ties of this CTA
  int bin, left;                  // the bin found, and the rank that is left within it
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

// Exclusive prefix sum over the block's threads; *total is the sum.  Two barriers.
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
  int p = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += x;
  }
  *total = __shfl_sync(0xffffffffu, p, 31);
  const int before = __shfl_sync(0xffffffffu, p, (warp + 31) & 31);
  __syncthreads();
  return inc - v + (warp ? before : 0);
}

__global__ void __launch_bounds__(kEvThreads) paged_evict_kernel(const PagedEvictArgs a) {
  extern __shared__ uint32_t keys[];  // this CTA's numbers, the first a.held of them
  __shared__ EvictSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int b = blockIdx.x / C;
  const EvictSeq q = evict_seq(a, b);
  const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
  int32_t* kept = a.kept + (int64_t)b * a.K;
  const int share = rank * kEvThreads + tid, shares = C * kEvThreads;
  if (q.bad && share == 0) set_status(a.status, MLA_ERR_KVLEN);

  // What needs no choice: the ends, or everything; the rest of the row.
  const int head = q.k < q.len ? q.s : q.k;
  for (int i = share; i < head; i += shares) kept[i] = i;
  for (int i = share; i < a.K - q.k; i += shares) kept[q.k + i] = -1;
  if (q.k < q.len)
    for (int i = share; i < q.r; i += shares) kept[q.k - q.r + i] = q.len - q.r + i;
  if (share == 0) a.kept_len[b] = q.k;

  // Pages past the kept rows, behind those of the sequences before.
  if (a.freed && rank == C - 1) {
    int before = 0, own_total;
    for (int i = tid; i < b; i += kEvThreads) {
      const EvictSeq o = evict_seq(a, i);
      before += pages_for(a, o.len) - pages_for(a, o.k);
    }
    block_scan(before, sm.part, &own_total);
    const int from = pages_for(a, q.k), n = pages_for(a, q.len) - from;
    for (int i = tid; i < n; i += kEvThreads) {
      const int page = table[from + i];
      if (page < 0 || page >= a.num_pages) set_status(a.status, MLA_ERR_PAGE);
      a.freed[own_total + i] = page;
    }
    if (b == a.B - 1 && tid == 0) a.n_freed[0] = own_total + n;
  }
  if (q.m == 0) return;  // the whole cluster: nothing to choose

  // This CTA's run of the rows between the ends.
  const int mid = q.len - q.s - q.r;  // > m
  const int per = (mid + C - 1) / C;
  const int i0 = min(rank * per, mid), n = min(per, mid - i0);
  const auto weigh = [&](int i) {
    const int row = q.s + i0 + i;
    const int page = table[row >> a.page_shift];
    if (page < 0 || page >= a.num_pages) {
      set_status(a.status, MLA_ERR_PAGE);
      return 0u;
    }
    return order_of(a.weights[((int64_t)page << a.page_shift) + (row & ((1 << a.page_shift) - 1))]);
  };
  const auto number = [&](int i) { return i < a.held ? keys[i] : weigh(i); };
  for (int i = tid; i < 3 * kBins; i += kEvThreads) (&sm.hist[0][0])[i] = 0;
  for (int i = tid; i < min(n, a.held); i += kEvThreads) keys[i] = weigh(i);
  __syncthreads();

  uint32_t found = 0;  // the digits of the m-th heaviest so far, from the top
  int left = q.m;      // its rank among the rows that agree with them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const uint32_t agree = pass == 0 ? 0u : ~0u << (shift + bits);
    for (int i = tid; i < n; i += kEvThreads) {
      const uint32_t v = number(i);
      if ((v & agree) == found) atomicAdd(&sm.hist[pass][(v >> shift) & ((1 << bits) - 1)], 1);
    }
    cluster_barrier();
    // Thread t adds up bins 2047 - 2 t and 2046 - 2 t, so that a prefix sum counts from the top.
    const int hi = kBins - 1 - 2 * tid, lo = hi - 1;
    int at_hi = 0, at_lo = 0;
    for (int c = 0; c < C; ++c) {
      at_hi += peer_load(&sm.hist[pass][hi], c);
      at_lo += peer_load(&sm.hist[pass][lo], c);
    }
    int total;
    const int above = block_scan(at_hi + at_lo, sm.part, &total);
    if (above < left && left <= above + at_hi + at_lo) {
      const bool first = left <= above + at_hi;
      sm.bin = first ? hi : lo;
      sm.left = left - above - (first ? 0 : at_hi);
    }
    __syncthreads();
    found |= (uint32_t)sm.bin << shift;
    left = sm.left;
    __syncthreads();
  }

  // `left` of the rows equal to `found` are kept, the lowest ones.  Warps have runs of rows.
  const int run = ((n + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int w0 = min(warp * run, n), w1 = min(w0 + run, n);
  int above = 0, ties = 0;
  for (int i = w0 + lane; i < w0 + ((w1 - w0 + 31) & ~31); i += 32) {
    const uint32_t v = i < w1 ? number(i) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < w1 && v > found));
    ties += __popc(__ballot_sync(0xffffffffu, i < w1 && v == found));
  }
  if (lane == 0) {
    sm.above[warp] = above;
    sm.ties[warp] = ties;
  }
  __syncthreads();
  if (warp == 0) {
    const int x = __reduce_add_sync(0xffffffffu, sm.above[lane]);
    const int y = __reduce_add_sync(0xffffffffu, sm.ties[lane]);
    if (lane == 0) {
      sm.cta[0] = x;
      sm.cta[1] = y;
    }
  }
  cluster_barrier();
  above = lane < warp ? sm.above[lane] : 0;
  ties = lane < warp ? sm.ties[lane] : 0;
  if (lane < rank) {  // at most 16 CTAs
    above += peer_load(&sm.cta[0], lane);
    ties += peer_load(&sm.cta[1], lane);
  }
  above = __reduce_add_sync(0xffffffffu, above);  // before this warp's run
  ties = __reduce_add_sync(0xffffffffu, ties);
  const uint32_t below = (1u << lane) - 1;
  for (int i = w0 + lane; i < w0 + ((w1 - w0 + 31) & ~31); i += 32) {
    const uint32_t v = i < w1 ? number(i) : 0u;
    const bool up = i < w1 && v > found, tie = i < w1 && v == found;
    const uint32_t ups = __ballot_sync(0xffffffffu, up), eqs = __ballot_sync(0xffffffffu, tie);
    const int my_ties = ties + __popc(eqs & below);
    const int at = q.s + above + __popc(ups & below) + min(my_ties, left);
    // (the bound holds unless someone writes the weights meanwhile)
    if ((up || (tie && my_ties < left)) && at < q.k - q.r) kept[at] = q.s + i0 + i;
    above += __popc(ups);
    ties += __popc(eqs);
  }
  cluster_barrier();  // no CTA leaves while another may read its counts
}

// ---- compaction -------------------------------------------------------------------------
// Row kept[i] of a sequence becomes its row i, for rising lists.  kept[i] >= i, so within a run of
// rows read at a time every source lies at or behind the run's own targets: a CTA that takes the
// runs in order, reads a whole run, and writes it after a barrier, never overwrites what is still
// to be read.  Columns do not meet, so a row's 1152 bytes are cut into slices, a CTA each.
// Bound by HBM: 2 * 1156 bytes per row that moves.
constexpr int kCpThreads = 256;
constexpr int kCpU = 8;  // rows of a thread in a run

struct CompactSeq {
  const int32_t* table;
  const int32_t* kept;
  int k;
};
// The slot of position p, or -1 where the table holds no page.
__device__ __forceinline__ int64_t slot_of(const LatentCompactArgs& a, const int32_t* table, int p) {
  const int page = table[p >> a.page_shift];
  if (page < 0 || page >= a.num_pages) {
    set_status(a.status, MLA_ERR_PAGE);
    return -1;
  }
  return ((int64_t)page << a.page_shift) + (p & ((1 << a.page_shift) - 1));
}
// Source and target of kept row i; false where it stays or the list is no such list.
__device__ __forceinline__ bool move_of(const LatentCompactArgs& a, const CompactSeq& q, int i,
                                        int64_t& from, int64_t& to) {
  if (i >= q.k) return false;
  const int p = q.kept[i];
  if (p == i) return false;
  if (p < i || p >= (int64_t)a.max_pages << a.page_shift) {
    set_status(a.status, MLA_ERR_KVLEN);
    return false;
  }
  from = slot_of(a, q.table, p);
  to = slot_of(a, q.table, i);
  return from >= 0 && to >= 0;
}

// kLanes: 16-byte pieces of a slice, a lane each.
template <typename V, int kLanes>
__device__ __forceinline__ void compact_rows(const LatentCompactArgs& a, const CompactSeq& q,
                                             V* base, int pitch, int col) {
  constexpr int kRowsPer = kCpThreads / kLanes;
  const int lane = threadIdx.x % kLanes, row = threadIdx.x / kLanes;
  for (int i0 = 0; i0 < q.k; i0 += kCpU * kRowsPer) {
    V v[kCpU];
    int64_t to[kCpU];
#pragma unroll
    for (int u = 0; u < kCpU; ++u) {
      int64_t from;
      const bool moves = move_of(a, q, i0 + u * kRowsPer + row, from, to[u]);
      if (moves)
        v[u] = base[from * pitch + col + lane];
      else
        to[u] = -1;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kCpU; ++u)
      if (to[u] >= 0) base[to[u] * pitch + col + lane] = v[u];
  }
}

template <int kLanes>
__global__ void __launch_bounds__(kCpThreads) latent_compact_kernel(const LatentCompactArgs a) {
  constexpr int kSlices = 64 / kLanes;  // of a latent row; the rotary key has 8 / kLanes
  const int slices = kSlices + 8 / kLanes + (a.weights ? 1 : 0);
  const int b = blockIdx.x / slices, slice = blockIdx.x % slices;
  CompactSeq q;
  q.table = a.block_table + (int64_t)b * a.max_pages;
  q.kept = a.kept + (int64_t)b * a.K;
  const int k = a.kept_len[b];
  q.k = (int)min((int64_t)min(max(k, 0), a.K), (int64_t)a.max_pages << a.page_shift);
  if (q.k != k) set_status(a.status, MLA_ERR_KVLEN);
  if (slice < kSlices)
    compact_rows<uint4, kLanes>(a, q, reinterpret_cast<uint4*>(a.c_pages), 64, slice * kLanes);
  else if (slice < kSlices + 8 / kLanes)
    compact_rows<uint4, kLanes>(a, q, reinterpret_cast<uint4*>(a.pe_pages), 8,
                                (slice - kSlices) * kLanes);
  else
    compact_rows<float, 1>(a, q, a.weights, 1, 0);
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictArgs& in, cudaStream_t stream) {
  PagedEvictArgs a = in;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const int64_t most = (int64_t)a.max_pages << a.page_shift;
  // CTAs of a sequence: as the SMs allow, each with 2048 rows or more where sequences can be as
  // long as the table; up to 16 of them (a cluster's size on this GPU).
  int C = 1;
  while (C < 16 && (int64_t)a.B * 2 * C <= sms && most > (int64_t)2048 * C) C *= 2;
  constexpr int kMostHeld = 49152;  // numbers that fit beside the histograms
  a.held = (int)std::min<int64_t>((most + C - 1) / C, kMostHeld);
  static std::atomic<uint64_t> attr_done{0};  // bit per device: attributes set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(paged_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMostHeld * 4);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(paged_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * C));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = (size_t)a.held * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_evict_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_latent_compact(const LatentCompactArgs& a, cudaStream_t stream) {
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const unsigned more = a.weights ? 1 : 0;
  // Slices of 128 bytes; of 32 where few sequences would leave SMs idle.
  if ((int64_t)a.B * 9 >= 2 * sms)
    latent_compact_kernel<8><<<(9 + more) * a.B, kCpThreads, 0, stream>>>(a);
  else
    latent_compact_kernel<2><<<(36 + more) * a.B, kCpThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
