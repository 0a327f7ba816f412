// paged.cu -- bookkeeping and append of a paged latent cache.
//
//   paged_plan_kernel     pages for a step's new tokens, and where every token goes
//   latent_append_kernel  rotary step on the new rows and their scatter into the pages
#include <cuda.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace mla {
namespace {

// ---- plan -------------------------------------------------------------------------------
// Two prefix sums over the sequences (new tokens, pages taken) and then independent work per
// token and per table entry.  The sums are redone by every block instead of passed between
// blocks: a chunk of 1024 sequences is two loads per thread and one block scan, less than a
// second launch would cost, and no block then waits on another.  Blocks write only table
// entries that no block reads (entries read lie below ceil(ctx / page_size)), so one launch
// does everything.  Bound by launch and latency: a decode step's plan moves 2 KB.
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 4;                              // sequences per thread and chunk
constexpr int kPlanChunk = kPlanThreads * kPlanPer;      // sequences per scan
constexpr int kPlanTok = 4;                              // consecutive tokens per thread

struct PlanSeq {
  int64_t ctx, n, kv;
  int have, take;
};
// Lengths clamped to what the table holds; *bad if they had to be.
__device__ __forceinline__ PlanSeq plan_seq(const PagedPlanArgs& a, int b, bool* bad) {
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  const int64_t ctx = a.ctx_len[b], n = a.new_len[b];
  PlanSeq s;
  s.ctx = min(max(ctx, (int64_t)0), cap);
  s.n = min(max(n, (int64_t)0), (int64_t)a.T);
  s.kv = min(s.ctx + s.n, cap);
  if (s.ctx != ctx || s.n != n || s.kv != s.ctx + s.n) *bad = true;
  const int64_t up = (1 << a.page_shift) - 1;
  s.have = (int)((s.ctx + up) >> a.page_shift);
  s.take = (int)((s.kv + up) >> a.page_shift) - s.have;
  return s;
}

__device__ __forceinline__ int pages_of(const PagedPlanArgs& a, int tokens) {
  return (int)(((int64_t)tokens + (1 << a.page_shift) - 1) >> a.page_shift);
}

// The k-th page a step takes, or -1 where the free list has run out or holds no page.
__device__ __forceinline__ int plan_page(const PagedPlanArgs& a, int64_t head, int64_t k) {
  const int64_t at = head + k;
  if (at >= a.n_free) return -1;
  const int page = a.free_pages[at];
  return page >= 0 && page < a.num_pages ? page : -1;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedPlanArgs a) {
  __shared__ int64_t s_tok[kPlanChunk + 1];  // first token of each sequence of the chunk
  __shared__ int64_t s_pg[kPlanChunk + 1];   // first page taken
  __shared__ int s_ctx[kPlanChunk], s_kv[kPlanChunk];
  __shared__ int s_par[64 + kPlanThreads * kPlanTok];  // parents of a turn's tokens, and before
  __shared__ int64_t s_warp[2][kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t head0 = a.free_head[0];
  const int64_t head = min(max(head0, (int64_t)0), (int64_t)a.n_free);
  if (head != head0 && tid == 0 && blockIdx.x == 0) set_status(a.status, MLA_ERR_PAGE);
  const int psize = 1 << a.page_shift;
  const int64_t last_pos = ((int64_t)a.max_pages << a.page_shift) - 1;

  // This block's tokens: an equal share of the T rows, in whole groups of kPlanTok.
  const int64_t groups = (a.T + kPlanTok - 1) / kPlanTok;
  const int64_t t0 = groups * blockIdx.x / gridDim.x * kPlanTok;
  const int64_t t1 = min(groups * (blockIdx.x + 1) / gridDim.x * kPlanTok, (int64_t)a.T);

  int64_t tok = 0, pg = 0;  // totals of the chunks before this one
  int chunk = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanChunk, ++chunk) {
    // Blocks share out the chunks' table rows; past its tokens and rows a block is done, but
    // block 0 goes on to the totals.
    const bool rows_mine = a.B <= kPlanChunk || chunk % gridDim.x == blockIdx.x;
    if (blockIdx.x != 0 && tok >= t1 && a.B > kPlanChunk) {
      int next = chunk;  // the next chunk whose rows this block writes
      while (next % gridDim.x != blockIdx.x) ++next;
      if ((int64_t)next * kPlanChunk >= a.B) break;
    }
    const int nb = min(kPlanChunk, a.B - b0);
    int64_t my_tok[kPlanPer], my_pg[kPlanPer], sum_tok = 0, sum_pg = 0;
    int ctx_of[kPlanPer] = {}, kv_of[kPlanPer] = {};
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      const int i = tid * kPlanPer + k;
      my_tok[k] = sum_tok;
      my_pg[k] = sum_pg;
      if (i < nb) {
        const PlanSeq s = plan_seq(a, b0 + i, &bad);
        sum_tok += s.n;
        sum_pg += s.take;
        ctx_of[k] = (int)s.ctx;
        kv_of[k] = (int)s.kv;
        if (a.parent && s.n > 64 && blockIdx.x == 0) set_status(a.status, MLA_ERR_TREE);
      }
    }
    if (bad && blockIdx.x == 0) set_status(a.status, MLA_ERR_KVLEN);
    int64_t inc_tok = sum_tok, inc_pg = sum_pg;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc_tok, o);
      const int64_t y = __shfl_up_sync(0xffffffffu, inc_pg, o);
      if (lane >= o) {
        inc_tok += x;
        inc_pg += y;
      }
    }
    __syncthreads();  // the previous chunk's sums have been used
    if (lane == 31) {
      s_warp[0][warp] = inc_tok;
      s_warp[1][warp] = inc_pg;
    }
    __syncthreads();
    int64_t base_tok = tok, base_pg = pg;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) {
        base_tok += s_warp[0][w];
        base_pg += s_warp[1][w];
      }
      tok += s_warp[0][w];
      pg += s_warp[1][w];
    }
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
      s_tok[tid * kPlanPer + k] = base_tok + inc_tok - sum_tok + my_tok[k];
      s_pg[tid * kPlanPer + k] = base_pg + inc_pg - sum_pg + my_pg[k];
      s_ctx[tid * kPlanPer + k] = ctx_of[k];
      s_kv[tid * kPlanPer + k] = kv_of[k];
    }
    if (tid == 0) s_tok[kPlanChunk] = tok;
    __syncthreads();

    // Per sequence: cu_q, kv_len and the fresh table entries.
    const auto take_of = [&](int i) { return pages_of(a, s_kv[i]) - pages_of(a, s_ctx[i]); };
    const auto lengths = [&](int i) {
      a.cu_q[b0 + i] = (int)min(s_tok[i], (int64_t)a.T);
      a.kv_len[b0 + i] = s_kv[i];
    };
    const auto fill = [&](int i, int k0, int step) {  // entries k0, k0 + step, ..
      const int have = pages_of(a, s_ctx[i]), take = pages_of(a, s_kv[i]) - have;
      int32_t* row = a.block_table + (int64_t)(b0 + i) * a.max_pages + have;
      bool none = false;
      for (int k = k0; k < take; k += step) {
        const int page = plan_page(a, head, s_pg[i] + k);
        row[k] = page;
        none |= page < 0;
      }
      if (none) set_status(a.status, MLA_ERR_PAGE);
    };
    if (a.B <= kPlanChunk) {
      // A single chunk is shared among the warps of all blocks, several to a sequence where its
      // table is long (a sequence of a million tokens: 9 us, 85 by one warp).
      const int w = blockIdx.x * (kPlanThreads / 32) + warp;
      const int warps = gridDim.x * (kPlanThreads / 32);
      const int parts = max(min(warps / nb, (a.max_pages + 255) / 256), 1);
      for (int i = w; i < nb * parts; i += warps) {
        if (i < nb && lane == 0) lengths(i);
        fill(i % nb, i / nb * 32 + lane, parts * 32);
      }
    } else if (rows_mine) {
      // Of many sequences most take few pages: a thread each, and the whole warp for the others
      // (4096 of one token: 15 us, 35 with a warp each).
      for (int i0 = 0; i0 < nb; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const bool few = i < nb && take_of(i) <= 4;
        if (i < nb) lengths(i);
        if (few) fill(i, 0, 1);
        for (uint32_t m = __ballot_sync(0xffffffffu, i < nb && !few); m != 0; m &= m - 1)
          fill(i0 + warp * 32 + __ffs(m) - 1, lane, 32);
      }
    }

    // Per token: the sequences of this chunk that reach into [t0, t1).
    const int64_t lo = max(t0, s_tok[0] / kPlanTok * kPlanTok), hi = min(t1, tok);
    for (int64_t turn = lo; turn < hi; turn += kPlanThreads * kPlanTok) {
      if (a.parent) {  // a path lies within the 64 tokens before its end
        __syncthreads();
        for (int i = tid; i < 64 + kPlanThreads * kPlanTok; i += kPlanThreads) {
          const int64_t at = turn - 64 + i;
          s_par[i] = at >= 0 && at < hi ? a.parent[at] : -1;
        }
        __syncthreads();
      }
      const int64_t t = turn + tid * kPlanTok;
      if (t >= hi) continue;
      int l = 0, r = nb;  // the last sequence of the chunk that starts at or before the token
      const int64_t tf = max(t, s_tok[0]);
      while (r - l > 1) {
        const int m = (l + r) >> 1;
        if (s_tok[m] <= tf) l = m; else r = m;
      }
      int ctx = 0, kv = 0, have = 0;
      int64_t end = -1;   // first token past sequence l
      int page = -1, page_k = -1;
      int slot[kPlanTok], pos[kPlanTok];
      int64_t mask[kPlanTok];
      bool whole = true;  // all tokens of the group belong to this chunk
      bool bad_tree = false, bad_page = false;
#pragma unroll
      for (int e = 0; e < kPlanTok; ++e) {
        slot[e] = -1; pos[e] = 0; mask[e] = 0;
        const int64_t te = t + e;
        if (te < s_tok[0] || te >= hi) {
          whole = false;
          continue;
        }
        while (te >= end) {  // skips sequences without new tokens
          if (end >= 0) ++l;
          end = l + 1 < nb ? s_tok[l + 1] : tok;
          if (te < end) {
            ctx = s_ctx[l];
            kv = s_kv[l];
            have = pages_of(a, ctx);
            page_k = -1;
          }
        }
        const int64_t i = te - s_tok[l];
        const int64_t p = ctx + i;
        if (p < kv) {
          const int k = (int)(p >> a.page_shift);
          if (k != page_k) {
            page_k = k;
            if (k >= have) {
              page = plan_page(a, head, s_pg[l] + k - have);
            } else {
              page = a.block_table[(int64_t)(b0 + l) * a.max_pages + k];
              if (page < 0 || page >= a.num_pages) {
                page = -1;
                bad_page = true;
              }
            }
          }
          if (page >= 0) slot[e] = (page << a.page_shift) + (int)(p & (psize - 1));
        }
        int64_t depth = i;
        if (a.parent) {
          // Up the path to the root; indexes fall at every step, so the walk ends.
          const int first = (int)(s_tok[l] - (turn - 64));  // >= 1 where i < 64
          uint64_t m = 0;
          depth = -1;
          int at = (int)i;
          if (i < 64) {
            for (;;) {
              m |= 1ull << at;
              ++depth;
              const int up = s_par[first + at];
              if (up < 0 || up >= at) {
                bad_tree |= up != -1;
                break;
              }
              at = up;
            }
          } else {
            depth = 0;
          }
          mask[e] = (int64_t)m;
        }
        pos[e] = (int)min(ctx + depth, last_pos);
      }
      if (whole) {
        *reinterpret_cast<int4*>(a.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (a.parent) {
          reinterpret_cast<longlong2*>(a.draft_mask + t)[0] = make_longlong2(mask[0], mask[1]);
          reinterpret_cast<longlong2*>(a.draft_mask + t)[1] = make_longlong2(mask[2], mask[3]);
        }
      } else {
        for (int e = 0; e < kPlanTok; ++e) {
          if (t + e < s_tok[0] || t + e >= hi) continue;
          a.slots[t + e] = slot[e];
          a.positions[t + e] = pos[e];
          if (a.parent) a.draft_mask[t + e] = mask[e];
        }
      }
      if (bad_tree) set_status(a.status, MLA_ERR_TREE);
      if (bad_page) set_status(a.status, MLA_ERR_PAGE);
    }
  }

  if (blockIdx.x == 0 && tid == 0) {
    if (tok > a.T) set_status(a.status, MLA_ERR_KVLEN);
    a.cu_q[a.B] = (int)min(tok, (int64_t)a.T);
    a.free_next[0] = (int)min(head + pg, (int64_t)a.n_free);
  }
  // Rows behind the last sequence.  A block that broke off above has none: its tokens lie
  // before the running total.
  for (int64_t t = max(t0, tok) + tid; t < t1; t += kPlanThreads) {
    a.slots[t] = -1;
    a.positions[t] = 0;
    if (a.parent) a.draft_mask[t] = 0;
  }
}

// ---- append -----------------------------------------------------------------------------
// One pass over the new rows, bound by HBM: per token 2304 bytes of latent row and rotary key
// in and out, and 256 H bytes of query.  The work is cut into 16-byte pieces: 4 H per token of
// the queries and 4 of the rotary key, each a pair of them (columns c .. c+7 and c+32 .. c+39, so
// that one thread rotates both and may write over its own input), and 64 of the latent row.  A
// thread takes kPer pieces a block apart, all loads before the first use: four of them, or one
// where that leaves SMs without a block.  Inputs, and the queries of a large call, are streamed
// past the caches: 16411 tokens of 64 heads take 48 us, 6.5 TB/s (62 with one token per block,
// 53 with plain stores).
constexpr int kAppThreads = 256;
constexpr int kRowPieces = 64 + 4;

struct Pair8 {
  uint4 lo, hi;
};
__device__ __forceinline__ Pair8 load_pair(const uint16_t* p) {
  return {__ldcs(reinterpret_cast<const uint4*>(p)), __ldcs(reinterpret_cast<const uint4*>(p + 32))};
}
// Rotates columns c .. and c + 32 .. by a row of the cos | sin table (null: as they are).
template <bool kStream>
__device__ __forceinline__ void store_rotated(const Pair8& x, uint16_t* dst, int c,
                                              const float* cs) {
  Pair8 y = x;
  if (cs) {
    float cosv[8], sinv[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      *reinterpret_cast<float4*>(cosv + 4 * k) = *reinterpret_cast<const float4*>(cs + c + 4 * k);
      *reinterpret_cast<float4*>(sinv + 4 * k) =
          *reinterpret_cast<const float4*>(cs + 32 + c + 4 * k);
    }
    y.lo = rope_rotate8(x.lo, x.hi, cosv, sinv, false);
    y.hi = rope_rotate8(x.hi, x.lo, cosv, sinv, true);
  }
  if constexpr (kStream) {
    __stcs(reinterpret_cast<uint4*>(dst), y.lo);
    __stcs(reinterpret_cast<uint4*>(dst + 32), y.hi);
  } else {
    *reinterpret_cast<uint4*>(dst) = y.lo;
    *reinterpret_cast<uint4*>(dst + 32) = y.hi;
  }
}
// The table row of token t (clamped to the table), or null without a table.
__device__ __forceinline__ const float* table_row(const LatentAppendArgs& a, int t) {
  if (!a.rope_table) return nullptr;
  const int raw = a.positions[t];
  const int p = min(max(raw, 0), a.table_rows - 1);
  if (p != raw) set_status(a.status, MLA_ERR_KVLEN);
  return a.rope_table + (size_t)p * 64;
}

template <int kPer>
__global__ void __launch_bounds__(kAppThreads) latent_append_kernel(const LatentAppendArgs a) {
  const bool rows = blockIdx.x >= a.q_blocks;  // latent rows and rotary keys, or queries
  const int per = rows ? kRowPieces : 4 * a.H;  // pieces per token
  const int64_t first = (int64_t)(rows ? blockIdx.x - a.q_blocks : blockIdx.x) * (kAppThreads * kPer);
  const int t0 = (int)(first / per), rem = (int)(first - (int64_t)t0 * per);
  int tok[kPer], piece[kPer], slot[kPer];
  Pair8 x[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int at = rem + k * kAppThreads + threadIdx.x;
    tok[k] = t0 + at / per;
    piece[k] = at % per;
    slot[k] = tok[k] < a.T ? a.slots[tok[k]] : -1;
    if (slot[k] >= a.rows && rows) {
      set_status(a.status, MLA_ERR_PAGE);
      slot[k] = -1;
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (slot[k] < 0) continue;
    if (!rows)
      x[k] = load_pair(a.q_pe + ((size_t)tok[k] * a.H + (piece[k] >> 2)) * 64 + (piece[k] & 3) * 8);
    else if (piece[k] < 64)
      x[k].lo = __ldcs(reinterpret_cast<const uint4*>(a.c_new + (size_t)tok[k] * 512) + piece[k]);
    else
      x[k] = load_pair(a.pe_new + (size_t)tok[k] * 64 + (piece[k] - 64) * 8);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (slot[k] < 0) continue;
    if (!rows) {
      const int c = (piece[k] & 3) * 8;
      store_rotated<(kPer > 1)>(x[k], a.q_pe_out + ((size_t)tok[k] * a.H + (piece[k] >> 2)) * 64 + c, c,
                    table_row(a, tok[k]));
    } else if (piece[k] < 64) {
      reinterpret_cast<uint4*>(a.c_pages + (size_t)slot[k] * 512)[piece[k]] = x[k].lo;
    } else {
      const int c = (piece[k] - 64) * 8;
      store_rotated<false>(x[k], a.pe_pages + (size_t)slot[k] * 64 + c, c, table_row(a, tok[k]));
    }
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t stream) {
  // Enough blocks for one group of tokens per thread, or one warp per sequence, within four
  // blocks per SM (each repeats the scan).
  const int sms = device_sm_count();
  const int64_t by_tok = ((int64_t)a.T + kPlanThreads * kPlanTok - 1) / (kPlanThreads * kPlanTok);
  const int64_t by_seq = ((int64_t)std::min(a.B, kPlanChunk) + 7) / 8;
  const int64_t grid = std::min<int64_t>(std::max(by_tok, by_seq), 4 * (sms > 0 ? sms : 152));
  paged_plan_kernel<<<(unsigned)grid, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_latent_append(const LatentAppendArgs& args, cudaStream_t stream) {
  LatentAppendArgs a = args;
  const int64_t q_pieces = (int64_t)a.T * 4 * a.H, row_pieces = (int64_t)a.T * kRowPieces;
  const int sms = device_sm_count();
  const bool small = q_pieces + row_pieces < (int64_t)(sms > 0 ? sms : 152) * kAppThreads * 4;
  const int per = kAppThreads * (small ? 1 : 4);
  a.q_blocks = (unsigned)((q_pieces + per - 1) / per);
  const int64_t blocks = a.q_blocks + (row_pieces + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (small)
    latent_append_kernel<1><<<(unsigned)blocks, kAppThreads, 0, stream>>>(a);
  else
    latent_append_kernel<4><<<(unsigned)blocks, kAppThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
