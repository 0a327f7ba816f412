// tree_proj.cu -- before and after the tree attention's split kernel: the query folded into the
// latent space (with the partition of the work), the merge of partial mixes, and the mix projected
// up, out = W_V mix.
//
// The two projections are one batched GEMM, a matrix per head:
//   fold  q_lat[t,h,:] = q_nope[t,h,:] W_K[h]      [T x 128] . [128 x 512]
//   up    out[t,h,:]   = mix[t,h,:] W_V[h]^T       [T x 512] . [512 x 128]
// with W_K[h], W_V[h] the first and second 128 rows of head h's 256 of kv_b_proj.  A block keeps
// its head's 128 KB of weight in shared memory and takes 128 tokens at a time: rows by TMA through
// a ring, MMAs into one of two TMEM tiles while the epilogue warps read the other.  Bound by the
// rows' traffic (1280 bytes per token and head for each); with mma.sync, whose fragments come from
// shared memory over and over, the two took 53 and 106 us for 1024 tokens and 64 heads.
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

constexpr int kLD = 512;
constexpr int kM = 128;               // tokens per tile
constexpr int kSub = 128 * 128;       // 128 rows x 64 columns, bf16, 128-byte swizzled
// Up to this many tokens the up-projection's blocks merge the partial mixes of their rows
// themselves, two rows per warp, which saves a kernel between two others (8 drafted tokens on 1000
// keys: 27.9 -> 23.0 us); with more, the merge's blocks all over the GPU are faster.
constexpr int kMergeTokens = 16;
constexpr int kMaxSlots = 5;          // ring of the rows' sub-tiles: 5, or 3 with 32 KB of output
constexpr int kOffRing = 8 * kSub;    // staging behind it; behind the weight's 8 sub-tiles
constexpr int kOffBar = kOffRing + kMaxSlots * kSub;
constexpr int kSmem = kOffBar + 256 + 1024;
static_assert(kSmem <= 232448 && kPartSmem <= kSmem, "shared memory per block");

struct ProjParams {
  CUtensorMap tm_x;  // rows    {K, T, H}, boxes {64, 128, 1}
  CUtensorMap tm_w;  // w_kvb   {512, H * 256}, boxes {64, 128}
  CUtensorMap tm_y;  // fold: q_lat {512, T, H}, boxes {64, 32, 1}; in two parts {1024, T, H}
  TreeArgs a;
  KeySteps steps;    // fold in two parts: what its last block but one makes
  int blocks_y;      // blocks per head and part along the tokens
  int parts;         // parts of the output columns, a block each: 1, or (few tokens) 2
  int merge;         // up: the blocks merge their rows themselves (up to kMergeTokens tokens)
};
struct PBars {
  uint64_t w_full;
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t d_full[2], d_free[2];  // accumulator tiles (d_free: 4 epilogue warps)
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(PBars) <= 256, "barrier block");

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]),
                 "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Merges row r of the unit that begins in slot s0: sum 2^(m_s - m) acc_s / sum 2^(m_s - m) l_s over
// its segments, to bf16, the up-projection's operand type.  A unit's segments lie in the slots of
// successive pairs: from the one marked first, each next pair's first slot (pairs without work
// have empty ones) to the one marked last.  One warp; lane owns columns 4 lane + 128 k.
__device__ __forceinline__ void merge_row(const TreeArgs& a, const int4* note, int s0, int r,
                                          int lane, uint2 (&w)[4]) {
  const int slots = 2 * a.pairs;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  bool last = false;
  for (int s = s0; !last && s < slots;) {  // up to 32 segments a round, lane i the i-th
    int slot = -1;
    for (int k = 0; k < 32 && !last && s < slots; s = (s | 1) + 1) {
      if (note[s].y == 0) continue;
      if (lane == k) slot = s;
      last = note[s].w != 0;
      ++k;
    }
    float2 ml = make_float2(-INFINITY, 0.f);
    if (slot >= 0) ml = reinterpret_cast<const float2*>(a.part_ml)[(size_t)slot * kRows + r];
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m2 = fmaxf(m, top), base = m2 == -INFINITY ? 0.f : m2;
    const float f0 = ex2_approx(m - base), f = ex2_approx(ml.x - base);
    float sum = ml.y * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f0 + sum;
    m = m2;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[k].x *= f0;
      acc[k].y *= f0;
      acc[k].z *= f0;
      acc[k].w *= f0;
    }
    const int have = __popc(__ballot_sync(0xffffffffu, slot >= 0));
    for (int k0 = 0; k0 < have; k0 += 4) {  // four partials' rows in flight
      float4 v[4][4];
      float fu[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = min(k0 + e, have - 1);
        const float x = __shfl_sync(0xffffffffu, f, at);
        const int sl = __shfl_sync(0xffffffffu, slot, at);
        fu[e] = k0 + e < have ? x : 0.f;
        const float4* src =
            reinterpret_cast<const float4*>(a.part_acc + ((size_t)sl * kRows + r) * kLD) + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[e][k] = k0 + e < have ? src[32 * k] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc[k].x = fmaf(fu[e], v[e][k].x, acc[k].x);
          acc[k].y = fmaf(fu[e], v[e][k].y, acc[k].y);
          acc[k].z = fmaf(fu[e], v[e][k].z, acc[k].z);
          acc[k].w = fmaf(fu[e], v[e][k].w, acc[k].w);
        }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv),
                      pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
}

// kUp: K = 512 in 8 sub-tiles, N = 128, weight K-major.  Fold: K = 128 in 2 sub-tiles, N = 512 in
// two blocks of 256, weight MN-major (its rows are the contraction).  Up to 128 tokens there is
// one block per head, most SMs are idle and the weight's load is the critical path: the fold's
// two column blocks then go to two blocks.
// Warps: 0 TMA, 1 MMA, 4-7 epilogue.  The fold launch has one block more, which makes the partition.
// It is the last: where the others fill every SM (8 heads from 2305 tokens on) it runs behind one of
// them, about 2 us of 35.
// kTwo (a fold): the result in two parts, and one block more, for the key weights' partition.
template <bool kUp, bool kTwo = false>
__global__ void __launch_bounds__(256, 1) tree_proj_kernel(const __grid_constant__ ProjParams p) {
  static_assert(!(kUp && kTwo), "two parts are a fold's");
  constexpr int kKs = kUp ? 8 : 2, kNb = kUp ? 1 : 2, kN = kUp ? 128 : 256;
  constexpr uint32_t kSlots = kUp ? 5 : 3;
  grid_dep_launch();
  const TreeArgs& a = p.a;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  if (!kUp && blockIdx.x == gridDim.x - 1) {
    tree_partition(a, smem_raw);
    return;
  }
  if (kTwo && blockIdx.x == gridDim.x - 2) {
    key_steps(a, p.steps);
    return;
  }
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sW = smem;
  uint8_t* sX = smem + kOffRing;
  PBars* bars = reinterpret_cast<PBars*>(smem + kOffBar);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % p.parts;
  const int h = blockIdx.x / p.parts / p.blocks_y, y = blockIdx.x / p.parts % p.blocks_y;
  const int nb0 = p.parts == 2 ? part : 0, nb1 = p.parts == 2 ? part + 1 : kNb;
  if (threadIdx.x == 0) {
    mbar_init(&bars->w_full, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->d_full[i], 1);
      mbar_init(&bars->d_free[i], 4);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = bars->tmem_base;
  // The weight is no kernel's output: it is on its way before the kernel in front is waited for.
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.tm_x);
    if (!kUp) prefetch_tmap(&p.tm_y);
    const int s0 = kUp ? 0 : 4 * nb0, s1 = kUp ? 8 : 4 * nb1;
    mbar_arrive_expect_tx(&bars->w_full, (s1 - s0) * kSub);
    for (int s = s0; s < s1; ++s)
      tma_load_2d(sW + s * kSub, &p.tm_w, &bars->w_full, 64 * s, h * 256 + (kUp ? 128 : 0));
  }
  if (kUp) grid_dep_wait();
  // Rows in front of the first sequence and behind the last are left as they are.
  const int row0 = kUp ? min(max(a.cu_q[0], 0), a.T) : 0;
  const int rows = kUp ? min(max(a.cu_q[a.B], 0), a.T) : a.T;
  const int tiles = (rows + kM - 1) / kM;
  const bool merge = kUp && p.merge;
  // Rows merged by this block lie 2 KB per sub-tile: what an MMA reads behind row 16 is another
  // sub-tile's, and goes into rows of the result that do not exist.
  constexpr int kMergeSub = kMergeTokens * 128;
  if (merge) {
    int4* note = reinterpret_cast<int4*>(sX + 4 * kSub);
    for (int i = threadIdx.x; i < 2 * a.pairs; i += 256) note[i] = a.part_note[i];
    __syncthreads();
    for (int t = warp; t < rows; t += 8) {
      const int row = t * a.H + h;
      int s0 = -1;  // the slot that begins the row's unit, if it was shared
      for (int i = lane; i < 2 * a.pairs; i += 32)
        if (note[i].z != 0 && row >= note[i].x && row < note[i].x + note[i].y) s0 = i;
      s0 = __reduce_max_sync(0xffffffffu, s0);
      uint2 w[4];
      if (s0 >= 0) {
        merge_row(a, note, s0, row - note[s0].x, lane, w);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = *reinterpret_cast<const uint2*>(a.q_lat + (size_t)row * kLD + 4 * lane + 128 * k);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint2*>(sX + (2 * k + (lane >> 4)) * kMergeSub + t * 128 +
                                  ((((lane & 15) >> 1) ^ (t & 7)) << 4) + 8 * (lane & 1)) = w[k];
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }

  if (warp == 0) {
    if (lane == 0 && merge) drain(&bars->w_full, 0);
    if (lane == 0 && !merge) {
      uint32_t u = 0;
      bool ok = true;
      for (int i = y; i < tiles && ok; i += p.blocks_y)
        for (int s = 0; s < kKs && ok; ++s, ++u) {
          const uint32_t slot = u % kSlots, n = u / kSlots;
          if (n > 0) ok = mbar_wait(&bars->empty[slot], (n - 1) & 1, a.status, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars->full[slot], kSub);
          tma_load_3d_nohint(sX + slot * kSub, &p.tm_x, &bars->full[slot], 64 * s, i * kM, h);
        }
      // Every copy has landed before shared memory is given up.
      drain(&bars->w_full, 0);
      for (uint32_t k = u > kSlots ? u - kSlots : 0; k < u; ++k)
        drain(&bars->full[k % kSlots], (k / kSlots) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t kId = tc::idesc_bf16_f32(128, kN, !kUp);
    const uint64_t d_x = tc::smem_desc_sw128(0, 16, 1024);
    const uint64_t d_w = tc::smem_desc_sw128(0, kUp ? 16 : kSub, 1024);
    const uint32_t x_lo = smem_u32(sX) >> 4, w_lo = smem_u32(sW) >> 4;
    uint32_t u = 0, d = 0;  // sub-tiles, accumulator tiles
    bool ok = __all_sync(0xffffffffu, mbar_wait(&bars->w_full, 0, a.status, abort_flag));
    for (int i = y; i < tiles && ok; i += p.blocks_y) {
      for (int nb = nb0; nb < nb1 && ok; ++nb, ++d) {
        if (d > 1) ok = mbar_wait(&bars->d_free[d & 1], ((d >> 1) - 1) & 1, a.status, abort_flag);
#pragma unroll 1
        for (int s = 0; s < kKs; ++s) {
          const uint32_t slot = (u + s) % kSlots, n = (u + s) / kSlots;
          if (!merge) ok = ok && mbar_wait(&bars->full[slot], n & 1, a.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              // up: sub-tile s of the weight, K-major; fold: rows 64 s + 16 kk .. of the weight,
              // MN-major, columns 256 nb .. in four sub-tiles
              const uint32_t w_at =
                  kUp ? w_lo + s * (kSub >> 4) + 2 * kk
                      : w_lo + 4 * nb * (kSub >> 4) + (4 * s + kk) * (2048 >> 4);
              const uint32_t x_at = merge ? s * (kMergeSub >> 4) : slot * (kSub >> 4);
              tc::mma_ss(tbase + (d & 1) * 256, d_x | (uint64_t)(x_lo + x_at + 2 * kk),
                         d_w | (uint64_t)w_at, kId, (s | kk) != 0 ? 1u : 0u);
            }
            if (nb == nb1 - 1) tc::commit(&bars->empty[slot]);
            if (s == kKs - 1) tc::commit(&bars->d_full[d & 1]);
          }
          __syncwarp();
        }
      }
      u += kKs;
    }
    // No MMA runs on when TMEM is released: the last tiles are waited for.
    if (ok)
      for (uint32_t k = d > 2 ? d - 2 : 0; k < d; ++k) drain(&bars->d_full[k & 1], (k >> 1) & 1);
    else if (tc::elect_one())
      tc::commit(&bars->w_full), drain(&bars->w_full, 1);
    __syncwarp();
  } else if (warp >= 4) {
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int r = (warp & 3) * 32 + lane;
    uint32_t d = 0;
    bool ok = true;
    for (int i = y; i < tiles && ok; i += p.blocks_y)
      for (int nb = nb0; nb < nb1 && ok; ++nb, ++d) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&bars->d_full[d & 1], (d >> 1) & 1, a.status, abort_flag));
        if (!ok) break;
        tc::fence_after_sync();
        const auto take = [&](int c, uint32_t (&o)[32], bool last) {  // columns 32 c ..
          tc::tmem_ld32(tbase + lane_off + (d & 1) * 256 + c * 32, o);
          tc::tmem_wait_ld();
          pin<32>(o);
          if (last) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->d_free[d & 1]);
          }
        };
        const auto pack8 = [](const uint32_t (&o)[32], int e) {  // columns 8 e .. of the 32
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]),
                               __uint_as_float(o[8 * e + 2 * k + 1]));
          return make_uint4(w[0], w[1], w[2], w[3]);
        };
        if constexpr (kUp) {
          const int t = i * kM + r;
          uint16_t* dst = a.out + ((size_t)t * a.H + h) * 128;
#pragma unroll 1
          for (int c = 0; c < kN / 32; ++c) {
            uint32_t o[32];
            take(c, o, c == kN / 32 - 1);
            if (t >= row0 && t < rows)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(dst + c * 32 + 8 * e) = pack8(o, e);
          }
        } else {
          // 64 columns of this warp's 32 rows at a time through one of its two 4 KB stages and a
          // tensor store (lanes writing their own rows touch 32 lines per instruction).
          const auto store = [&](const uint8_t* stage, int col) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              // A group for every stage, also where all its rows lie behind T: the wait for a free
              // stage counts groups.
              if (i * kM + (warp & 3) * 32 < a.T)
                tma_store_3d(&p.tm_y, stage, col, i * kM + (warp & 3) * 32, h);
              bulk_commit_group();
            }
          };
#pragma unroll 1
          for (int c = 0; c < kN / 64; ++c) {
            uint8_t* stages = smem + kOffRing + kSlots * kSub + (warp & 3) * 2 * 4096;
            if constexpr (kTwo) {
              uint32_t o[2][32];
              take(2 * c, o[0], false);
              take(2 * c + 1, o[1], c == kN / 64 - 1);
#pragma unroll
              for (int part = 0; part < 2; ++part) {
                if (lane == 0) bulk_wait_read_but_one();  // this part's last store has read the stage
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    *reinterpret_cast<uint4*>(stages + part * 4096 + lane * 128 +
                                              (((4 * q + e) ^ (lane & 7)) << 4)) = pack8(o[q], e);
                    if (part == 0)
#pragma unroll
                      for (int k = 8 * e; k < 8 * e + 8; ++k) {  // what the rounding leaves, exactly
                        const float x = __uint_as_float(o[q][k]);
                        o[q][k] = __float_as_uint(x - bf16lo_to_f32(pack_bf16x2(x, 0.f)));
                      }
                  }
                store(stages + part * 4096, 512 * part + 256 * nb + 64 * c);
              }
            } else {
              uint8_t* stage = stages + (c & 1) * 4096;
              if (lane == 0) bulk_wait_read_but_one();  // the stage's last store has read it
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                uint32_t o[32];
                take(2 * c + q, o, c == kN / 64 - 1 && q == 1);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * q + e) ^ (lane & 7)) << 4)) =
                      pack8(o, e);
              }
              store(stage, 256 * nb + 64 * c);
            }
          }
        }
      }
    if (!kUp && lane == 0) bulk_wait_all();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, 512);
  }
}

// The merge as a kernel of its own: a block per slot and 8 rows, a warp per row; blocks of slots
// that no unit begins in end at once.  Bound by reading the partials.
constexpr int kMergeRows = 8;
__global__ void __launch_bounds__(32 * kMergeRows) tree_merge_kernel(const TreeArgs a) {
  grid_dep_launch();
  __shared__ int4 note[512];
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = 2 * a.pairs;
  const int s0 = blockIdx.x / (kRows / kMergeRows);
  const int r0 = (blockIdx.x % (kRows / kMergeRows)) * kMergeRows, r = r0 + warp;
  const int4 n0 = a.part_note[s0];
  if (n0.z == 0 || r0 >= n0.y) return;  // empty, no unit's first segment, or fewer rows
  for (int i = threadIdx.x; i < slots; i += 32 * kMergeRows) note[i] = a.part_note[i];
  __syncthreads();
  if (r >= n0.y) return;
  uint2 w[4];
  merge_row(a, note, s0, r, lane, w);
  uint16_t* dst = a.q_lat + ((size_t)n0.x + r) * kLD;
#pragma unroll
  for (int k = 0; k < 4; ++k) *reinterpret_cast<uint2*>(dst + 4 * lane + 128 * k) = w[k];
}

// Tensor maps, cached by pointers and sizes, two entries a call (see tree.cu).
struct MapKey {
  const void* x;
  const void* w;
  const void* y;
  int T, H, up, parts;
  bool operator==(const MapKey& o) const {
    return x == o.x && w == o.w && y == o.y && T == o.T && H == o.H && up == o.up &&
           parts == o.parts;
  }
};
struct MapEntry {
  MapKey key;
  CUtensorMap maps[3];
  bool valid;
};
std::mutex g_mu;
MapEntry g_maps[16];
int g_next = 0;

bool proj_maps(const TreeArgs& a, bool up, int parts, ProjParams* p) {
  const MapKey key = {up ? a.q_lat : a.q_nope, a.w_kvb, a.q_lat, a.T, a.H, up, parts};
  std::lock_guard<std::mutex> lk(g_mu);
  for (const MapEntry& e : g_maps)
    if (e.valid && e.key == key) {
      p->tm_x = e.maps[0];
      p->tm_w = e.maps[1];
      p->tm_y = e.maps[2];
      return true;
    }
  const uint64_t width = up ? kLD : 128;
  const uint64_t dims[3] = {width, (uint64_t)a.T, (uint64_t)a.H};
  const uint64_t strides[2] = {(uint64_t)a.H * width * 2, width * 2};
  const uint32_t box[3] = {64, kM, 1};
  const uint64_t wdims[2] = {kLD, (uint64_t)a.H * 256};
  const uint64_t wstrides[1] = {kLD * 2};
  const uint32_t wbox[2] = {64, 128};
  const uint64_t ywidth = (uint64_t)kLD * parts;
  const uint64_t ydims[3] = {ywidth, (uint64_t)a.T, (uint64_t)a.H};
  const uint64_t ystrides[2] = {(uint64_t)a.H * ywidth * 2, ywidth * 2};
  const uint32_t ybox[3] = {64, 32, 1};
  if (!encode_bf16_tiled(&p->tm_x, key.x, 3, dims, strides, box) ||
      !encode_bf16_tiled(&p->tm_w, key.w, 2, wdims, wstrides, wbox) ||
      !encode_bf16_tiled(&p->tm_y, a.q_lat, 3, ydims, ystrides, ybox))
    return false;
  MapEntry& e = g_maps[g_next];
  g_next = (g_next + 1) % 16;
  e.key = key;
  e.maps[0] = p->tm_x;
  e.maps[1] = p->tm_w;
  e.maps[2] = p->tm_y;
  e.valid = true;
  return true;
}

cudaError_t set_attributes() {
  static std::atomic<uint64_t> attr_done{0};  // bit per device: smem attributes set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (attr_done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(tree_proj_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(tree_proj_kernel<false, true>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(tree_proj_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmem);
  if (e != cudaSuccess) return e;
  attr_done.fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

// Blocks per head: as many as there are SMs for, and token tiles.
int blocks_per_head(const TreeArgs& a) {
  return std::min((a.T + kM - 1) / kM, std::max(1, 2 * a.pairs / a.H));
}

}  // namespace

cudaError_t launch_tree_fold(const TreeArgs& a, cudaStream_t stream) {
  cudaError_t e = set_attributes();
  if (e != cudaSuccess) return e;
  ProjParams p;
  if (!proj_maps(a, false, 1, &p)) return cudaErrorInvalidValue;
  p.a = a;
  p.blocks_y = blocks_per_head(a);
  p.parts = a.T <= kM && a.H <= a.pairs ? 2 : 1;
  p.merge = 0;
  tree_proj_kernel<false><<<a.H * p.blocks_y * p.parts + 1, 256, kSmem, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree_fold_two(const TreeArgs& a, const KeySteps& steps, cudaStream_t stream) {
  cudaError_t e = set_attributes();
  if (e != cudaSuccess) return e;
  ProjParams p;
  if (!proj_maps(a, false, 2, &p)) return cudaErrorInvalidValue;
  p.a = a;
  p.steps = steps;
  p.blocks_y = blocks_per_head(a);
  p.parts = a.T <= kM && a.H <= a.pairs ? 2 : 1;
  p.merge = 0;
  tree_proj_kernel<false, true><<<a.H * p.blocks_y * p.parts + 2, 256, kSmem, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree_up(const TreeArgs& a, cudaStream_t stream) {
  ProjParams p;
  if (!proj_maps(a, true, 1, &p)) return cudaErrorInvalidValue;
  p.a = a;
  p.blocks_y = blocks_per_head(a);
  p.parts = 1;
  p.merge = a.T <= kMergeTokens;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (!p.merge) {
    cfg.gridDim = dim3(2 * a.pairs * (kRows / kMergeRows));
    cfg.blockDim = dim3(32 * kMergeRows);
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel, a);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(a.H * p.blocks_y);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = kSmem;
  e = cudaLaunchKernelEx(&cfg, tree_proj_kernel<true>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
