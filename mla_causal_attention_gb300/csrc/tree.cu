// tree.cu -- attention of packed new tokens over the paged latent cache.
//
// For new token t of sequence b and head h, over the keys j the token sees,
//   s_j = scale * (q_lat[t,h] . c_j + q_pe[t,h] . k_pe_j),   q_lat = W_K[h]^T q_nope
//   out = W_V[h] (sum_j softmax(s)_j c_j)
// (the up-projection kv_b_proj folded into the query and applied once to the mix).
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

// The keys of a sequence and the part of them that are new tokens, clamped for safety.
struct TreeSeq {
  int q0, n, kv, ctx;
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool* bad) {
  const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], k = a.kv_len[b];
  TreeSeq s;
  s.q0 = min(max(c0, 0), a.T);
  s.n = min(max(c1, s.q0), a.T) - s.q0;
  s.kv = (int)min((int64_t)max(k, 0), (int64_t)a.max_pages << a.page_shift);
  s.ctx = max(s.kv - s.n, 0);
  if (s.q0 != c0 || s.q0 + s.n != c1 || s.kv != k || s.kv < s.n) *bad = true;
  return s;
}

// One block per (token, head): warps take keys in turn, lane l holds latent columns
// 16 l .. 16 l + 15 and rotary columns 2 l, 2 l + 1.
__global__ void __launch_bounds__(kWarps * 32) latent_tree_kernel(const TreeArgs a) {
  __shared__ float s_acc[kWarps][512];
  __shared__ float s_m[kWarps], s_l[kWarps];
  const int t = blockIdx.x, h = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int lo = 0, hi = a.B;  // the last sequence that starts at or before t
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.cu_q[m] <= t) lo = m; else hi = m;
  }
  const int b = lo;
  bool bad = false;
  const TreeSeq s = tree_seq(a, b, &bad);
  if (bad && tid == 0) set_status(a.status, MLA_ERR_KVLEN);
  if (t < s.q0 || t >= s.q0 + s.n) return;
  if (a.draft_mask && s.n > 64 && tid == 0) set_status(a.status, MLA_ERR_TREE);
  const int i = t - s.q0;
  const uint64_t mask = a.draft_mask ? (uint64_t)a.draft_mask[t] : 0;
  const size_t row = (size_t)t * a.H + h;
  float q[16], qr[2], acc[16], m = -INFINITY, l = 0.f;
  for (int k = 0; k < 16; ++k) {
    q[k] = __uint_as_float((uint32_t)a.q_lat[row * 512 + lane * 16 + k] << 16);
    acc[k] = 0.f;
  }
  for (int k = 0; k < 2; ++k)
    qr[k] = __uint_as_float((uint32_t)a.q_pe[row * 64 + lane * 2 + k] << 16);
  for (int j = warp; j < s.kv; j += kWarps) {
    if (j >= s.ctx) {
      const int k = j - s.ctx;
      if (a.draft_mask ? (k > 63 || !((mask >> k) & 1)) : k > i) continue;
    }
    const int page = a.block_table[(size_t)b * a.max_pages + (j >> a.page_shift)];
    const bool in = page >= 0 && page < a.num_pages;
    if (!in && lane == 0) set_status(a.status, MLA_ERR_PAGE);
    const size_t slot = ((size_t)(in ? page : 0) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
    float c[16], dot = 0.f;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.c_pages + slot * 512 + lane * 16);
    for (int k = 0; k < 8; ++k) {
      const uint32_t w = in ? src[k] : 0u;
      c[2 * k] = bf16lo_to_f32(w);
      c[2 * k + 1] = bf16hi_to_f32(w);
      dot += q[2 * k] * c[2 * k] + q[2 * k + 1] * c[2 * k + 1];
    }
    const uint32_t pe = in ? reinterpret_cast<const uint32_t*>(a.pe_pages + slot * 64)[lane] : 0u;
    dot += qr[0] * bf16lo_to_f32(pe) + qr[1] * bf16hi_to_f32(pe);
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float x = dot * a.scale_log2;
    const float m2 = fmaxf(m, x);
    const float f = ex2_approx(m - m2), p = ex2_approx(x - m2);
    l = l * f + p;
    for (int k = 0; k < 16; ++k) acc[k] = acc[k] * f + p * c[k];
    m = m2;
  }
  for (int k = 0; k < 16; ++k) s_acc[warp][lane * 16 + k] = acc[k];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  const float base = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) total += s_l[w] * ex2_approx(s_m[w] - base);
  const float inv = total > 0.f ? 1.f / total : 0.f;
  float mix[2];
  for (int k = 0; k < 2; ++k) {
    mix[k] = 0.f;
    for (int w = 0; w < kWarps; ++w)
      mix[k] += s_acc[w][tid + 256 * k] * ex2_approx(s_m[w] - base);
  }
  __syncthreads();
  for (int k = 0; k < 2; ++k) s_acc[0][tid + 256 * k] = mix[k] * inv;
  __syncthreads();
  if (tid < 128) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(a.w_kvb + ((size_t)h * 256 + 128 + tid) * 512);
    float y = 0.f;
    for (int k = 0; k < 256; ++k)
      y += bf16lo_to_f32(w[k]) * s_acc[0][2 * k] + bf16hi_to_f32(w[k]) * s_acc[0][2 * k + 1];
    a.out[row * 128 + tid] = (uint16_t)(pack_bf16x2(y, 0.f) & 0xffffu);
  }
}

}  // namespace

cudaError_t launch_latent_tree(const TreeArgs& a, cudaStream_t stream) {
  LatentArgs l{};
  l.q_nope = a.q_nope;
  l.w_kvb = a.w_kvb;
  l.q_lat = a.q_lat;
  l.B = a.T;
  l.H = a.H;
  const cudaError_t e = launch_latent_absorb(l, stream);
  if (e != cudaSuccess) return e;
  latent_tree_kernel<<<dim3((unsigned)a.T, (unsigned)a.H), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mla
