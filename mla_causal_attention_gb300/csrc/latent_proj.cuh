// latent_proj.cuh -- the two small per-head projections of the latent paths: the query folded
// into the latent space before the attention, and the mix projected up after it.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace mla {
namespace proj {

constexpr int kLD = 512;           // latent width (kv_lora_rank)

// Warp-level bf16 MMA (m16n8k16, fp32 accumulate) for the two per-head projections: small
// GEMMs (64 sequences x 128 columns x 128, 64 x 32 x 512) whose operands sit in padded
// shared memory and are read with ldmatrix.  Fragments (g = lane / 4, c = lane % 4): A a0
// (row g, cols 2c, 2c+1), a1 (row g+8), a2 (cols + 8), a3 (row g+8, cols + 8); B b0 (rows
// k = 2c, 2c+1, col g), b1 (k + 8); C c0, c1 (row g, cols 2c, 2c+1), c2, c3 (row g+8).
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four 8x8 bf16 matrices from shared memory; lane l gives the row address of matrix l / 8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
// The same, each matrix transposed.
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_all;" ::: "memory");
}

constexpr int kPB = 64;            // sequences per projection CTA
constexpr int kAbN = 128;          // latent columns per absorb CTA
constexpr int kAbRow = 128 + 8;    // padded bf16 row (128 values) of the absorb operands
constexpr int kAbsorbSmem = (128 + kPB) * kAbRow * 2;
constexpr int kCuB = 32;           // sequences per merge + up-projection CTA
constexpr int kUpRow = kLD + 8;    // padded bf16 row (512 values)
constexpr int kCuSmem = (128 + kCuB) * kUpRow * 2;

// q_lat[b,h,n] = sum_k W_K[h][k][n] q_nope[b,h,k] for one head, a quarter of the 512 latent
// columns and 64 sequences: [64 x 128] . [128 x 128].  W_K[h] = rows h*256 .. h*256+127 of
// kv_b_proj (k = no-rope key dim, n = latent dim).  Warp w: row tile w % 4 (16 sequences),
// columns 64 (w / 4) .. +63.
__device__ __forceinline__ void absorb_block(const uint16_t* q_nope, const uint16_t* w_kvb,
                                             uint16_t* q_lat, int B, int H, int h, int n0,
                                             int b0) {
  extern __shared__ __align__(16) uint8_t ab_smem[];
  uint16_t* sw = reinterpret_cast<uint16_t*>(ab_smem);  // W_K slice: 128 rows (k) x 128 (n)
  uint16_t* sq = sw + 128 * kAbRow;                      // q_nope: 64 rows (b) x 128 (k)
  const int nb = min(kPB, B - b0);
  for (int i = threadIdx.x; i < 128 * 16; i += blockDim.x) {
    const int r = i >> 4, c = i & 15;
    cp_async16(sw + r * kAbRow + c * 8, w_kvb + ((size_t)h * 256 + r) * kLD + n0 + c * 8);
  }
  for (int i = threadIdx.x; i < kPB * 16; i += blockDim.x) {
    const int r = i >> 4, c = i & 15;
    if (r < nb)
      cp_async16(sq + r * kAbRow + c * 8, q_nope + ((size_t)(b0 + r) * H + h) * 128 + c * 8);
    else
      *reinterpret_cast<uint4*>(sq + r * kAbRow + c * 8) = make_uint4(0u, 0u, 0u, 0u);
  }
  cp_async_wait_all();
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = warp & 3, nh = warp >> 2;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  float acc[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
  for (int k0 = 0; k0 < 128; k0 += 16) {
    uint32_t af[4];
    ldsm4(af, sq + (mt * 16 + (lane & 15)) * kAbRow + k0 + (lane >> 4) * 8);
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      // B[k][n] row-major: transposed loads give two n-tiles' (b0, b1)
      uint32_t bf[4];
      ldsm4t(bf, sw + (k0 + (lane & 15)) * kAbRow + nh * 64 + np * 16 + (lane >> 4) * 8);
      mma16816(acc[2 * np], af, bf[0], bf[1]);
      mma16816(acc[2 * np + 1], af, bf[2], bf[3]);
    }
  }
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const int col = n0 + nh * 64 + n * 8 + c2;
    const int r = mt * 16 + g;
    if (r < nb)
      *reinterpret_cast<uint32_t*>(q_lat + ((size_t)(b0 + r) * H + h) * kLD + col) =
          pack_bf16x2(acc[n][0], acc[n][1]);
    if (r + 8 < nb)
      *reinterpret_cast<uint32_t*>(q_lat + ((size_t)(b0 + r + 8) * H + h) * kLD + col) =
          pack_bf16x2(acc[n][2], acc[n][3]);
  }
}

// W_V[h] (rows h*256+128 .. h*256+255 of kv_b_proj) on its way to padded shared memory.
__device__ __forceinline__ void up_load_weight(uint16_t* sw, const uint16_t* w_kvb, int h) {
  for (int i = threadIdx.x; i < 128 * (kLD / 8); i += blockDim.x) {
    const int r = i / (kLD / 8), c = i % (kLD / 8);
    cp_async16(sw + r * kUpRow + c * 8, w_kvb + ((size_t)h * 256 + 128 + r) * kLD + c * 8);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// [32 rows of so x 512] . [512 x 128 of sw]: warp w of 16 computes output columns
// 16 (w % 8) .. + 15 of row tile w / 8; row r < nb goes to out + r * out_stride.
__device__ __forceinline__ void up_project(const uint16_t* so, const uint16_t* sw, uint16_t* out,
                                           size_t out_stride, int nb) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const int mt = warp >> 3, nw = warp & 7;
  float acc[2][4];  // [column tile]
#pragma unroll
  for (int n = 0; n < 2; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll 4
  for (int k0 = 0; k0 < kLD; k0 += 16) {
    uint32_t af[4], bf[4];
    ldsm4(af, so + (mt * 16 + (lane & 15)) * kUpRow + k0 + (lane >> 4) * 8);
    // W_V rows are n with k contiguous (B column-major): matrices (n 0-7, k0), (n 0-7,
    // k0+8), (n 8-15, k0), (n 8-15, k0+8)
    ldsm4(bf, sw + (nw * 16 + (lane & 7) + ((lane >> 4) << 3)) * kUpRow + k0 +
                   ((lane >> 3) & 1) * 8);
    mma16816(acc[0], af, bf[0], bf[1]);
    mma16816(acc[1], af, bf[2], bf[3]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int col = nw * 16 + n * 8 + c2;
    const int r = mt * 16 + g;
    if (r < nb)
      *reinterpret_cast<uint32_t*>(out + r * out_stride + col) =
          pack_bf16x2(acc[n][0], acc[n][1]);
    if (r + 8 < nb)
      *reinterpret_cast<uint32_t*>(out + (r + 8) * out_stride + col) =
          pack_bf16x2(acc[n][2], acc[n][3]);
  }
}

}  // namespace proj
}  // namespace mla
