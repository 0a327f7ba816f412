// rope_apply.cu -- the rotary step by itself, on [T, H, R] slices of wider tensors.
//
// Pair d < R/2 of a row at position p, (u, v), becomes
//   (u c - v s, v c + u s),   c, s = columns d and R/2 + d of the table's row p  (s negated: back)
// where u, v are elements d and R/2 + d (half layout) or 2 d and 2 d + 1 (interleaved); the result
// may be written in the other layout.  fp32 arithmetic, rounded once to the tensors' type.  The step
// is linear with an orthogonal matrix (times the table's ratio), so its gradient is the step back
// from y's layout to x's.
//
// Bound by HBM: 2 R elements moved per row, three operations each.  A thread takes 16 bytes' worth
// of pairs, two 16-byte pieces to read and two to write in either layout, so the layouts cost
// nothing.  The R / (2 * 16 bytes) threads of a row lie in one warp, which reads all of its rows
// before it writes any: in place in another layout a thread writes where others read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kApplyThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }

__device__ __forceinline__ const float* table_row(const RopeApplyArgs& a, int t) {
  const int p = a.positions[t], at = min(max(p, 0), a.table_rows - 1);
  if (at != p) set_status(a.status, MLA_ERR_KVLEN);
  return a.table + (size_t)at * a.R;
}

// 16 bytes of a row's elements.
template <typename T>
struct Piece {
  static constexpr int kN = 16 / sizeof(T);
  union {
    uint4 raw;
    T e[16 / sizeof(T)];
  };
  __device__ __forceinline__ Piece() {}
};

// One piece's worth of pairs: lo, hi are the row's two pieces, elements u.. and v.. in the half
// layout, pairs one behind the other in the interleaved one.
template <typename T>
__device__ __forceinline__ void turn(Piece<T>& lo, Piece<T>& hi, const float* c, const float* s,
                                     bool from_pairs, bool to_pairs) {
  constexpr int N = Piece<T>::kN;
  T in[2 * N], out[2 * N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    in[e] = lo.e[e];
    in[N + e] = hi.e[e];
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float u = to_f32(from_pairs ? in[2 * e] : in[e]);
    const float v = to_f32(from_pairs ? in[2 * e + 1] : in[N + e]);
    const T y0 = from_f32<T>(fmaf(u, c[e], -v * s[e])), y1 = from_f32<T>(fmaf(v, c[e], u * s[e]));
    if (to_pairs) {
      out[2 * e] = y0;
      out[2 * e + 1] = y1;
    } else {
      out[e] = y0;
      out[N + e] = y1;
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    lo.e[e] = out[e];
    hi.e[e] = out[N + e];
  }
}

// Rows are (token, head).  A warp takes 32 / P of them at a time, P threads each, kU times over.
// kShared: those of one token (its heads), whose cosines and sines a thread then reads once;
// otherwise, with fewer heads than that, any rows in order.
template <typename T, bool kShared, bool kFromPairs, bool kToPairs>
__global__ void __launch_bounds__(kApplyThreads) rope_apply_kernel(const RopeApplyArgs a) {
  constexpr int N = Piece<T>::kN, kU = kShared ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int P = a.R / (2 * N), per = 32 / P;  // threads of a row, rows of a warp
  const int k = lane % P, row = lane / P;
  const int64_t warps = (int64_t)gridDim.x * (kApplyThreads / 32);
  const int64_t warp = (int64_t)blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5);
  const int blocks = kShared ? (a.H + kU * per - 1) / (kU * per) : 1;  // of a token's heads
  const int64_t rows = (int64_t)a.T * a.H;
  const int64_t units = kShared ? (int64_t)a.T * blocks : (rows + kU * per - 1) / (kU * per);
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  // the row's pieces: columns N k and R/2 + N k, or 2 N k and 2 N k + N
  const int x0 = kFromPairs ? 2 * N * k : N * k, x1 = kFromPairs ? x0 + N : x0 + a.R / 2;
  const int y0 = kToPairs ? 2 * N * k : N * k, y1 = kToPairs ? y0 + N : y0 + a.R / 2;
  for (int64_t u = warp; u < units; u += warps) {
    Piece<T> lo[kU], hi[kU];
    float c[kShared ? 1 : kU][N], s[kShared ? 1 : kU][N];
    int64_t to[kU];
    const int tok = kShared ? (int)(u / blocks) : 0;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      int t, h;
      bool real = row < per;
      if (kShared) {
        t = tok;
        h = (int)(u - (int64_t)tok * blocks) * kU * per + i * per + row;
        real = real && h < a.H;
      } else {
        const int64_t r = u * kU * per + i * per + row;
        real = real && r < rows;
        t = real ? (int)(r / a.H) : 0;
        h = (int)(r - (int64_t)t * a.H);
      }
      to[i] = real ? t * a.y_row + h * a.y_head : -1;
      if (real) {
        const T* src = x + t * a.x_row + h * a.x_head;
        lo[i].raw = __ldcs(reinterpret_cast<const uint4*>(src + x0));
        hi[i].raw = __ldcs(reinterpret_cast<const uint4*>(src + x1));
      }
      if (kShared ? i == 0 : real) {
        const float* cs = table_row(a, t);
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const float4 cv = *reinterpret_cast<const float4*>(cs + N * k + e);
          const float4 sv = *reinterpret_cast<const float4*>(cs + a.R / 2 + N * k + e);
          const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            c[i][e + q] = cc[q];
            s[i][e + q] = a.sign * ss[q];
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      if (to[i] < 0) continue;
      turn<T>(lo[i], hi[i], c[kShared ? 0 : i], s[kShared ? 0 : i], kFromPairs, kToPairs);
      *reinterpret_cast<uint4*>(y + to[i] + y0) = lo[i].raw;
      *reinterpret_cast<uint4*>(y + to[i] + y1) = hi[i].raw;
    }
  }
}

// Any width, strides and alignment: a warp per row, a pair per lane and turn.  Element by element, which
// takes its time: 16411 tokens of 64 heads and 64 columns 316 us in bf16 (852 GB/s) with x one element
// past 16 bytes, 42 aligned; 256 in fp32 (2.1 TB/s), 89 aligned; 62 columns in bf16 309; 64 rows 2.
template <typename T>
__global__ void __launch_bounds__(kApplyThreads) rope_apply_any_kernel(const RopeApplyArgs a) {
  constexpr int kMost = kMaxRopeDim / 64;  // pairs of a lane
  const int lane = threadIdx.x & 31, half = a.R / 2;
  const int64_t rows = (int64_t)a.T * a.H, warps = (int64_t)gridDim.x * (kApplyThreads / 32);
  for (int64_t r = (int64_t)blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5); r < rows;
       r += warps) {
    const int t = (int)(r / a.H), h = (int)(r - (int64_t)t * a.H);
    const float* cs = table_row(a, t);
    const T* x = static_cast<const T*>(a.x) + t * a.x_row + h * a.x_head;
    T* y = static_cast<T*>(a.y) + t * a.y_row + h * a.y_head;
    float u[kMost], v[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int d = lane + 32 * i;
      if (d < half) {
        u[i] = to_f32(x[a.from_pairs ? 2 * d : d]);
        v[i] = to_f32(x[a.from_pairs ? 2 * d + 1 : half + d]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int d = lane + 32 * i;
      if (d < half) {
        const float c = cs[d], s = a.sign * cs[half + d];
        y[a.to_pairs ? 2 * d : d] = from_f32<T>(fmaf(u[i], c, -v[i] * s));
        y[a.to_pairs ? 2 * d + 1 : half + d] = from_f32<T>(fmaf(v[i], c, u[i] * s));
      }
    }
    __syncwarp();
  }
}

unsigned grid_of(int64_t warps) {
  const int sms = device_sm_count();
  const int64_t per = kApplyThreads / 32;
  return (unsigned)std::max<int64_t>(
      1, std::min<int64_t>((warps + per - 1) / per, (int64_t)(sms > 0 ? sms : 152) * 16));
}

template <typename T, bool kShared>
void launch_layouts(const RopeApplyArgs& a, unsigned grid, cudaStream_t stream) {
  if (a.from_pairs && a.to_pairs)
    rope_apply_kernel<T, kShared, true, true><<<grid, kApplyThreads, 0, stream>>>(a);
  else if (a.from_pairs)
    rope_apply_kernel<T, kShared, true, false><<<grid, kApplyThreads, 0, stream>>>(a);
  else if (a.to_pairs)
    rope_apply_kernel<T, kShared, false, true><<<grid, kApplyThreads, 0, stream>>>(a);
  else
    rope_apply_kernel<T, kShared, false, false><<<grid, kApplyThreads, 0, stream>>>(a);
}

template <typename T>
cudaError_t launch_type(const RopeApplyArgs& a, cudaStream_t stream) {
  constexpr int N = 16 / (int)sizeof(T);
  const int64_t rows = (int64_t)a.T * a.H;
  // A dimension of one element has no stride that is used.
  const auto whole = [&](const void* p, int64_t row, int64_t head) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.T == 1 || row % N == 0) &&
           (a.H == 1 || head % N == 0);
  };
  if (a.R % (2 * N) != 0 || !whole(a.x, a.x_row, a.x_head) || !whole(a.y, a.y_row, a.y_head)) {
    rope_apply_any_kernel<T><<<grid_of(rows), kApplyThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const int per = 32 / (a.R / (2 * N));
  if (a.H >= per)
    launch_layouts<T, true>(a, grid_of((int64_t)a.T * ((a.H + 4 * per - 1) / (4 * per))), stream);
  else
    launch_layouts<T, false>(a, grid_of((rows + 2 * per - 1) / (2 * per)), stream);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_apply(const RopeApplyArgs& a, cudaStream_t stream) {
  switch (a.type) {
    case MLA_TYPE_BF16: return launch_type<__nv_bfloat16>(a, stream);
    case MLA_TYPE_FP16: return launch_type<__half>(a, stream);
    default: return launch_type<float>(a, stream);
  }
}

}  // namespace mla
