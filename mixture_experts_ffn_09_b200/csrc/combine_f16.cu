// Weighted combine of expert outputs in block-scaled fp16:
//
//   out[t, :] = sum_k w[t, k] * scale[pos[t, k], d / 64] * Y[pos[t, k], d]
//
// Bound by memory: a token's K rows of Y are read once and its row of out is
// written once.  A thread takes C chunks of 8 columns, 1024 apart (16-byte
// loads, one scale each), and has the loads of a batch of slots for all of
// them on the way before it uses any: about eight rows in flight whatever K
// is.  The terms are added in fp32 in slot order, rounded once.  A CTA is one
// token and 1024 * C columns, C smaller where few tokens would leave SMs idle.
// 4096 tokens, K = 2, 4096 columns: 22 us (C = 1: 35).
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 8;

template <int C>
__global__ void __launch_bounds__(kThreads) combine_f16_kernel(const __half* __restrict__ Y,
                                                               const float* __restrict__ scales,
                                                               const float* __restrict__ w,
                                                               const int* __restrict__ pos, int K, int D,
                                                               __nv_bfloat16* __restrict__ out) {
  constexpr int B = kBatch / C;                  // slots per batch
  __shared__ int sp[kMaxExperts];
  __shared__ float sw[kMaxExperts];
  const size_t t = blockIdx.x;
  for (int k = threadIdx.x; k < K; k += kThreads) {
    sp[k] = __ldg(pos + t * K + k);
    sw[k] = __ldg(w + t * K + k);
  }
  __syncthreads();
  const int d0 = blockIdx.y * (kThreads * 8 * C) + threadIdx.x * 8;
  const int blocks = (D + 63) / 64;
  float acc[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[c][i] = 0.f;
  for (int k0 = 0; k0 < K; k0 += B) {
    uint4 q[C][B];
    float f[C][B];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int r = k0 + j < K ? sp[k0 + j] : -1;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int d = d0 + c * kThreads * 8;
        q[c][j] = make_uint4(0u, 0u, 0u, 0u);
        f[c][j] = 0.f;
        if (r >= 0 && d < D) {                   // D is a multiple of 16
          q[c][j] = __ldg(reinterpret_cast<const uint4*>(Y + static_cast<size_t>(r) * D + d));
          f[c][j] = __ldg(scales + static_cast<size_t>(r) * blocks + d / 64);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (k0 + j >= K || sp[k0 + j] < 0) continue;       // an unused slot's weight is not looked at
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float s = sw[k0 + j] * f[c][j];
        const __half2* h = reinterpret_cast<const __half2*>(&q[c][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __half22float2(h[i]);
          acc[c][2 * i] = fmaf(s, v.x, acc[c][2 * i]);
          acc[c][2 * i + 1] = fmaf(s, v.y, acc[c][2 * i + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int d = d0 + c * kThreads * 8;
    if (d >= D) continue;
    uint4 o;
    __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(acc[c][2 * i], acc[c][2 * i + 1]);
    *reinterpret_cast<uint4*>(out + t * D + d) = o;
  }
}

}  // namespace

cudaError_t launch_combine_f16(const void* Y, const float* scales, const float* w, const int* pos, int T,
                               int K, int D, void* out, cudaStream_t s) {
  int C = K <= 2 ? 4 : K <= 4 ? 2 : 1;
  auto chunks = [&] { return (D + kThreads * 8 * C - 1) / (kThreads * 8 * C); };
  while (C > 1 && static_cast<long long>(T) * chunks() < 4LL * num_sms()) C >>= 1;
  const dim3 g(T, chunks());
  const auto* y = static_cast<const __half*>(Y);
  auto* o = static_cast<__nv_bfloat16*>(out);
  if (C == 4) return launch_k(combine_f16_kernel<4>, g, dim3(kThreads), 0, s, false, 1, y, scales, w, pos, K, D, o);
  if (C == 2) return launch_k(combine_f16_kernel<2>, g, dim3(kThreads), 0, s, false, 1, y, scales, w, pos, K, D, o);
  return launch_k(combine_f16_kernel<1>, g, dim3(kThreads), 0, s, false, 1, y, scales, w, pos, K, D, o);
}

}  // namespace moe
