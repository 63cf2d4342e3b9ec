// Residual RMS norm with an 8-bit output, and the block quantiser.
//
//   h = round_dt(x + r)            (h = x without a residual)
//   y = h * rsqrt(mean(h^2) + eps) * weight
//   sum_out = h, out = round_dt(y), (q, scales) = 128-column blocks of y
//
// y stays in fp32 up to its one rounding to out's type or to e4m3 (of the
// fp32 y, not of the rounded out).  h is rounded before the norm because h is
// what the next layer reads from memory: the result is that of an addition
// followed by a norm.
//
// HBM-bound: each row is read once and kept in registers between the sum of
// squares and the outputs.  One CTA per row.  A warp owns units of
// consecutive columns: 256 columns, 8 per lane, with 16-byte loads (a
// 128-column scale block is then 16 lanes), or, where D is not a multiple of
// 8 and rows start at any alignment, 128 columns, 4 per lane 32 columns
// apart, so that a scale block is one warp and loads still coalesce.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 8 consecutive values at a 16-byte aligned address.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 q;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = q;
}

// A lane's columns of unit u: 8 consecutive ones (kVec) or 4, 32 apart.
template <bool kVec>
struct Unit {
  static constexpr int kCols = kVec ? 256 : 128;
  static constexpr int N = kVec ? 8 : 4;
  __device__ static int col(int u, int lane, int i) {
    return kVec ? u * 256 + lane * 8 + i : u * 128 + i * 32 + lane;
  }
  template <typename T>
  __device__ static void load(const T* row, int u, int lane, int D, float (&v)[N]) {
    if constexpr (kVec) {
      const int c = u * 256 + lane * 8;
      if (c < D) {
        load8(row + c, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = col(u, lane, i);
        v[i] = c < D ? to_f<T>(row[c]) : 0.f;
      }
    }
  }
  template <typename T>
  __device__ static void store(T* row, int u, int lane, int D, const float (&v)[N]) {
    if constexpr (kVec) {
      const int c = u * 256 + lane * 8;
      if (c < D) store8(row + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = col(u, lane, i);
        if (c < D) row[c] = from_f<T>(v[i]);
      }
    }
  }
  // The largest |v| of this lane's block (16 lanes, or the warp).
  __device__ static float largest(const float (&v)[N]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int o = kVec ? 8 : 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  }
  // The unit's blocks of v = u * by to e4m3 and their scales.
  __device__ static void quantize(uint8_t* qrow, float* srow, int unit, int lane, int D,
                                  const float (&v)[N], const float (&u)[N], float by) {
    const float m = largest(u);
    float amax = m * by;
    const bool direct = fp8_direct(m) && amax >= kQuantFloor;
    float t[N];
    if (__any_sync(0xffffffffu, !direct)) {      // zeros, extremes: from v itself
      const float mv = largest(v);               // (all lanes meet in it)
      amax = direct ? amax : mv;
      const float s = fp8_scale(amax);
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = v[i] / s;
    } else {
      const float r = 1.f / m;
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = fp8_quotient(u[i], m, r);
    }
    const float s = fp8_scale(amax);
    if constexpr (kVec) {
      const int c = unit * 256 + lane * 8;
      if (c < D) {
        uint2 q;
        q.x = fp8_pack4(t[0], t[1], t[2], t[3]);
        q.y = fp8_pack4(t[4], t[5], t[6], t[7]);
        *reinterpret_cast<uint2*>(qrow + c) = q;
        if ((lane & 15) == 0) srow[c / kQuantBlock] = s;
      }
    } else {
      if (unit * 128 < D) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = col(unit, lane, i);
          if (c < D) qrow[c] = static_cast<uint8_t>(fp8_pack2(t[i], 0.f));
        }
        if (lane == 0) srow[unit] = s;
      }
    }
  }
};

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* sum_out;
  void* out;
  uint8_t* q;
  float* scales;
  float eps;
  int D;
};

// sum_out and out may be x or residual themselves: a row's loads all come
// before the barrier, its other stores after it, and each thread stores the
// columns it loaded.
template <typename T, bool kVec, int U>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(const NormArgs a) {
  using L = Unit<kVec>;
  constexpr int kAhead = 16 / L::N;      // units whose residual or weight is held at once
  __shared__ float part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  const int D = a.D;
  const size_t row = static_cast<size_t>(blockIdx.x) * D;
  const T* x = static_cast<const T*>(a.x) + row;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + row : nullptr;
  const T* w = static_cast<const T*>(a.weight);

  float h[U][L::N];
#pragma unroll
  for (int j = 0; j < U; ++j) L::load(x, warp + j * warps, lane, D, h[j]);
  if (r) {
    constexpr int P = U < kAhead ? U : kAhead;
#pragma unroll
    for (int j0 = 0; j0 < U; j0 += P) {
      float rv[P][L::N];
#pragma unroll
      for (int j = 0; j < P; ++j) L::load(r, warp + (j0 + j) * warps, lane, D, rv[j]);
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < L::N; ++i)
          h[j0 + j][i] = to_f<T>(from_f<T>(h[j0 + j][i] + rv[j][i]));
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < U; ++j)
#pragma unroll
    for (int i = 0; i < L::N; ++i) ss = fmaf(h[j][i], h[j][i], ss);
  ss = warp_sum(ss);
  if (lane == 0) part[warp] = ss;
  // the weights' latency hides behind the barrier while they fit the registers
  constexpr bool kEarly = U <= kAhead;
  float wv[kEarly ? U : 1][L::N];
  if constexpr (kEarly) {
#pragma unroll
    for (int j = 0; j < U; ++j) L::load(w, warp + j * warps, lane, D, wv[j]);
  }
  __syncthreads();
  ss = warp_sum(lane < warps ? part[lane] : 0.f);
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(D) + a.eps);

#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = warp + j * warps;
    if constexpr (!kEarly) L::load(w, u, lane, D, wv[0]);
    if (a.sum_out) L::store(static_cast<T*>(a.sum_out) + row, u, lane, D, h[j]);
    float y[L::N], hw[L::N];                     // hw: exact for bf16, what the blocks are divided from
#pragma unroll
    for (int i = 0; i < L::N; ++i) {
      hw[i] = h[j][i] * wv[kEarly ? j : 0][i];
      y[i] = h[j][i] * rstd * wv[kEarly ? j : 0][i];
    }
    if (a.out) L::store(static_cast<T*>(a.out) + row, u, lane, D, y);
    if (a.q) {
      const int nb = (D + kQuantBlock - 1) / kQuantBlock;
      L::quantize(a.q + row, a.scales + static_cast<size_t>(blockIdx.x) * nb, u, lane, D, y, hw, rstd);
    }
  }
}

template <typename T, bool kVec>
cudaError_t launch_norm(const NormArgs& a, int64_t rows, cudaStream_t s) {
  // Few rows: one unit per warp, for the shortest chain.  More rows than CTAs
  // fit: 64 bytes of each tensor per thread, which keeps more loads in flight
  // per SM and has fewer warps meet at a row's barrier (16384 x 2048 bf16 with
  // a residual: 57 us with 16 bytes, 54 with 32, 52 with 64; 4096 x 5120 fp32:
  // 62 us with 32, 60 with 64, 68 with 128).  Where lanes load single values,
  // four units at most and four warps a row: the chain of a unit's 4 values is
  // longer there and wants warps to hide it (9000 x 2567 bf16: 103 us with 8
  // units of a warp, 86 with 4, 90 with 2, 97 with 1; 12000 x 516: 43, 43, 31, 28).
  const int units = (a.D + Unit<kVec>::kCols - 1) / Unit<kVec>::kCols;
  int U = rows <= 2 * num_sms() ? 1 : kVec ? 8 / static_cast<int>(sizeof(T)) : 4;
  while (!kVec && U > 1 && units < 4 * U) U /= 2;
  while (U > 1 && U > units) U /= 2;
  while (units > 32 * U) U *= 2;
  const dim3 grid(static_cast<unsigned>(rows)), block(32 * ((units + U - 1) / U));
  switch (U) {
    case 1: return launch_k(add_rmsnorm_kernel<T, kVec, 1>, grid, block, 0, s, false, 1, a);
    case 2: return launch_k(add_rmsnorm_kernel<T, kVec, 2>, grid, block, 0, s, false, 1, a);
    case 4: return launch_k(add_rmsnorm_kernel<T, kVec, 4>, grid, block, 0, s, false, 1, a);
    default:                                   // kNormMaxD columns: 128 or 256 units
      if constexpr (!kVec) return launch_k(add_rmsnorm_kernel<T, kVec, 8>, grid, block, 0, s, false, 1, a);
      return cudaErrorInvalidValue;
  }
}

// ------------------------------------------------------------- the quantiser
// Rows: a warp per unit of columns of one row.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T* x, int64_t rows, int D,
                                                            uint8_t* q, float* scales) {
  using L = Unit<kVec>;
  const int lane = threadIdx.x & 31;
  const int units = (D + L::kCols - 1) / L::kCols;
  const int nb = (D + kQuantBlock - 1) / kQuantBlock;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= rows * units) return;
  const int64_t row = at / units;
  const int u = static_cast<int>(at - row * units);
  float v[L::N];
  L::load(x + row * D, u, lane, D, v);
  L::quantize(q + row * D, scales + row * nb, u, lane, D, v, v, 1.f);
}

// Matrices: a CTA per 128 x 128 block; a warp takes 16 of its rows, a lane
// the columns lane, lane + 32, lane + 64 and lane + 96 of each.  Run once
// when weights are loaded.
template <typename T>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const T* x, int rows, int cols,
                                                              uint8_t* q, float* scales) {
  __shared__ float part[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nr = (rows + kQuantBlock - 1) / kQuantBlock, nc = (cols + kQuantBlock - 1) / kQuantBlock;
  const int64_t b = blockIdx.x;
  const int64_t mat = b / (static_cast<int64_t>(nr) * nc);
  const int br = static_cast<int>(b / nc % nr), bc = static_cast<int>(b % nc);
  const int64_t base = mat * rows * static_cast<int64_t>(cols);
  float v[16][4];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = br * kQuantBlock + i * 8 + warp, c = bc * kQuantBlock + j * 32 + lane;
      v[i][j] = r < rows && c < cols ? to_f<T>(x[base + static_cast<int64_t>(r) * cols + c]) : 0.f;
      m = fmaxf(m, fabsf(v[i][j]));
    }
  m = warp_max(m);
  if (lane == 0) part[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, part[w]);
  const float s = fp8_scale(m);
  const bool direct = fp8_direct(m);
  const float inv = 1.f / m;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = br * kQuantBlock + i * 8 + warp, c = bc * kQuantBlock + j * 32 + lane;
      if (r < rows && c < cols)
        q[base + static_cast<int64_t>(r) * cols + c] = 
            static_cast<uint8_t>(fp8_pack2(direct ? fp8_quotient(v[i][j], m, inv) : v[i][j] / s, 0.f));
    }
  if (threadIdx.x == 0) scales[b] = s;
}

template <typename T>
cudaError_t launch_quantize_t(const void* x, int64_t matrices, int64_t rows, int cols, int block_rows,
                              uint8_t* q, float* scales, cudaStream_t s) {
  const T* p = static_cast<const T*>(x);
  if (block_rows > 1) {
    const int64_t blocks = matrices * ((rows + 127) / 128) * ((cols + 127) / 128);
    return launch_k(quantize_blocks_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                    false, 1, p, static_cast<int>(rows), cols, q, scales);
  }
  const int64_t all = matrices * rows;
  if (cols % 8 == 0)
    return launch_k(quantize_rows_kernel<T, true>,
                    dim3(static_cast<unsigned>((all * ((cols + 255) / 256) + 7) / 8)), dim3(256), 0, s,
                    false, 1, p, all, cols, q, scales);
  return launch_k(quantize_rows_kernel<T, false>,
                  dim3(static_cast<unsigned>((all * ((cols + 127) / 128) + 7) / 8)), dim3(256), 0, s,
                  false, 1, p, all, cols, q, scales);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* x, const void* residual, const void* weight, float eps,
                               int64_t T, int D, int dt, void* sum_out, void* out, uint8_t* q,
                               float* scales, cudaStream_t s) {
  const NormArgs a{x, residual, weight, sum_out, out, q, scales, eps, D};
  if (dt == kBF16)
    return D % 8 == 0 ? launch_norm<__nv_bfloat16, true>(a, T, s)
                      : launch_norm<__nv_bfloat16, false>(a, T, s);
  return D % 8 == 0 ? launch_norm<float, true>(a, T, s) : launch_norm<float, false>(a, T, s);
}

cudaError_t launch_quantize_fp8(const void* x, int dt, int64_t matrices, int64_t rows, int cols,
                                int block_rows, uint8_t* q, float* scales, cudaStream_t s) {
  if (dt == kBF16)
    return launch_quantize_t<__nv_bfloat16>(x, matrices, rows, cols, block_rows, q, scales, s);
  return launch_quantize_t<float>(x, matrices, rows, cols, block_rows, q, scales, s);
}

}  // namespace moe
