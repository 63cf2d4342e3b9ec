// C entry points of the 8-bit path: the residual norm, the routing with
// groups, the block-scaled product and the experts of one layer in 8 bits.
// Validation first, on the host; nothing is launched and no output touched
// when an argument is refused.
#include <limits.h>
#include <math.h>

#include <initializer_list>

#include "../../include/moe.h"
#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

// One CTA per 32-token block (the permutation's blocks).  Counts within a
// block come from shared-memory adds of integers: their order is free.
__global__ void __launch_bounds__(256) count_selected_kernel(const int64_t* __restrict__ selected,
                                                             int T, int K, int E,
                                                             int* __restrict__ idx32,
                                                             int* __restrict__ blockcounts) {
  __shared__ int hist[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * kRouterTokensPerCta * K;
  const int64_t hi = min(static_cast<int64_t>(T) * K, lo + kRouterTokensPerCta * K);
  for (int64_t s = lo + threadIdx.x; s < hi; s += blockDim.x) {
    const int64_t v = selected[s];
    const int e = v >= 0 && v < E ? static_cast<int>(v) : E;
    idx32[s] = e;
    if (e < E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    blockcounts[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
}

// The whole permutation of a small batch in one CTA: counts, offsets, and each
// slot's row (stable, by slot).  Slots are taken 1024 at a time in order; a
// slot's rank is that within its warp (match), behind the earlier warps'
// counts and the earlier slots' rows.  One launch instead of three (counts,
// scan, scatter) for batches that the gate_up GEMM does not sort itself: 12 -> 4
// us, measured with 192 slots of 64 experts.  The other path's start costs more
// the more experts there are, this one's turns with the slots.  A whole call
// (widths of 128) against the other path, us: 8 experts, 2000 slots 24.3 | 24.6,
// 2400 28.0 | 27.5; 32 experts, 2000 25.9 | 26.7, 2600 27.9 | 27.3; 64 experts,
// 3000 29.4 | 29.7, 3400 30.7 | 29.9; 128 experts, 4096 34.5 | 36.5; 256 experts,
// 4096 37.8 | 48.9.
constexpr int kSmallThreads = 1024;
bool permute_in_one_cta(int64_t slots, int E) { return slots <= 1800 + 20LL * E && slots <= 4096; }

__global__ void __launch_bounds__(kSmallThreads) permute_small_kernel(const int64_t* __restrict__ selected,
                                                                      int slots, int E,
                                                                      int* __restrict__ offsets,
                                                                      int* __restrict__ perm,
                                                                      int* __restrict__ pos) {
  __shared__ int run[kMaxExperts];                       // an expert's next row
  __shared__ int wc[kSmallThreads / 32][kMaxExperts];    // its slots in a warp's 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < kMaxExperts; e += kSmallThreads) run[e] = 0;
  for (int e = lane; e < E; e += 32) wc[warp][e] = 0;
  __syncthreads();
  auto expert = [&](int s) {
    if (s >= slots) return -1;
    const int64_t v = __ldg(selected + s);
    return v >= 0 && v < E ? static_cast<int>(v) : -1;
  };
  for (int s = threadIdx.x; s < slots; s += kSmallThreads) {
    const int e = expert(s);
    if (e >= 0) atomicAdd(&run[e], 1);                   // integers: the order is free
  }
  __syncthreads();
  if (warp == 0) {
    // exclusive sums of the counts, eight experts a lane
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = run[lane * 8 + i];
      sum += c[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int at = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      run[e] = at;
      if (e <= E) offsets[e] = at;
      at += c[i];
    }
    if (lane == 31 && E == kMaxExperts) offsets[E] = at;
  }
  __syncthreads();
  for (int s0 = 0; s0 < slots; s0 += kSmallThreads) {
    const int s = s0 + threadIdx.x;
    const int e = expert(s);
    const unsigned int same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) wc[warp][e] = __popc(same);
    __syncthreads();
    if (e >= 0) {
      int r = run[e] + rank;
      for (int w = 0; w < warp; ++w) r += wc[w][e];
      perm[r] = s;
      pos[s] = r;
    } else if (s < slots) {
      pos[s] = -1;
    }
    __syncthreads();
    if (s0 + kSmallThreads < slots) {
      for (int q = threadIdx.x; q < E; q += kSmallThreads) {
        int add = 0;
        for (int w = 0; w < kSmallThreads / 32; ++w) {
          add += wc[w][q];
          wc[w][q] = 0;
        }
        run[q] += add;
      }
      __syncthreads();
    }
  }
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

moe_status_t check_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned(p, 16))
      return fail_status(MOE_ERR_ALIGNMENT, "device pointers must be 16-byte aligned");
  return MOE_OK;
}

moe_status_t check_dt(moe_dtype_t dt) {
  if (dt != MOE_F32 && dt != MOE_BF16)
    return fail_status(MOE_ERR_DTYPE, "dtype %d not supported (f32 or bf16)", static_cast<int>(dt));
  return MOE_OK;
}

moe_status_t launched(cudaError_t e, cudaStream_t s, const char* what) {
  if (e != cudaSuccess) return fail_status(MOE_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return debug_sync_passed(s, what) ? MOE_OK : MOE_ERR_TIMEOUT;
}

// The choice's arguments; fills everything of a but its pointers.
moe_status_t check_select(int64_t T, int E, int K, int norm, const moe_group_opts_t* o, SelectArgs* a) {
  if (T <= 0 || E <= 0)
    return fail_status(MOE_ERR_INVALID_ARG, "dimensions must be positive (T=%lld E=%d)",
                       static_cast<long long>(T), E);
  if (E > MOE_MAX_EXPERTS)
    return fail_status(MOE_ERR_SHAPE, "E=%d exceeds MOE_MAX_EXPERTS=%d", E, MOE_MAX_EXPERTS);
  if (T > INT_MAX) return fail_status(MOE_ERR_SHAPE, "T=%lld exceeds 2^31-1", static_cast<long long>(T));
  const moe_group_opts_t none{};
  if (!o) o = &none;
  if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID)
    return fail_status(MOE_ERR_INVALID_ARG, "unknown score function %d", static_cast<int>(o->score));
  if (o->group_score != MOE_GROUP_MAX && o->group_score != MOE_GROUP_TOP2)
    return fail_status(MOE_ERR_INVALID_ARG, "unknown group score %d", static_cast<int>(o->group_score));
  const int groups = o->groups == 0 ? 1 : o->groups;
  const int top = o->top_groups == 0 ? groups : o->top_groups;
  if (groups < 1 || E % groups != 0)
    return fail_status(MOE_ERR_INVALID_ARG, "groups=%d does not divide E=%d", groups, E);
  if (top < 1 || top > groups)
    return fail_status(MOE_ERR_INVALID_ARG, "top_groups=%d outside [1, groups=%d]", top, groups);
  if (K < 1 || K > top * (E / groups))
    return fail_status(MOE_ERR_INVALID_ARG, "top_k=%d outside [1, %d experts of the kept groups]", K,
                       top * (E / groups));
  if (!(fabsf(o->scale) < 1e30f))
    return fail_status(MOE_ERR_INVALID_ARG, "scale must be finite");
  if (o->selection_bias && !aligned(o->selection_bias, 16))
    return fail_status(MOE_ERR_ALIGNMENT, "selection_bias must be 16-byte aligned");
  *a = SelectArgs{};
  a->T = T;
  a->E = E;
  a->K = K;
  a->norm = norm ? 1 : 0;
  a->score = o->score == MOE_SCORE_SIGMOID ? 1 : 0;
  a->bias = o->selection_bias;
  a->groups = groups;
  a->top_groups = top;
  a->group_score = o->group_score == MOE_GROUP_TOP2 ? 1 : 0;
  a->scale = o->scale == 0.f ? 1.f : o->scale;
  return MOE_OK;
}

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Workspace of moe_experts_forward_fp8.
struct Layout {
  size_t idx32, bcount, bbase, totals, offsets, perm, pos, xperm, h, hscales, y, yscales, total;
  int B;
  bool gather;      // gate_up fetches its rows of x by token
};

Layout layout(int64_t T, int64_t D, int64_t F, int E, int K) {
  Layout L{};
  const int64_t R = T * K;
  L.B = static_cast<int>((T + kRouterTokensPerCta - 1) / kRouterTokensPerCta);
  // few rows per expert: their copies hide under the weight stream
  L.gather = R <= 16LL * E;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 1024);
    return at;
  };
  L.idx32 = take(sizeof(int) * R);
  L.bcount = take(sizeof(int) * static_cast<size_t>(L.B) * E);
  L.bbase = take(sizeof(int) * static_cast<size_t>(L.B) * E);
  L.totals = take(sizeof(int) * E);
  L.offsets = take(sizeof(int) * (E + 1));
  L.perm = take(sizeof(int) * R);
  L.pos = take(sizeof(int) * R);
  L.xperm = take(L.gather ? 0 : static_cast<size_t>(R) * D);
  L.h = take(static_cast<size_t>(R) * F);
  L.hscales = take(sizeof(float) * R * ((F + kQuantBlock - 1) / kQuantBlock));
  L.y = take(2 * static_cast<size_t>(R) * D);
  L.yscales = take(sizeof(float) * R * ((D + 63) / 64));
  L.total = o;
  return L;
}

moe_status_t check_experts(int64_t T, int64_t D, int64_t F, int E, int K) {
  if (T <= 0 || D <= 0 || F <= 0 || E <= 0)
    return fail_status(MOE_ERR_INVALID_ARG, "dimensions must be positive (T=%lld D=%lld F=%lld E=%d)",
                       static_cast<long long>(T), static_cast<long long>(D), static_cast<long long>(F),
                       E);
  if (K < 1 || K > E) return fail_status(MOE_ERR_INVALID_ARG, "top_k=%d outside [1, E=%d]", K, E);
  if (E > MOE_MAX_EXPERTS)
    return fail_status(MOE_ERR_SHAPE, "E=%d exceeds MOE_MAX_EXPERTS=%d", E, MOE_MAX_EXPERTS);
  // D: the combine's grid has a row of CTAs per 1024 columns, 65535 of them at most
  if (T > INT_MAX || T * K > INT_MAX - 128 || D > 65535LL * 1024 || F > INT_MAX / 2 ||
      static_cast<int64_t>(E) * 2 * F + 256 > INT_MAX || static_cast<int64_t>(E) * D + 256 > INT_MAX)
    return fail_status(MOE_ERR_SHAPE, "sizes exceed 32-bit indexing");
  if (D % 16 != 0 || F % 16 != 0)
    return fail_status(MOE_ERR_ALIGNMENT, "the 8-bit path needs D and F multiples of 16 (D=%lld F=%lld)",
                       static_cast<long long>(D), static_cast<long long>(F));
  return MOE_OK;
}

}  // namespace

cudaError_t launch_count_selected(const int64_t* selected, int T, int K, int E, int* idx32,
                                  int* blockcounts, cudaStream_t s) {
  const int B = (T + kRouterTokensPerCta - 1) / kRouterTokensPerCta;
  return launch_k(count_selected_kernel, dim3(B), dim3(256), 0, s, false, 1, selected, T, K, E, idx32,
                  blockcounts);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_add_rmsnorm(const void* x, const void* residual, const void* weight, float eps,
                             int64_t T, int64_t D, moe_dtype_t dt, void* sum_out, void* out,
                             void* out_fp8, float* scales, void* stream) {
  set_last_error("");
  moe_status_t st = check_dt(dt);
  if (st != MOE_OK) return st;
  if (T <= 0 || D <= 0)
    return fail_status(MOE_ERR_INVALID_ARG, "dimensions must be positive (T=%lld D=%lld)",
                       static_cast<long long>(T), static_cast<long long>(D));
  if (!x || !weight) return fail_status(MOE_ERR_INVALID_ARG, "x and weight are required");
  if (!out && !out_fp8) return fail_status(MOE_ERR_INVALID_ARG, "one of out and out_fp8 is required");
  if ((out_fp8 == nullptr) != (scales == nullptr))
    return fail_status(MOE_ERR_INVALID_ARG, "out_fp8 and scales go together");
  if (out && out == sum_out)
    return fail_status(MOE_ERR_INVALID_ARG, "out and sum_out must be different buffers");
  if (!(eps >= 0.f) || !(eps < 1e30f))
    return fail_status(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (D > kNormMaxD)
    return fail_status(MOE_ERR_SHAPE, "D=%lld exceeds %d", static_cast<long long>(D), kNormMaxD);
  if (T > INT_MAX) return fail_status(MOE_ERR_SHAPE, "T=%lld exceeds 2^31-1", static_cast<long long>(T));
  if ((st = check_aligned({x, residual, weight, sum_out, out, out_fp8, scales})) != MOE_OK) return st;
  unsigned int* err = nullptr;
  if ((st = device_ready(&err)) != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(launch_add_rmsnorm(x, residual, weight, eps, T, static_cast<int>(D),
                                     dt == MOE_BF16 ? kBF16 : kF32, sum_out, out,
                                     static_cast<uint8_t*>(out_fp8), scales, s),
                  s, "rms norm");
}

moe_status_t moe_quantize_fp8(const void* x, moe_dtype_t dt, int64_t matrices, int64_t rows,
                              int64_t cols, int block_rows, void* out_fp8, float* scales,
                              void* stream) {
  set_last_error("");
  moe_status_t st = check_dt(dt);
  if (st != MOE_OK) return st;
  if (matrices <= 0 || rows <= 0 || cols <= 0)
    return fail_status(MOE_ERR_INVALID_ARG, "dimensions must be positive (matrices=%lld rows=%lld cols=%lld)",
                       static_cast<long long>(matrices), static_cast<long long>(rows),
                       static_cast<long long>(cols));
  if (block_rows != 1 && block_rows != kQuantBlock)
    return fail_status(MOE_ERR_INVALID_ARG, "block_rows=%d must be 1 or %d", block_rows, kQuantBlock);
  if (!x || !out_fp8 || !scales)
    return fail_status(MOE_ERR_INVALID_ARG, "x, out_fp8 and scales are required");
  // rows are a grid dimension of up to 2^31 - 1 CTAs, a row or a block each at most
  if (rows > INT_MAX / matrices || cols > INT_MAX - 256 ||
      matrices * rows > INT_MAX / ((cols + kQuantBlock - 1) / kQuantBlock))
    return fail_status(MOE_ERR_SHAPE, "matrices * rows * blocks of 128 columns exceeds 2^31-1");
  if ((st = check_aligned({x, out_fp8, scales})) != MOE_OK) return st;
  unsigned int* err = nullptr;
  if ((st = device_ready(&err)) != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(launch_quantize_fp8(x, dt == MOE_BF16 ? kBF16 : kF32, matrices, rows,
                                      static_cast<int>(cols), block_rows,
                                      static_cast<uint8_t*>(out_fp8), scales, s),
                  s, "quantiser");
}

moe_status_t moe_select_experts(const float* logits, int64_t T, int E, int K, int norm_topk_prob,
                                const moe_group_opts_t* opts, int64_t* selected_experts,
                                float* routing_weights, void* stream) {
  set_last_error("");
  SelectArgs a;
  moe_status_t st = check_select(T, E, K, norm_topk_prob, opts, &a);
  if (st != MOE_OK) return st;
  if (!logits || !selected_experts || !routing_weights)
    return fail_status(MOE_ERR_INVALID_ARG, "logits, selected_experts and routing_weights are required");
  if ((st = check_aligned({logits, selected_experts, routing_weights})) != MOE_OK) return st;
  unsigned int* err = nullptr;
  if ((st = device_ready(&err)) != MOE_OK) return st;
  a.logits = logits;
  a.selected = selected_experts;
  a.weights = routing_weights;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(launch_select_experts(a, s), s, "expert selection");
}

moe_status_t moe_route_groups(const void* x, const void* router, const float* router_bias, int64_t T,
                              int64_t D, int E, int K, int norm_topk_prob, moe_dtype_t dt,
                              const moe_group_opts_t* opts, float* router_logits,
                              int64_t* selected_experts, float* routing_weights, void* stream) {
  set_last_error("");
  moe_status_t st = check_dt(dt);
  if (st != MOE_OK) return st;
  if (D <= 0 || D > INT_MAX)
    return fail_status(D <= 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_SHAPE, "D=%lld outside [1, 2^31-1]",
                       static_cast<long long>(D));
  SelectArgs a;
  if ((st = check_select(T, E, K, norm_topk_prob, opts, &a)) != MOE_OK) return st;
  if (!x || !router || !router_logits || !selected_experts || !routing_weights)
    return fail_status(MOE_ERR_INVALID_ARG,
                       "x, router, router_logits, selected_experts and routing_weights are required");
  if ((st = check_aligned({x, router, router_bias, router_logits, selected_experts, routing_weights})) !=
      MOE_OK)
    return st;
  if (dt == MOE_BF16 && D % 8 != 0)
    return fail_status(MOE_ERR_ALIGNMENT, "bf16 path needs D a multiple of 8 (D=%lld)",
                       static_cast<long long>(D));
  unsigned int* err = nullptr;
  if ((st = device_ready(&err)) != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the router kernel writes its logits and nothing else (no dependent launch)
  RouteArgs r{};
  r.x = x;
  r.router = router;
  r.router_bias = router_bias;
  r.T = static_cast<int>(T);
  r.D = static_cast<int>(D);
  r.E = E;
  r.K = 1;
  r.dt = dt == MOE_BF16 ? kBF16 : kF32;
  r.logits = router_logits;
  r.err = err;
  st = launched(dt == MOE_BF16 ? launch_router_tc(r, s) : launch_router(r, s), s, "router");
  if (st != MOE_OK) return st;
  a.logits = router_logits;
  a.selected = selected_experts;
  a.weights = routing_weights;
  return launched(launch_select_experts(a, s), s, "expert selection");
}

moe_status_t moe_gemm_fp8(const void* a, const float* a_scales, const void* w, const float* w_scales,
                          const int* offsets, int E, int64_t M, int64_t N, int64_t K, void* out,
                          moe_dtype_t out_dt, void* stream) {
  set_last_error("");
  moe_status_t st = check_dt(out_dt);
  if (st != MOE_OK) return st;
  if (E <= 0 || M <= 0 || N <= 0 || K <= 0)
    return fail_status(MOE_ERR_INVALID_ARG, "dimensions must be positive (E=%d M=%lld N=%lld K=%lld)", E,
                       static_cast<long long>(M), static_cast<long long>(N), static_cast<long long>(K));
  if (!a || !a_scales || !w || !w_scales || !out)
    return fail_status(MOE_ERR_INVALID_ARG, "a, a_scales, w, w_scales and out are required");
  if (E > 1 && !offsets) return fail_status(MOE_ERR_INVALID_ARG, "offsets are required for E=%d", E);
  if (E > MOE_MAX_EXPERTS)
    return fail_status(MOE_ERR_SHAPE, "E=%d exceeds MOE_MAX_EXPERTS=%d", E, MOE_MAX_EXPERTS);
  if (M > INT_MAX - 128 || N > INT_MAX - 256 || K > INT_MAX - 256 ||
      static_cast<int64_t>(E) * N + 256 > INT_MAX)
    return fail_status(MOE_ERR_SHAPE, "sizes exceed 32-bit indexing");
  // the kernels count tiles of 128 rows x 128 columns in 32 bits
  if ((M / 128 + E) * ((N + 127) / 128) > INT_MAX)
    return fail_status(MOE_ERR_SHAPE, "more than 2^31-1 tiles");
  if (K % 16 != 0 || N % 8 != 0)
    return fail_status(MOE_ERR_ALIGNMENT, "the 8-bit product needs K a multiple of 16 and N of 8 (K=%lld N=%lld)",
                       static_cast<long long>(K), static_cast<long long>(N));
  if ((st = check_aligned({a, a_scales, w, w_scales, out})) != MOE_OK) return st;
  if (offsets && !aligned(offsets, 4))
    return fail_status(MOE_ERR_ALIGNMENT, "offsets must be 4-byte aligned");
  unsigned int* err = nullptr;
  if ((st = device_ready(&err)) != MOE_OK) return st;
  GemmFp8Args g{};
  g.a = a;
  g.a_scales = a_scales;
  g.w = w;
  g.w_scales = w_scales;
  g.offsets = offsets;
  g.a_rows = g.M = static_cast<int>(M);
  g.E = E;
  g.N = static_cast<int>(N);
  g.K = static_cast<int>(K);
  g.out = out;
  g.out_f32 = out_dt == MOE_F32;
  g.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(launch_gemm_fp8(g, s), s, "fp8 GEMM");
}

size_t moe_experts_workspace_size_fp8(int64_t T, int64_t D, int64_t F, int E, int K) {
  return check_experts(T, D, F, E, K) == MOE_OK ? layout(T, D, F, E, K).total : 0;
}

moe_status_t moe_experts_forward_fp8(const void* x_fp8, const float* x_scales,
                                     const int64_t* selected_experts, const float* routing_weights,
                                     const void* gate_up_proj, const float* gate_up_scales,
                                     const void* down_proj, const float* down_scales, void* out,
                                     int64_t T, int64_t D, int64_t F, int E, int K, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  set_last_error("");
  moe_status_t st = check_experts(T, D, F, E, K);
  if (st != MOE_OK) return st;
  if (!x_fp8 || !x_scales || !selected_experts || !routing_weights || !gate_up_proj ||
      !gate_up_scales || !down_proj || !down_scales || !out)
    return fail_status(MOE_ERR_INVALID_ARG, "every tensor of moe_experts_forward_fp8 is required");
  if ((st = check_aligned({x_fp8, x_scales, selected_experts, routing_weights, gate_up_proj,
                           gate_up_scales, down_proj, down_scales, out, workspace})) != MOE_OK)
    return st;
  const Layout L = layout(T, D, F, E, K);
  if (!workspace || workspace_bytes < L.total)
    return fail_status(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", L.total,
                       workspace ? workspace_bytes : static_cast<size_t>(0));
  unsigned int* err = nullptr;
  if ((st = device_ready(&err)) != MOE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* idx32 = reinterpret_cast<int*>(ws + L.idx32);
  int* bcount = reinterpret_cast<int*>(ws + L.bcount);
  int* bbase = reinterpret_cast<int*>(ws + L.bbase);
  int* totals = reinterpret_cast<int*>(ws + L.totals);
  int* offsets = reinterpret_cast<int*>(ws + L.offsets);
  int* perm = reinterpret_cast<int*>(ws + L.perm);
  int* pos = reinterpret_cast<int*>(ws + L.pos);
  float* hscales = reinterpret_cast<float*>(ws + L.hscales);
  const int Ti = static_cast<int>(T), Di = static_cast<int>(D), Fi = static_cast<int>(F);
  const int R = Ti * K;

  // no programmatic dependent launch here, whatever moe_set_pdl says
  StageScope scope(s);
  scope.begin();
  const bool sorts = gemm_fp8_sorts(R, L.gather);     // in the gate_up GEMM
  if (!sorts && permute_in_one_cta(R, E)) {
    st = launched(launch_k(permute_small_kernel, dim3(1), dim3(kSmallThreads), 0, s, false, 1,
                           selected_experts, R, E, offsets, perm, pos),
                  s, "permutation");
    if (st != MOE_OK) return st;
  } else if (!sorts) {
    st = launched(launch_count_selected(selected_experts, Ti, K, E, idx32, bcount, s), s, "expert counts");
    if (st != MOE_OK) return st;
    const bool own_scan = static_cast<long long>(L.B) * E <= kScatterScansItself;
    if (!own_scan) {
      st = launched(launch_permute_scan(bcount, L.B, E, bbase, totals, false, s), s, "permute scan");
      if (st != MOE_OK) return st;
    }
    st = launched(launch_permute_scatter(idx32, own_scan ? nullptr : bbase, own_scan ? nullptr : totals,
                                         bcount, Ti, K, E, offsets, perm, pos, nullptr, nullptr, false, s),
                  s, "permute scatter");
    if (st != MOE_OK) return st;
  }
  if (!L.gather) {
    st = launched(launch_gather_rows(perm, offsets, pos, Ti, E, K, x_fp8, Di, ws + L.xperm, false, s), s,
                  "row gather");
    if (st != MOE_OK) return st;
  }
  scope.end(1);

  GemmFp8Args g{};
  g.a = L.gather ? x_fp8 : ws + L.xperm;
  g.a_scales = x_scales;
  g.w = gate_up_proj;
  g.w_scales = gate_up_scales;
  g.offsets = offsets;
  g.perm = perm;
  g.slots = K;
  g.selected = sorts ? selected_experts : nullptr;
  g.offsets_out = offsets;
  g.pos_out = pos;
  g.gather = L.gather;
  g.a_rows = L.gather ? Ti : R;
  g.M = R;
  g.E = E;
  g.N = Fi;
  g.K = Di;
  g.out = ws + L.h;
  g.q_scales = hscales;
  g.err = err;
  scope.begin();
  if ((st = launched(launch_gemm_fp8(g, s), s, "gate_up fp8 GEMM")) != MOE_OK) return st;
  scope.end(2);

  GemmFp8Args d{};
  d.a = ws + L.h;
  d.a_scales = hscales;
  d.w = down_proj;
  d.w_scales = down_scales;
  d.offsets = offsets;
  d.a_rows = d.M = R;
  d.E = E;
  d.N = Di;
  d.K = Fi;
  d.out = ws + L.y;
  d.f16_scales = reinterpret_cast<float*>(ws + L.yscales);
  d.err = err;
  scope.begin();
  if ((st = launched(launch_gemm_fp8(d, s), s, "down fp8 GEMM")) != MOE_OK) return st;
  scope.end(3);

  scope.begin();
  st = launched(launch_combine_f16(ws + L.y, d.f16_scales, routing_weights, pos, Ti, K, Di, out, s), s,
                "combine");
  if (st != MOE_OK) return st;
  scope.end(4);
  return MOE_OK;
}

}  // extern "C"
