// Routing from logits: scores, a bias that only chooses, groups, top-k.
//
//   s = softmax(l) or sigmoid(l)          c = s + bias   (c = l without a bias:
//                                         both scores rise with the logit)
//   a group's score is its largest c, or the sum of its two largest s + bias;
//   the top_groups best groups stay (equal scores: the lower group), and of
//   their experts the K largest c are chosen (equal: the lower expert)
//   w = s_sel / (sum s_sel + 1e-9) if normalised, else s_sel; times scale
//
// One warp per token; lane i owns experts [i * EPL, (i + 1) * EPL), so the
// lowest lane of a tie holds the lowest expert.  A choice is one
// __reduce_max_sync over order-preserving 32-bit keys and one ballot.
//
// Which of two near scores is larger decides whole numbers, so the choice is
// the one of scores computed in 64 bits: the fp32 scores are taken while
// every comparison that decided something is wider than their error, and a
// token with a closer one (under 1% of them with 256 experts) is chosen again
// in fp64 by the same warp.  Logits ranked without a bias need no such check.
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr unsigned int kFull = 0xffffffffu;

// Order-preserving map of a float (no NaN) to unsigned; 0 is below all.
__device__ __forceinline__ unsigned int order_key(float v) {
  v += 0.f;                                             // -0 ranks as +0
  const unsigned int u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct Shared {
  float by[kWarps][kMaxExperts];        // what groups are ranked by
  unsigned char keep[kWarps][kMaxExperts];   // group stays
  int sel[kWarps][kMaxExperts];
  float val[kWarps][kMaxExperts];
};

// A logit as the scores take it: NaN never ranks, +inf counts as the largest
// finite value.
__device__ __forceinline__ float clean(float l) { return isnan(l) ? -INFINITY : fminf(l, FLT_MAX); }

// Half-width of the fp32 scores' error, doubled for a difference of two.
// sigmoid: expf, 1 + e and the quotient are each within 2^-23 relative, s <= 1.
// softmax: the exponent's rounding moves e^(l - m) by at most 2^-24 / e, the
// sum of at most 256 terms by 13 roundings.
__device__ __forceinline__ float score_tol(int score) { return score == 0 ? 3.8147e-6f : 9.5367e-7f; }

// True when a > b for sure: each is a score plus a bias, rounded once or
// (groups) twice.
__device__ __forceinline__ bool surely_above(float a, float b, float tol) {
  return a - b > tol + 4.7684e-7f * (fabsf(a) + fabsf(b));
}

// The whole choice in fp64 (the same definitions), for the tokens whose fp32
// scores are too close.  Writes sh.sel and sh.val.
template <int EPL>
__device__ __noinline__ void select_exact(const SelectArgs& a, const float* lrow, Shared& sh, int warp,
                                          int lane) {
  double sc[EPL], rk[EPL];
  double m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    sc[i] = e < a.E ? static_cast<double>(clean(lrow[e])) : -INFINITY;
    m = fmax(m, sc[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    rk[i] = sc[i];
    if (a.score == 0) {
      sc[i] = m == -INFINITY ? 0.0 : exp(sc[i] - m);
      sum += sc[i];
    } else {
      sc[i] = 1.0 / (1.0 + exp(-sc[i]));
    }
  }
  if (a.score == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    const double by = sum > 0.0 ? sum : 1.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] /= by;
  }
  unsigned int open = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    if (e >= a.E) continue;
    open |= 1u << i;
    if (a.bias) {
      const double c = sc[i] + static_cast<double>(a.bias[e]);
      rk[i] = isnan(c) ? -INFINITY : fmin(c, static_cast<double>(FLT_MAX));
    }
  }
  if (a.groups > 1) {
    // a group's two largest values, group after group over the whole warp
    const int size = a.E / a.groups;
    double mine = -INFINITY;       // of group `lane` + 32 * (g / 32), one chunk of 32 groups at a time
    double score[kMaxExperts / 32];
#pragma unroll
    for (int c = 0; c < kMaxExperts / 32; ++c) score[c] = -INFINITY;
    for (int g = 0; g < a.groups; ++g) {
      double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        if (e < g * size || e >= (g + 1) * size) continue;
        const double v = a.bias || a.group_score == 0 ? rk[i] : sc[i];
        if (v > m1) { m2 = m1; m1 = v; } else m2 = fmax(m2, v);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
        m2 = fmax(fmin(m1, o1), fmax(m2, o2));
        m1 = fmax(m1, o1);
      }
      mine = a.group_score == 0 || size == 1 ? m1 : m1 + m2;
#pragma unroll
      for (int c = 0; c < kMaxExperts / 32; ++c)
        if (c == (g >> 5) && lane == (g & 31)) score[c] = mine;
    }
    for (int g = 0; g < a.groups; ++g) {
      double v = 0.0;
#pragma unroll
      for (int c = 0; c < kMaxExperts / 32; ++c) {
        const double w = __shfl_sync(kFull, score[c], g & 31);
        if (c == (g >> 5)) v = w;
      }
      int ahead = 0;
#pragma unroll
      for (int c = 0; c < kMaxExperts / 32; ++c) {
        const int h = c * 32 + lane;
        if (h < a.groups && (score[c] > v || (score[c] == v && h < g))) ++ahead;
      }
      ahead = __reduce_add_sync(kFull, ahead);
      if (ahead >= a.top_groups) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane * EPL + i;
          if (e >= g * size && e < (g + 1) * size) open &= ~(1u << i);
        }
      }
    }
  }
  for (int k = 0; k < a.K; ++k) {
    double bv = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if ((open >> i & 1u) && (be == 0x7fffffff || rk[i] > bv)) {
        bv = rk[i];
        be = lane * EPL + i;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kFull, bv, o);
      const int oe = __shfl_xor_sync(kFull, be, o);
      if (oe != 0x7fffffff && (be == 0x7fffffff || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane * EPL + i == be) {
        open &= ~(1u << i);
        sh.sel[warp][k] = be;
        sh.val[warp][k] = static_cast<float>(sc[i]);
      }
  }
}

template <int EPL>
__global__ void __launch_bounds__(kWarps * 32) select_experts_kernel(const SelectArgs a) {
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= a.T) return;
  const int E = a.E;
  const float* lrow = a.logits + t * E;

  float l[EPL], sc[EPL];
  float m = -INFINITY;
  if (EPL % 4 == 0 && E == 32 * EPL) {
    // rows are whole 16-byte vectors (the pointer is 16-byte aligned)
#pragma unroll
    for (int i = 0; i < EPL / 4; ++i) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(lrow + lane * EPL) + i);
      l[4 * i] = q.x; l[4 * i + 1] = q.y; l[4 * i + 2] = q.z; l[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      l[i] = e < E ? __ldg(lrow + e) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = clean(l[i]);
    m = fmaxf(m, l[i]);
  }
  if (a.score == 0) {
    m = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      sc[i] = m == -INFINITY ? 0.f : expf(l[i] - m);
      sum += sc[i];
    }
    sum = warp_sum(sum);
    const float by = sum > 0.f ? sum : 1.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] = sc[i] / by;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sc[i] = 1.f / (1.f + expf(-l[i]));
  }
  // what experts are ranked by, in l from here on; key 0 = not to be chosen
  unsigned int key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    if (a.bias && e < E) {
      const float c = sc[i] + __ldg(a.bias + e);
      l[i] = clean(c);
    }
    key[i] = e < E ? order_key(l[i]) : 0u;
  }
  const float tol = score_tol(a.score);
  bool sure = true;

  if (a.groups > 1) {
    const bool top2 = a.group_score == 1;
    const bool by_rank = a.bias || !top2;
    const int size = E / a.groups;
    const bool exact = !a.bias && !top2;        // logits: no rounding to doubt
    if (E == 32 * EPL && a.groups <= 32 && (32 % a.groups) == 0) {
      // a group is a power-of-two run of whole lanes: butterflies inside it
      const int run = 32 / a.groups;
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float v = by_rank ? l[i] : sc[i];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      for (int o = 1; o < run; o <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      const float v = top2 && size > 1 ? m1 + m2 : m1;
      const int g = lane / run;
      int ahead = 0;
      for (int h = 0; h < a.groups; ++h) {
        const float w = __shfl_sync(kFull, v, h * run);
        ahead += w > v || (w == v && h < g) ? 1 : 0;
      }
      const bool keep = ahead < a.top_groups;
      if (!exact && a.top_groups < a.groups) {
        const float worst = -warp_max(keep ? -v : -INFINITY);
        const float next = warp_max(keep ? -INFINITY : v);
        sure = surely_above(worst, next, 2.f * tol);
      }
      if (!keep) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = 0u;
      }
    } else {
      // groups of any size: through shared memory, a lane per group
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        if (e < E) sh.by[warp][e] = by_rank ? l[i] : sc[i];
      }
      __syncwarp();
      for (int g = lane; g < a.groups; g += 32) {
        float m1 = -INFINITY, m2 = -INFINITY;
        for (int e = g * size; e < (g + 1) * size; ++e) {
          const float v = sh.by[warp][e];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
        sh.val[warp][g] = top2 && size > 1 ? m1 + m2 : m1;
      }
      __syncwarp();
      float worst = INFINITY, next = -INFINITY;
      for (int g = lane; g < a.groups; g += 32) {
        const float v = sh.val[warp][g];
        int ahead = 0;
        for (int h = 0; h < a.groups; ++h) {
          const float w = sh.val[warp][h];
          ahead += w > v || (w == v && h < g) ? 1 : 0;
        }
        const bool keep = ahead < a.top_groups;
        sh.keep[warp][g] = keep;
        if (keep) worst = fminf(worst, v); else next = fmaxf(next, v);
      }
      if (!exact && a.top_groups < a.groups) {
        worst = -warp_max(-worst);
        next = warp_max(next);
        sure = surely_above(worst, next, 2.f * tol);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        if (e < E && !sh.keep[warp][e / size]) key[i] = 0u;
      }
      __syncwarp();                              // sh.val is written again below
    }
  }

  // K choices, each the largest key left; with a bias one more than that, to
  // know how far the first one left out is
  float last = 0.f;
  const int rounds = a.bias ? a.K + 1 : a.K;
  unsigned int best = 0u;
#pragma unroll
  for (int i = 0; i < EPL; ++i) best = max(best, key[i]);
  for (int k = 0; k < rounds; ++k) {
    const unsigned int top = __reduce_max_sync(kFull, best);
    if (top == 0u) break;                        // all that may be chosen are
    const int owner = __ffs(__ballot_sync(kFull, best == top)) - 1;
    if (a.bias) {
      const unsigned int u = (top & 0x80000000u) ? top & 0x7fffffffu : ~top;
      const float v = __uint_as_float(u);
      if (k > 0 && !surely_above(last, v, tol)) sure = false;
      last = v;
    }
    if (lane == owner && k < a.K) {
      int at = 0;
      float s = 0.f;
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i)
        if (key[i] == top) {
          at = i;
          s = sc[i];
        }
      sh.sel[warp][k] = lane * EPL + at;
      sh.val[warp][k] = s;
      best = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (i == at) key[i] = 0u;
        best = max(best, key[i]);
      }
    }
  }
  if (!sure) select_exact<EPL>(a, lrow, sh, warp, lane);
  __syncwarp();

  float part = 0.f;
  for (int k = lane; k < a.K; k += 32) part += sh.val[warp][k];
  const float denom = a.norm ? warp_sum(part) + 1e-9f : 1.f;
  for (int k = lane; k < a.K; k += 32) {
    const int64_t o = t * a.K + k;
    a.selected[o] = sh.sel[warp][k];
    a.weights[o] = sh.val[warp][k] / denom * a.scale;
  }
}

}  // namespace

cudaError_t launch_select_experts(const SelectArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.T + kWarps - 1) / kWarps)), block(kWarps * 32);
  switch ((a.E + 31) / 32) {
    case 1: return launch_k(select_experts_kernel<1>, grid, block, 0, s, false, 1, a);
    case 2: return launch_k(select_experts_kernel<2>, grid, block, 0, s, false, 1, a);
    case 3: return launch_k(select_experts_kernel<3>, grid, block, 0, s, false, 1, a);
    case 4: return launch_k(select_experts_kernel<4>, grid, block, 0, s, false, 1, a);
    case 5: return launch_k(select_experts_kernel<5>, grid, block, 0, s, false, 1, a);
    case 6: return launch_k(select_experts_kernel<6>, grid, block, 0, s, false, 1, a);
    case 7: return launch_k(select_experts_kernel<7>, grid, block, 0, s, false, 1, a);
    default: return launch_k(select_experts_kernel<8>, grid, block, 0, s, false, 1, a);
  }
}

}  // namespace moe
