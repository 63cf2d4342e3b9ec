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
// __reduce_max_sync over order-preserving 32-bit keys and one ballot.  The
// kernel is bound by instruction issue, not by memory (at 16384 tokens of 256
// experts the logits alone would take 3 us), so what ranks experts is computed
// with the fast exponential and reciprocal, and only the K chosen scores are
// computed again with expf and a division.  16384 tokens, 256 experts, 8 of
// them from 4 of 8 groups: 25 us, some 920 instructions a token (50 us with
// expf and a division for all, a scan for each choice and an fp64 path of
// 25000 cycles).
//
// Which of two near scores is larger decides whole numbers, so the choice is
// the one of scores computed in 64 bits: the fp32 scores are taken while
// every comparison that decided something is wider than their error, and a
// token with a closer one (under 1% of them with 256 experts) is chosen again
// in fp64 by the same warp.  Masked experts and groups cost nothing more, unless
// a token has fewer than K experts left (16384 tokens, 256 experts: 48 us).
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
  union {
    float slack[kWarps][kMaxExperts + 1];      // group scores' error
    int sel[kWarps][kMaxExperts + 1];
  };
  float val[kWarps][kMaxExperts + 1];   // group scores, then the ranks of the chosen
};

// A logit as the scores take it: NaN never ranks, +inf counts as the largest
// finite value.
__device__ __forceinline__ float clean(float l) { return isnan(l) ? -INFINITY : fminf(l, FLT_MAX); }

// The fp32 scores' error, doubled for a difference of two.  The fast
// exponential is within 2^-22 and |x| 2^-24 (its argument's rounding) relative,
// the fast reciprocal within 2^-23.  sigmoid, s <= 1 and s (1 - s) |l| < 0.23:
// under 0.25 * 2^-22 + 0.23 * 2^-24 + 2^-23 + 2^-24 = 2.6e-7, doubled 5.2e-7.
// softmax, e^-x x < 0.37, the sum of at most 256 terms with 13 roundings: under
// 2^-22 + 0.37 * 2^-24 + 14 * 2^-24 + 2^-23 = 1.3e-6, doubled 2.6e-6.
__device__ __forceinline__ float score_tol(int score) { return score == 0 ? 3.8147e-6f : 9.5367e-7f; }

// True when a > b for sure, where both are read from keys (up to 2^-20 too low)
// and a + tol may be off for other reasons.  A finite one is above -inf, which
// is exact (an expert that is masked).
__device__ __forceinline__ bool surely_above(float a, float b, float tol) {
  if (b == -INFINITY) return a > b;
  return a - b > tol + 1.2e-6f * (fabsf(a) + fabsf(b));
}

// How far a group's score, the sum of its two largest c (pair) or the largest,
// may be off for c's relative error as in surely_above: it goes with the two
// terms and does not shrink where they cancel.  A -inf among them (m2 <= m1) is
// one in 64 bits as well.  What the score is for sure is least to most; an
// overflow leaves both open.  (least is above -inf for a group of -inf, so that
// it is not in doubt where all others are -inf too: the lower group is taken.)
__device__ __forceinline__ float group_slack(float m1, float m2, bool pair) {
  const float low = pair ? m2 : m1;
  return low == -INFINITY ? 0.f : 1.2e-6f * (fabsf(m1) + (pair ? fabsf(m2) : 0.f));
}
__device__ __forceinline__ float group_least(float v, float slack) {
  return slack <= FLT_MAX ? fmaxf(v - slack, -FLT_MAX) : -INFINITY;
}
__device__ __forceinline__ float group_most(float v, float slack) {
  return slack <= FLT_MAX ? v + slack : INFINITY;
}

// A lane's i-th rank as a sortable key: the rank without its lowest three
// bits, then 7 - i, so that of equal ones the lower expert is larger.  What
// the truncation hides is close enough to be taken for unsure.
__device__ __forceinline__ unsigned int rank_key(float v, int i) {
  return (order_key(v) & ~7u) | static_cast<unsigned int>(7 - i);
}
__device__ __forceinline__ float key_value(unsigned int k) {
  k &= ~7u;
  if (k < 0x00800000u) return -INFINITY;         // below the key of -FLT_MAX
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Eight keys in descending order (a sorting network of 19 exchanges).
__device__ __forceinline__ void sort8(unsigned int (&k)[8]) {
  auto cx = [&](int a, int b) {
    const unsigned int hi = max(k[a], k[b]);
    k[b] = min(k[a], k[b]);
    k[a] = hi;
  };
  cx(0, 2); cx(1, 3); cx(4, 6); cx(5, 7);
  cx(0, 4); cx(1, 5); cx(2, 6); cx(3, 7);
  cx(0, 1); cx(2, 3); cx(4, 5); cx(6, 7);
  cx(2, 4); cx(3, 5);
  cx(1, 4); cx(3, 6);
  cx(1, 2); cx(3, 4); cx(5, 6);
}

// Order-preserving map of a double (no NaN) to unsigned; 0 is below all.
__device__ __forceinline__ unsigned long long order_key64(double v) {
  v += 0.0;                                             // -0 ranks as +0
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v));
  return (u >> 63) ? ~u : u | 1ull << 63;
}

// The whole choice in fp64 (the same definitions), for the tokens whose fp32
// scores are too close.  Writes sh.sel.  Few tokens come here, but the last
// of them ends the kernel, so it is kept short: 64-bit keys, whose largest is
// two 32-bit reductions.
template <int EPL>
__device__ __noinline__ void select_exact(const SelectArgs& a, const float* lrow, Shared& sh, int warp,
                                          int lane) {
  double sc[EPL], rk[EPL];
  double m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    sc[i] = e < a.E ? static_cast<double>(clean(lrow[e])) : -INFINITY;
    rk[i] = sc[i];
    m = fmax(m, sc[i]);
  }
  if (a.bias || a.group_score == 1) {            // else only the logits are compared
    if (a.score == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        sc[i] = m == -INFINITY ? 0.0 : exp(sc[i] - m);
        sum += sc[i];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const double by = sum > 0.0 ? sum : 1.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] /= by;
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) sc[i] = 1.0 / (1.0 + exp(-sc[i]));
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        if (e >= a.E) continue;
        const double c = sc[i] + static_cast<double>(a.bias[e]);
        rk[i] = isnan(c) ? -INFINITY : fmin(c, static_cast<double>(FLT_MAX));
      }
    }
  }
  unsigned int open = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (lane * EPL + i < a.E) open |= 1u << i;

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    const bool by_rank = a.bias || a.group_score == 0;
    const bool pair = a.group_score == 1 && size > 1;
    auto merge = [](double& m1, double& m2, double v) {
      m2 = fmax(m2, fmin(m1, v));
      m1 = fmax(m1, v);
    };
    if (a.E == 32 * EPL && a.groups <= 32 && 32 % a.groups == 0) {
      const int run = 32 / a.groups;
      double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) merge(m1, m2, by_rank ? rk[i] : sc[i]);
      for (int o = 1; o < run; o <<= 1) {
        const double o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
        m2 = fmax(fmin(m1, o1), fmax(m2, o2));
        m1 = fmax(m1, o1);
      }
      const double v = pair ? m1 + m2 : m1;
      const int g = lane / run;
      int ahead = 0;
      for (int h = 0; h < a.groups; ++h) {
        const double w = __shfl_sync(kFull, v, h * run);
        ahead += w > v || (w == v && h < g) ? 1 : 0;
      }
      if (ahead >= a.top_groups) open = 0;
    } else {
      // groups of any size: a group's two largest, group after group over the
      // whole warp; lane g % 32 keeps group g's score
      double score[kMaxExperts / 32];
#pragma unroll
      for (int c = 0; c < kMaxExperts / 32; ++c) score[c] = -INFINITY;
      for (int g = 0; g < a.groups; ++g) {
        double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane * EPL + i;
          if (e >= g * size && e < (g + 1) * size) merge(m1, m2, by_rank ? rk[i] : sc[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const double o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
          m2 = fmax(fmin(m1, o1), fmax(m2, o2));
          m1 = fmax(m1, o1);
        }
#pragma unroll
        for (int c = 0; c < kMaxExperts / 32; ++c)
          if (c == (g >> 5) && lane == (g & 31)) score[c] = pair ? m1 + m2 : m1;
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
        if (__reduce_add_sync(kFull, ahead) >= a.top_groups) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const int e = lane * EPL + i;
            if (e >= g * size && e < (g + 1) * size) open &= ~(1u << i);
          }
        }
      }
    }
  }

  unsigned long long key[EPL], best = 0ull;
  int at = 0;
  auto head = [&] {                              // the largest key left, the lowest expert of equal ones
    best = 0ull;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
  };
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = open >> i & 1u ? order_key64(rk[i]) : 0ull;
  head();
  for (int k = 0; k < a.K; ++k) {
    const unsigned int hi = static_cast<unsigned int>(best >> 32);
    const unsigned int top = __reduce_max_sync(kFull, hi);
    const unsigned int lo = hi == top ? static_cast<unsigned int>(best) : 0u;
    const unsigned int low = __reduce_max_sync(kFull, lo);
    const bool mine = hi == top && lo == low;
    if (lane == __ffs(__ballot_sync(kFull, mine)) - 1) {
      sh.sel[warp][k] = lane * EPL + at;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i == at) key[i] = 0ull;
      head();
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

  float l[EPL];
  float m = -INFINITY, total = 1.f, inv_total = 1.f;
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
  for (int i = 0; i < EPL; ++i) l[i] = clean(l[i]);
  if (a.score == 0) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum += m == -INFINITY ? 0.f : __expf(l[i] - m);
    sum = warp_sum(sum);
    total = sum > 0.f ? sum : 1.f;
    inv_total = __fdividef(1.f, total);
  }
  // the score that experts are ranked by, from a logit
  auto score = [&](float v) {
    if (a.score != 0) return __fdividef(1.f, 1.f + __expf(-v));
    return m == -INFINITY ? 0.f : __expf(v - m) * inv_total;
  };
  const bool top2 = a.group_score == 1;
  const int size = E / a.groups;
  const bool pair = top2 && size > 1;            // a group's score is a sum
  const bool whole = E == 32 * EPL && a.groups <= 32 && 32 % a.groups == 0;   // groups are runs of lanes
  const float tol = score_tol(a.score);
  bool sure = true;

  // what experts are ranked by (loops apart, so that no test of an option is
  // repeated for every expert)
  float rank[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) rank[i] = l[i];
  if (a.bias) {
    float b[EPL];
    if (EPL % 4 == 0 && E == 32 * EPL) {
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(a.bias + lane * EPL) + i);
        b[4 * i] = q.x; b[4 * i + 1] = q.y; b[4 * i + 2] = q.z; b[4 * i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        b[i] = e < E ? __ldg(a.bias + e) : 0.f;
      }
    }
    if (a.score != 0) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) rank[i] = __fdividef(1.f, 1.f + __expf(-l[i]));
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) rank[i] = score(l[i]);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) rank[i] = clean(rank[i] + b[i]);
  }
  // as keys; 0 = not to be chosen
  unsigned int key[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    key[i] = 0u;
    if (i < EPL && lane * EPL + i < E) key[i] = rank_key(rank[i < EPL ? i : 0], i);
  }

  if (a.groups > 1 && !whole) {
    // groups of any size: through shared memory, a lane per group
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      if (e < E) sh.by[warp][e] = a.bias || !top2 ? rank[i] : score(l[i]);
    }
    __syncwarp();
    for (int g = lane; g < a.groups; g += 32) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int e = g * size; e < (g + 1) * size; ++e) {
        const float v = sh.by[warp][e];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
      sh.val[warp][g] = pair ? m1 + m2 : m1;
      sh.slack[warp][g] = group_slack(m1, m2, pair);
    }
    __syncwarp();
    float worst = INFINITY, next = -INFINITY;    // of the kept, the least; of the others, the most
    for (int g = lane; g < a.groups; g += 32) {
      const float v = sh.val[warp][g];
      int ahead = 0;
      for (int h = 0; h < a.groups; ++h) {
        const float w = sh.val[warp][h];
        ahead += w > v || (w == v && h < g) ? 1 : 0;
      }
      const bool keep = ahead < a.top_groups;
      sh.keep[warp][g] = keep;
      const float slack = sh.slack[warp][g];
      if (keep) worst = fminf(worst, group_least(v, slack)); else next = fmaxf(next, group_most(v, slack));
    }
    if ((a.bias || top2) && a.top_groups < a.groups)       // the largest logit is exact here
      sure = -warp_max(-worst) - warp_max(next) > 2.f * tol;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      if (e < E && !sh.keep[warp][e / size]) key[i] = 0u;
    }
    __syncwarp();                                // sh.val is written again below
  }
  sort8(key);

  if (a.groups > 1 && whole) {
    // a group is a power-of-two run of lanes: butterflies inside it, on the
    // ranks at the head of the sorted lists
    const int run = 32 / a.groups;
    float m1 = key_value(key[0]), m2 = EPL > 1 ? key_value(key[1]) : -INFINITY;
    if (top2 && !a.bias) {
      // Scores of logits: the two largest of l itself.  A truncated logit is off
      // by up to |l| 2^-20, whatever its score, and of more than two logits that
      // agree but for the truncated bits the list's head need not hold the largest.
      float l1 = -INFINITY, l2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        l2 = fmaxf(l2, fminf(l1, l[i]));
        l1 = fmaxf(l1, l[i]);
      }
      m1 = score(l1);
      if (EPL > 1) m2 = score(l2);
    }
    for (int o = 1; o < run; o <<= 1) {
      const float o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
      m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
      m1 = fmaxf(m1, o1);
    }
    const float v = pair ? m1 + m2 : m1;
    const int g = lane / run;
    int ahead = 0;
    for (int h = 0; h < a.groups; ++h) {
      const float w = __shfl_sync(kFull, v, h * run);
      ahead += w > v || (w == v && h < g) ? 1 : 0;
    }
    const bool keep = ahead < a.top_groups;
    if (a.top_groups < a.groups) {
      const float slack = group_slack(m1, m2, pair);
      sure = -warp_max(keep ? -group_least(v, slack) : -INFINITY) -
                 warp_max(keep ? -INFINITY : group_most(v, slack)) >
             (a.bias || top2 ? 2.f * tol : 0.f);
    }
    if (!keep) key[0] = 0u;                      // (the rest of the list is not reached)
  }

  // K choices, each the largest head of the lanes' lists, and one more, to know
  // how far the first one left out is
  auto choose = [&](unsigned int& top) {         // the lane that holds it, which moves on
    top = __reduce_max_sync(kFull, key[0]);
    const int owner = __ffs(__ballot_sync(kFull, key[0] == top)) - 1;
    const bool mine = lane == owner;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = mine ? (i + 1 < EPL ? key[i + 1] : 0u) : key[i];
    return owner;
  };
  // s times the token's normalisation, to the outputs of slot k
  auto put = [&](int k, int e, float s, float denom) {
    const int64_t o = t * a.K + k;
    a.selected[o] = e;
    a.weights[o] = s / denom * a.scale;
  };
  // a chosen score, exactly this time
  auto exact_score = [&](int e) {
    const float v = clean(__ldg(lrow + e));
    return a.score == 0 ? (m == -INFINITY ? 0.f : expf(v - m) / total) : 1.f / (1.f + expf(-v));
  };
  const float rank_tol = a.bias ? tol : 0.f;
  if (a.K < 32) {
    // lane k keeps the k-th choice
    unsigned int top = 0u;
    int from = 0;
    for (int k = 0; k <= a.K; ++k) {
      unsigned int best;
      const int owner = choose(best);
      top = lane == k ? best : top;
      from = lane == k ? owner : from;
    }
    // every choice has to be surely above the next one (0: there is none)
    const unsigned int after = __shfl_down_sync(kFull, top, 1);
    const bool close = lane < a.K && after != 0u && !surely_above(key_value(top), key_value(after), rank_tol);
    int e = from * EPL + 7 - static_cast<int>(top & 7u);
    if (!sure || __any_sync(kFull, close)) {
      select_exact<EPL>(a, lrow, sh, warp, lane);
      __syncwarp();
      e = lane < a.K ? sh.sel[warp][lane] : 0;
    }
    const float s = lane < a.K ? exact_score(e) : 0.f;
    const float denom = a.norm ? warp_sum(s) + 1e-9f : 1.f;
    if (lane < a.K) put(lane, e, s, denom);
    return;
  }
  int found = 0;
  for (; found <= a.K; ++found) {
    unsigned int best;
    const int owner = choose(best);
    if (best == 0u) break;                       // all that may be chosen are
    if (lane == 0) {
      sh.sel[warp][found] = owner * EPL + 7 - static_cast<int>(best & 7u);
      sh.val[warp][found] = key_value(best);
    }
  }
  __syncwarp();
  bool close = false;
  for (int k = lane; k + 1 < found; k += 32)
    close = close || !surely_above(sh.val[warp][k], sh.val[warp][k + 1], rank_tol);
  if (!sure || __any_sync(kFull, close)) select_exact<EPL>(a, lrow, sh, warp, lane);
  __syncwarp();
  float part = 0.f;
  for (int k = lane; k < a.K; k += 32) {
    const float s = exact_score(sh.sel[warp][k]);
    sh.val[warp][k] = s;
    part += s;
  }
  const float denom = a.norm ? warp_sum(part) + 1e-9f : 1.f;
  for (int k = lane; k < a.K; k += 32) put(k, sh.sel[warp][k], sh.val[warp][k], denom);
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
