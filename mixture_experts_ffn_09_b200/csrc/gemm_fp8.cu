// Block-scaled e4m3 grouped GEMM on the sm_100a tensor cores.
//
//   C[i, n] = sum_kb sa[i, kb] sw[e][n / 128, kb] sum_{k in block kb} A[i, k] W[e][n, k]
//
// for the rows i of expert e (offsets), kb over blocks of 128 columns.  The
// inner sum of a block is four tcgen05.mma kind::f8f6f4 (K = 32 each) into a
// fresh fp32 accumulator in TMEM; the scales differ from block to block in
// both operands, so the outer sum is kept in fp32 registers: the epilogue
// warps read each block's accumulator and add it, times sa * sw, to their
// own.  The tensor cores work on block kb + 1 in the other half of TMEM
// meanwhile.
//
// One persistent CTA per SM, 320 threads:
//   warp 0      TMA producer: A tile 128 x 128 and B tile 256 x 128 (two
//               128-row boxes) per block into a 4-stage ring.  A row block
//               of few rows is loaded by a lower box (8 to 128 rows); the
//               rest of the stage keeps what it held and feeds only
//               accumulator rows that are never read;
//   warp 1      allocates 512 TMEM columns; one lane issues the MMAs
//               (M = 128, N = 256) into two 256-column accumulators in turn;
//   warps 2..9  epilogue: a warp reads its 32 TMEM lanes (rows) and half of
//               the columns: 64 of the first 128 and 64 of the second, so
//               that in the gated form it holds the gate and the up value
//               of the same features.  128 fp32 sums per thread.
//
// Epilogues (columns of the output per tile):
//   kOutBf16, kOutF32   the sums, rounded once (256 columns);
//   kSiluQuant    B = 128 gate rows and the matching 128 up rows; h =
//                 silu(gate) * up in fp32, then e4m3 with one scale for the
//                 row's 128 columns: a row's largest |h| is a maximum over
//                 two threads (128 columns).
//
// Rows outside [offsets[0], offsets[E]) are not touched.  Every mbarrier wait
// is bounded (common.cuh).
#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;                        // bytes = e4m3 values = one scale block
constexpr int BN = 256;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK;               // 16 KB
constexpr int B_BYTES = BN * BK;               // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 512;
constexpr int kBoxes = 5;                      // A boxes of 8, 16, 32, 64 and 128 rows

enum { kOutBf16 = 0, kOutF32 = 1, kSiluQuant = 2 };

struct AMaps {
  CUtensorMap m[kBoxes];
};

struct Params {
  const int* offsets;    // (E + 1) first row of each expert, or null: one expert, all M rows
  const int* perm;       // row -> (token, slot): the row of the scales is perm[row] / slots; or null
  int slots;
  int gather;            // 1: the rows of A are fetched by token too (its map is one row high)
  int M, E;
  int n_out;             // output columns
  int num_kb;
  int w_rows;            // weight rows per expert
  int w_blocks;          // scale rows per expert
  int up_row, up_block;  // first up row and scale row of an expert (gated)
  const float* sa;       // (rows, num_kb)
  const float* sw;       // (E, w_blocks, num_kb)
  void* out;             // (M, n_out) bf16, fp32 or e4m3
  float* out_scales;     // (M, ceil(n_out / 128)), kSiluQuant
  unsigned int* err;
};

struct Tail {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t xfull[2];        // gated: every epilogue warp has written its amax[tile parity]
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  int total_tiles;
  int tile_start[kMaxExperts + 1];
  int off[kMaxExperts + 1];
  float amax[2][2][BM];     // [tile parity][column half][row]
};

constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulator.
__device__ __forceinline__ void umma_fp8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4: e4m3 A and B (format 0), both
// K-major, fp32 accumulator, shape M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Waits for the loads issued so far; v is what the last one filled, so that
// no use of it moves ahead of the wait.
__device__ __forceinline__ void tmem_wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                 "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Four rows of A (128 columns from c0) into 512 contiguous bytes with the
// swizzle of a tiled load (the map's box is 128 x 1).
__device__ __forceinline__ void tma_gather4(const CUtensorMap* map, uint64_t* bar, void* dst, int c0,
                                            int r0, int r1, int r2, int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(r0), "r"(r1), "r"(r2),
      "r"(r3)
      : "memory");
}

// acc + v * s on two neighbouring columns at once.
__device__ __forceinline__ void fma2(float2& acc, uint32_t v0, uint32_t v1, float s) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %4};\n\t"
      "mov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\t"
      "mov.b64 {%0, %1}, c;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "r"(v0), "r"(v1), "f"(s));
}

struct Tile {
  int e, row0, rows, n_blk;    // rows of the expert left from row0 on (may exceed BM)
};

// Tiles of an expert: row block fastest, so CTAs side by side share a
// weight tile through L2.
__device__ __forceinline__ Tile decode_tile(const Tail* st, int E, int n_tiles, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (st->tile_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Tile r;
  r.e = lo;
  const int local = t - st->tile_start[lo];
  const int mt = (st->tile_start[lo + 1] - st->tile_start[lo]) / n_tiles;
  r.n_blk = local / mt;
  r.row0 = st->off[lo] + (local - r.n_blk * mt) * BM;
  r.rows = st->off[lo + 1] - r.row0;
  return r;
}

// Bounded wait on the way out, regardless of the abort flag.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned int* err,
                                           unsigned int site) {
  int dummy = 0;
  mbar_wait(bar, parity, &dummy, err, site);
}

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ AMaps tmA, const __grid_constant__ CUtensorMap tmB,
                    const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * A_BYTES;
  Tail* st = reinterpret_cast<Tail*>(smem + STAGES * STAGE_BYTES);

  constexpr int BN_OUT = EPI == kSiluQuant ? 128 : 256;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const int n_tiles = (p.n_out + BN_OUT - 1) / BN_OUT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&st->full[s], 1);
      mbar_init(&st->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&st->tfull[a], 1);
      mbar_init(&st->tempty[a], EPI_WARPS);
      mbar_init(&st->xfull[a], EPI_WARPS);
    }
    mbar_init(&st->mma_done, 1);
    st->abort = 0;
    // offsets are device data: kept within [0, M] and in order, so that no
    // address below depends on their being right
    int acc = 0, at = p.offsets ? min(max(p.offsets[0], 0), p.M) : 0;
    for (int e = 0; e < E; ++e) {
      const int next = p.offsets ? min(max(p.offsets[e + 1], at), p.M) : p.M;
      st->off[e] = at;
      st->tile_start[e] = acc;
      acc += (next - at + BM - 1) / BM * n_tiles;
      at = next;
    }
    st->off[E] = at;
    st->tile_start[E] = acc;
    st->total_tiles = acc;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tmB);
  if (warp == 1) {
    tmem_alloc(&st->tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = st->tmem_base;
  const int total = st->total_tiles;
  volatile int* abort = &st->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0, used = 0, last_parity = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
      if (!__shfl_sync(0xffffffffu, lane == 0 ? static_cast<int>(!*abort) : 0, 0)) break;
      const Tile tl = decode_tile(st, E, n_tiles, t);
      const int rowB0 = tl.e * p.w_rows + tl.n_blk * BN_OUT;
      const int rowB1 = EPI == kSiluQuant ? rowB0 + p.up_row : rowB0 + 128;
      const int rows = min(BM, tl.rows);
      int tok[4] = {0, 0, 0, 0};
      int gather_lanes = 0, box = 0, a_bytes;
      if (p.gather) {
        gather_lanes = (rows + 3) >> 2;
        a_bytes = gather_lanes * 512;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = min(4 * lane + i, rows - 1);       // past the last row: that row again
          tok[i] = __ldg(p.perm + tl.row0 + r) / p.slots;
        }
      } else {
        while ((8 << box) < rows) ++box;
        a_bytes = (8 << box) * BK;
      }
      bool ok = true;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        int good = 1;
        if (lane == 0) {
          good = mbar_wait(&st->empty[stage], phase ^ 1u, abort, p.err, SITE_FP8_PRODUCER) ? 1 : 0;
          if (good) mbar_arrive_expect_tx(&st->full[stage], a_bytes + B_BYTES);
        }
        if (!__shfl_sync(0xffffffffu, good, 0)) { ok = false; break; }
        if (lane < gather_lanes)
          tma_gather4(&tmA.m[0], &st->full[stage], sA + stage * A_BYTES + lane * 512, kb * BK, tok[0],
                      tok[1], tok[2], tok[3]);
        if (lane == 0) {
          if (!p.gather)
            tma_load_2d(&tmA.m[box], &st->full[stage], sA + stage * A_BYTES, kb * BK, tl.row0);
          tma_load_2d(&tmB, &st->full[stage], sB + stage * B_BYTES, kb * BK, rowB0);
          tma_load_2d(&tmB, &st->full[stage], sB + stage * B_BYTES + B_BYTES / 2, kb * BK, rowB1);
          used |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
    // let every issued load land before the CTA can leave
    if (lane == 0)
      for (int s = 0; s < STAGES; ++s)
        if (used & (1u << s)) drain_wait(&st->full[s], (last_parity >> s) & 1u, p.err, SITE_FP8_PRODUCER);
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(BM, BN);
      int stage = 0;
      uint32_t phase = 0, i = 0;                  // i: blocks issued so far
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        for (int kb = 0; kb < p.num_kb; ++kb, ++i) {
          const uint32_t acc = i & 1u;
          if (!mbar_wait(&st->tempty[acc], ((i >> 1) & 1u) ^ 1u, abort, p.err, SITE_FP8_MMA) ||
              !mbar_wait(&st->full[stage], phase, abort, p.err, SITE_FP8_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + stage * A_BYTES);
          const uint32_t b0 = smem_u32(sB + stage * B_BYTES);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            umma_fp8(tmem + acc * BN, sw128_kmajor_desc(a0 + k * 32), sw128_kmajor_desc(b0 + k * 32),
                     idesc, k != 0 ? 1u : 0u);
          umma_commit(&st->empty[stage]);
          umma_commit(&st->tfull[acc]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // all MMAs issued by this thread complete before TMEM / smem go away
      umma_commit(&st->mma_done);
      drain_wait(&st->mma_done, 0, p.err, SITE_FP8_MMA);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;                   // TMEM lanes this warp may access
    const int half = (warp - 2) >> 2;
    const int r = quad * 32 + lane;              // row of the tile
    const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 64;
    uint32_t i = 0;                              // blocks read so far
    bool ok = true;
    int n = 0;                                   // tiles begun before this one
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++n) {
      const int parity = n & 1;
      const Tile tl = decode_tile(st, E, n_tiles, t);
      const bool live = quad * 32 < tl.rows;     // warp-uniform
      const bool rvalid = r < tl.rows;
      const int grow = tl.row0 + (rvalid ? r : 0);
      const int srow = p.perm ? __ldg(p.perm + grow) / p.slots : grow;
      const float* sa = p.sa + static_cast<size_t>(srow) * p.num_kb;
      const int b0 = EPI == kSiluQuant ? tl.n_blk : 2 * tl.n_blk;
      const int b1 = EPI == kSiluQuant ? p.up_block + tl.n_blk : min(b0 + 1, p.w_blocks - 1);
      const float* sw0 = p.sw + (static_cast<size_t>(tl.e) * p.w_blocks + b0) * p.num_kb;
      const float* sw1 = p.sw + (static_cast<size_t>(tl.e) * p.w_blocks + b1) * p.num_kb;
      float2 acc[64];                            // [0, 32) the first 64 columns, [32, 64) the second
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
      float na = __ldg(sa), n0 = __ldg(sw0), n1 = __ldg(sw1);
      for (int kb = 0; kb < p.num_kb; ++kb, ++i) {
        const float s0 = na * n0, s1 = na * n1;
        if (kb + 1 < p.num_kb) {                 // the next block's scales, behind this one's wait
          na = __ldg(sa + kb + 1);
          n0 = __ldg(sw0 + kb + 1);
          n1 = __ldg(sw1 + kb + 1);
        }
        const uint32_t buf = i & 1u;
        // every lane must agree before the warp-collective TMEM loads
        const bool got = mbar_wait(&st->tfull[buf], (i >> 1) & 1u, abort, p.err, SITE_FP8_EPILOGUE);
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        tc_fence_after();
        if (live) {
          const uint32_t src = tb + buf * BN;
          uint32_t v[2][16];
          tmem_ld16(src, v[0]);
          tmem_wait16(v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {          // 4 chunks of 16 columns of each half
            if (c < 7) tmem_ld16(src + ((c + 1) >> 2) * 128 + ((c + 1) & 3) * 16, v[(c + 1) & 1]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              fma2(acc[c * 8 + j], v[c & 1][2 * j], v[c & 1][2 * j + 1], c < 4 ? s0 : s1);
            if (c < 7) tmem_wait16(v[(c + 1) & 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->tempty[buf]);
      }
      if (!ok) break;

      if constexpr (EPI == kSiluQuant) {
        // columns [half * 64, half * 64 + 64) of the tile's 128
        const int col0 = tl.n_blk * 128 + half * 64;
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          const float g = j & 1 ? acc[j >> 1].y : acc[j >> 1].x;
          const float u = j & 1 ? acc[32 + (j >> 1)].y : acc[32 + (j >> 1)].x;
          const float v = col0 + j < p.n_out ? silu_bf16_epilogue(g) * u : 0.f;
          if (j & 1) acc[j >> 1].y = v; else acc[j >> 1].x = v;
          m = fmaxf(m, fabsf(v));
        }
        st->amax[parity][half][r] = m;
        // meet the other half's warps (a bounded wait: one of them may have given up)
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->xfull[parity]);
        if (!__all_sync(0xffffffffu, mbar_wait(&st->xfull[parity], (n >> 1) & 1u, abort, p.err,
                                               SITE_FP8_EPILOGUE)))
          break;
        const float s = fp8_scale(fmaxf(st->amax[parity][0][r], st->amax[parity][1][r]));
        const float inv = 1.f / s;
        if (rvalid) {
          uint8_t* q = static_cast<uint8_t*>(p.out) + static_cast<size_t>(grow) * p.n_out + col0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (col0 + 16 * c < p.n_out) {       // n_out is a multiple of 16
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = fp8_pack4(acc[8 * c + 2 * j].x * inv, acc[8 * c + 2 * j].y * inv,
                                 acc[8 * c + 2 * j + 1].x * inv, acc[8 * c + 2 * j + 1].y * inv);
              *reinterpret_cast<uint4*>(q + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          if (half == 0)
            p.out_scales[static_cast<size_t>(grow) * ((p.n_out + 127) / 128) + tl.n_blk] = s;
        }
      } else if (rvalid) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col0 = tl.n_blk * 256 + c * 128 + half * 64;
#pragma unroll
          for (int j = 0; j < 8; ++j) {          // 8 columns: n_out is a multiple of 8
            const int col = col0 + 8 * j;
            if (col >= p.n_out) continue;
            const float2* a = acc + c * 32 + 4 * j;
            const size_t o = static_cast<size_t>(grow) * p.n_out + col;
            if constexpr (EPI == kOutBf16) {
              uint4 w;
              __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
              for (int q = 0; q < 4; ++q) b[q] = __floats2bfloat162_rn(a[q].x, a[q].y);
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o) = w;
            } else {
              float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
              d[0] = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
              d[1] = make_float4(a[2].x, a[2].y, a[3].x, a[3].y);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Row-major (rows, cols) bytes, boxes of box_rows x 128 columns with the
// 128-byte swizzle; out-of-range elements read as zero.
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(BK), box_rows};
  const cuuint32_t estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int EPI>
cudaError_t launch_epi(const AMaps& a, const CUtensorMap& b, const Params& p, int grid,
                       cudaStream_t s) {
  // the shared-memory opt-in is a per-device function attribute
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      err = cudaFuncSetAttribute(gemm_fp8_kernel<EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemBytes));
      if (err != cudaSuccess) return err;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  return launch_k(gemm_fp8_kernel<EPI>, dim3(grid), dim3(THREADS), kSmemBytes, s, false, 1, a, b, p);
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmFp8Args& g, cudaStream_t s) {
  const bool gated = g.q_scales != nullptr;
  Params p{};
  p.offsets = g.offsets;
  p.perm = g.perm;
  p.slots = g.slots;
  p.gather = g.gather ? 1 : 0;
  p.M = g.M;
  p.E = g.E;
  p.n_out = g.N;
  p.num_kb = (g.K + BK - 1) / BK;
  const int blocks = (g.N + 127) / 128;
  p.w_rows = gated ? 2 * g.N : g.N;
  p.w_blocks = gated ? 2 * blocks : blocks;
  p.up_row = g.N;
  p.up_block = blocks;
  p.sa = g.a_scales;
  p.sw = g.w_scales;
  p.out = g.out;
  p.out_scales = g.q_scales;
  p.err = g.err;
  AMaps ma;
  CUtensorMap mb;
  for (int i = 0; i < kBoxes; ++i)
    if (!make_map(&ma.m[i], g.a, static_cast<uint64_t>(g.a_rows), static_cast<uint64_t>(g.K),
                  g.gather ? 1u : 8u << i))
      return cudaErrorInvalidValue;
  if (!make_map(&mb, g.w, static_cast<uint64_t>(g.E) * p.w_rows, static_cast<uint64_t>(g.K), 128u))
    return cudaErrorInvalidValue;
  const int bn_out = gated ? 128 : 256;
  const long long n_tiles = (g.N + bn_out - 1) / bn_out;
  // With at most 128 rows per expert on average (weight streaming) each
  // touched expert has one row block: size the grid so that every CTA takes
  // the same number of tiles.  Else bound the tiles from above.
  const long long touched = g.M < g.E ? g.M : g.E;
  long long tiles = (static_cast<long long>(g.M) / BM + touched) * n_tiles;
  if (g.M <= 128LL * g.E) tiles = touched * n_tiles;
  const long long sms = num_sms();
  const long long waves = (tiles + sms - 1) / sms;
  const int grid = static_cast<int>((tiles + waves - 1) / waves);
  if (gated) return launch_epi<kSiluQuant>(ma, mb, p, grid, s);
  if (g.out_f32) return launch_epi<kOutF32>(ma, mb, p, grid, s);
  return launch_epi<kOutBf16>(ma, mb, p, grid, s);
}

}  // namespace moe
