// Block-scaled e4m3 grouped GEMM on the sm_100a tensor cores.
//
//   C[i, n] = sum_kb sa[i, kb] sw[e][n / 128, kb] sum_{k in block kb} A[i, k] W[e][n, k]
//
// for the rows i of expert e (offsets), kb over blocks of 128 columns.  The
// inner sum of a block is four tcgen05.mma kind::f8f6f4 (K = 32 each) into a
// fresh fp32 accumulator in TMEM; the scales differ from block to block in
// both operands, so the outer sum is kept in fp32 registers: the epilogue
// warps read each block's accumulator and add it, times sa * sw, to their
// own, while the tensor cores work on the next ones.
//
// What limits such a kernel is the round trip accumulator ready -> read ->
// free -> next MMA, some 1100 cycles long with 256 columns against the 512
// that a block's MMAs take, and the epilogue warps' own chain of waits.  So the
// 256 weight rows of a tile are two halves of 128 that run apart from each
// other: an MMA warp, two TMEM buffers and four epilogue warps each.  Three
// forms, chosen by rows per expert (launch_gemm_fp8):
//   kOne   128 rows x 256 on one CTA;
//   kPair  256 rows x 256 on two CTAs: half the weight bytes per CTA;
//   kFew   32 rows x 256, for weight streaming: the MMAs are as tall as
//          kOne's, but only 32 rows of A are loaded (by token, with gather4,
//          where the rows are not sorted yet), and where tiles are few a
//          cluster shares out a tile's blocks and adds its sums over
//          distributed shared memory.  The second half's rows are made
//          accumulator rows 32..63 (its A operand starts 32 rows early), so
//          that four warps read a block, a half and a weight block each, and
//          no longer take longer than its MMAs (16 rows of 4096 x 14336: 20.7
//          -> 18.7 us).
// 8192 rows of 4096 x 14336 (kPair): 435 us in short runs, 2.21 PFLOP/s at 1.45
// GHz with the tensor pipe active in 64% of cycles; 500 us in runs of seconds,
// at the board's power limit.  9973 rows over 64 experts of 1408 x 2048,
// unevenly (kOne): 60 us, 70 in runs of seconds.  16 rows of 4096 x 14336 (kFew):
// 19 us, the weights at 3.1 TB/s.
//
// One persistent CTA per SM (or pair of CTAs per two SMs), 384 threads:
//   warp 0      TMA producer: A rows x 128 columns and B rows (256, or this CTA's
//               128 of a pair) x 128 per block into a ring.  Without a pair,
//               a row block of few rows is loaded by a lower box (8 to 128
//               rows); the rest of the stage keeps what it held and feeds
//               only accumulator rows that are never read;
//   warps 1, 2  issue the MMAs of one half each (M = 128 or 256, N = 128);
//               warp 1 allocates the 512 TMEM columns;
//   warp 3      scale loader: 8 blocks' scales of the CTA's 128 rows at a
//               time, read along the rows and left by block in shared memory
//               (two such groups), so that an epilogue warp's read is one
//               conflict-free access;
//   warps 4..11 epilogue: four warps per half, 32 TMEM lanes (rows) each, all
//               128 columns of the half: 128 fp32 sums per thread.  In kFew
//               the warps of lanes 0..63 read, 64 sums per thread, and all
//               eight finish the rows.
// Registers move from warps 0..3 (72 each) to the epilogue (216): 128 * 72 +
// 256 * 216 of the launch's 384 * 168.
//
// A half is 64 rows of the first 128-row weight block and 64 of the second,
// so in the gated form (B = 128 gate rows and the matching 128 up rows) it
// holds the gate and the up value of the same 64 features.  On a pair each
// CTA stages its own A rows and one of the two weight blocks (cta_group::2
// reads both CTAs' shared memory): 32 KB per block and CTA instead of 48.
//
// Epilogues (columns of the output per tile):
//   kOutBf16, kOutF32   the sums, rounded once (256 columns);
//   kOutF16             the sums in fp16 times a power of two, one for each 64
//                       columns of a row: what the experts' outputs are kept
//                       in until they are summed.  bf16 would take the same
//                       bytes and round eight times as coarsely;
//   kSiluQuant          h = silu(gate) * up in fp32, then e4m3 with one scale
//                       for the row's 128 columns: a row's largest |h| is a
//                       maximum over the two threads (halves) that share it.
//
// Rows outside [offsets[0], offsets[E]) are not touched.  Every mbarrier wait
// is bounded (common.cuh); after a timeout the epilogue runs through its loop
// without waiting, so that no warp is left at a barrier.
#include <cuda_fp16.h>
#include <float.h>

#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

// The roles in the device error word, behind common.cuh's.
enum : unsigned int {
  SITE_FP8_PRODUCER = 1u << 18,
  SITE_FP8_MMA = 1u << 19,
  SITE_FP8_EPILOGUE = 1u << 20,
  SITE_FP8_SCALES = 1u << 21,
};
static_assert(SITE_FP8_PRODUCER == SITE_PROBE << 1, "bits 8 to 17 are common.cuh's");

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Up to 4096 tries (0.1 ms and more) in a loop of four instructions, for waits
// on a short loop's critical path: mbar_wait reads %globaltimer as soon as its
// first try fails, and a try without success so far is the usual case there.
// False is not final: go on with mbar_wait, out of the usual path.
__device__ __forceinline__ bool mbar_try_loop(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n\t"
      "TRY_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 4096;\n\t"
      "@q bra TRY_%=;\n\t"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// The same for a whole (converged) warp: lane 0 tries, a vote makes the result
// uniform (and no more than that: see warp_wait).
__device__ __forceinline__ bool mbar_try_loop_warp(uint32_t bar, uint32_t parity, int lane) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .u32 n;\n\t"
      "setp.eq.u32 e, %3, 0;\n\t"
      "setp.ne.u32 p, 0, 0;\n\t"
      "mov.u32 n, 0;\n\t"
      "TRY_%=:\n\t"
      "@e mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.any.pred p, p, 0xffffffff;\n\t"
      "@p bra.uni DONE_%=;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 4096;\n\t"
      "@q bra.uni TRY_%=;\n\t"
      "DONE_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(static_cast<uint32_t>(lane))
      : "memory");
  return ok != 0;
}

// Tries two barriers at once: their latencies overlap, and one branch on the
// result serves for both.
__device__ __forceinline__ bool mbar_try_both(uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                              uint32_t parity1) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar0), "r"(parity0), "r"(bar1), "r"(parity1)
      : "memory");
  return ok != 0;
}

constexpr int BM = 128;                        // rows per CTA
constexpr int BK = 128;                        // bytes = e4m3 values = one scale block
constexpr int BN = 256;                        // weight rows per tile
constexpr int BH = 128;                        // columns of a half
constexpr int EPI_WARP0 = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int SCALE_KB = 8;                    // blocks per group of scales
constexpr uint32_t TMEM_COLS = 512;
constexpr int kBoxes = 5;                      // A boxes of 8, 16, 32, 64 and 128 rows
constexpr int kRowGroup = 16;                  // row blocks that share a pass over the weights


// kOne: a CTA, 128 rows.  kPair: a CTA pair, 256 rows.  kFew: a CTA, 32 rows.
enum { kOne = 0, kPair = 1, kFew = 2 };

template <int MODE>
struct Cfg {
  static constexpr int TILE_M = MODE == kPair ? 2 * BM : MODE == kFew ? 32 : BM;
  static constexpr int STAGES = MODE == kPair ? 6 : MODE == kFew ? 5 : 4;
  static constexpr int A_BYTES = (MODE == kFew ? TILE_M : BM) * BK;
  static constexpr int B_BYTES = (MODE == kPair ? BN / 2 : BN) * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int QUADS = MODE == kFew ? 1 : 4;   // groups of 32 rows
  static constexpr int READERS = MODE == kFew ? 2 : 4; // warps that read a half's accumulators
};

enum { kOutBf16 = 0, kOutF32 = 1, kSiluQuant = 2, kOutF16 = 3 };

struct AMaps {
  CUtensorMap m[kBoxes];
};

struct Params {
  const int* offsets;    // (E + 1) first row of each expert, or null: one expert, all M rows
  const int* perm;       // row -> (token, slot): the row of the scales is perm[row] / slots; or null
  int slots;
  const int64_t* selected;   // set (kFew, gated, M <= THREADS): every CTA sorts the M slots itself
  int* offsets_out;          // and the first one writes offsets and the slots' rows
  int* pos_out;
  int gather;            // 1: the rows of A are fetched by token too (its map is one row high)
  int M, E;
  int n_out;             // output columns
  int num_kb;
  int w_rows;            // weight rows per expert
  int w_blocks;          // scale rows per expert
  int up_row, up_block;  // first up row and scale row of an expert (gated)
  int split;             // kFew: CTAs of a cluster that share a tile's blocks
  const float* sa;       // (rows, num_kb)
  const float* sw;       // (E, w_blocks, num_kb)
  void* out;             // (M, n_out) bf16, fp32 or e4m3
  float* out_scales;     // (M, ceil(n_out / 128)), kSiluQuant; (M, ceil(n_out / 64)), kOutF16
  unsigned int* err;
};

constexpr int kPartStride = BN + 4;

template <int MODE>
struct Tail {
  uint64_t full[Cfg<MODE>::STAGES];    // the stage is loaded (pair: the leader's, for both CTAs)
  uint64_t empty[Cfg<MODE>::STAGES];   // both halves' MMAs have read it
  alignas(16) uint64_t tfull[2][2];    // [half][buffer] accumulator ready
  alignas(16) uint64_t tempty[2][2];                // its readers are done (pair: the leader's, for both CTAs)
  uint64_t xfull[2];        // kFew: the tile's sums are in part; gated, else: its amax[tile parity] is in place
  uint64_t xempty;          // kFew: the tile's rows are finished, part is free
  uint64_t sfull[2];        // a group of scales is in place
  uint64_t sempty[2];       // every epilogue warp is done with it
  uint64_t mma_done[2];
  uint32_t tmem_base;
  int abort;
  int total_tiles, workers;
  int tile_start[kMaxExperts + 1];
  int off[kMaxExperts + 1];
  alignas(16) float amax[2][2][MODE == kFew ? 1 : BM];   // [tile parity][half][row]
  alignas(16) float sa[2][SCALE_KB][32 * Cfg<MODE>::QUADS];
  int perm[MODE == kFew ? THREADS : 1];
  // kFew: the tile's sums, a row of 256 columns after the other; 16 bytes more
  // per row keep row-per-lane accesses free of bank conflicts
  alignas(16) float part[MODE == kFew ? 32 : 1][kPartStride];
  alignas(16) uint8_t stage[MODE == kFew ? 1 : EPI_WARPS][2048];   // an epilogue warp's way out
  alignas(16) float2 sw[2][SCALE_KB];   // of the first and the second 128 weight rows
};

template <int MODE>
constexpr size_t smem_bytes() {
  return 1024 + Cfg<MODE>::STAGES * Cfg<MODE>::STAGE_BYTES + sizeof(Tail<MODE>);
}
static_assert(smem_bytes<kOne>() <= 227 * 1024 && smem_bytes<kPair>() <= 227 * 1024 &&
              smem_bytes<kFew>() <= 227 * 1024, "shared memory");
// An M = 128 MMA of kFew reads 96 rows around the stage's 32, up to 32 of them
// in front (accumulator rows that are never looked at): they have to be there.
static_assert(sizeof(Tail<kFew>) >= 96 * BK && Cfg<kFew>::STAGES * Cfg<kFew>::B_BYTES >= 32 * BK,
              "A reads stay inside this CTA's shared memory");

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Four floats at the shared-memory address `addr` of the cluster's CTA `rank`.
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, int rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t map_to_rank0(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// An arrival where `on` holds, as a predicated instruction instead of a
// branch; of a pair on the leader's barrier (a cluster address).  What that
// hands over are TMEM columns that tcgen05.wait::ld has seen read, no memory:
// a release at cluster scope would flush this thread's accesses, 1300 cycles
// in the epilogue's loop.
template <bool CLUSTER>
__device__ __forceinline__ void arrive_if(bool on, uint32_t bar) {
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(on))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(on))
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulator.
template <bool PAIR>
__device__ __forceinline__ void umma_fp8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives once on `bar` (of a pair in the CTAs of the mask) when the MMAs that
// this thread has issued are complete.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar, uint16_t ctas = 3) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(ctas)
        : "memory");
  else
    umma_commit(bar);
}

template <bool PAIR>
__device__ __forceinline__ void tmem_get(uint32_t* dst) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, TMEM_COLS);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t taddr) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(TMEM_COLS)
                 : "memory");
  else
    tmem_dealloc(taddr, TMEM_COLS);
}

// Tiled load whose bytes are counted on the barrier at `bar` (a cluster
// address; of a pair the leader's).
template <bool PAIR>
__device__ __forceinline__ void load_box(const CUtensorMap* map, uint32_t bar, void* dst, int c0, int c1) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4: e4m3 A and B (format 0), both
// K-major, fp32 accumulator, shape M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
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

// Two neighbouring columns in one 64-bit register.  fma.rn.f32x2 does the work
// of two FMAs in one issue slot (at their rate, two cycles).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 both(float s) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s));
  return r;
}
// (volatile: x and y come from a TMEM load, and no use of them may move ahead
// of the wait for it)
__device__ __forceinline__ void fma2(f32x2& acc, uint32_t x, uint32_t y, f32x2 s) {
  asm volatile("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
               : "+l"(acc)
               : "r"(x), "r"(y), "l"(s));
}
__device__ __forceinline__ f32x2 pack(float2 v) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 unpack(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

struct Tile {
  int e, row0, rows, n_blk;    // rows of the expert left from row0 on (may exceed the tile's)
};

// Tiles of an expert: in groups of kRowGroup row blocks, weight block by
// weight block, the row block fastest.  CTAs side by side then share weight
// tiles through L2, and a group's rows stay there while the weights pass by
// once per group.
__device__ __forceinline__ Tile decode_tile(const int* tile_start, const int* off, int E, int n_tiles,
                                            int tile_m, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  Tile r;
  r.e = lo;
  const int local = t - tile_start[lo];
  const int mt = (tile_start[lo + 1] - tile_start[lo]) / n_tiles;
  const int g0 = local / (kRowGroup * n_tiles) * kRowGroup;      // the group's first row block
  const int in = local - g0 * n_tiles;
  const int gm = min(kRowGroup, mt - g0);
  r.n_blk = in / gm;
  r.row0 = off[lo] + (g0 + in - r.n_blk * gm) * tile_m;
  r.rows = off[lo + 1] - r.row0;
  return r;
}

// Bounded wait on the way out, regardless of the abort flag.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, unsigned int* err,
                                           unsigned int site) {
  int dummy = 0;
  mbar_wait(bar, parity, &dummy, err, site);
}

// Bounded wait with a short loop first.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* err,
                                     unsigned int site) {
  if (__builtin_expect(mbar_try_loop(smem_u32(bar), parity), 1)) return true;
  return mbar_wait(bar, parity, abort, err, site);
}
// The same for a converged warp, with the same result in every lane.  The vote
// tells the lanes what lane 0 has seen but orders no memory; __syncwarp makes
// what the barrier hands over theirs too.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int lane, volatile int* abort,
                                          unsigned int* err, unsigned int site) {
  if (__builtin_expect(mbar_try_loop_warp(smem_u32(bar), parity, lane), 1)) {
    __syncwarp();
    return true;
  }
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, site));
}

// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// The power of two that brings a block with largest finite magnitude amax to
// the top of fp16's range (its inverse is what is stored); 1 for zeros.
__device__ __forceinline__ float f16_scale(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23);         // biased exponent, amax >= 0
  if (e == 0) return 1.f;
  return __uint_as_float(static_cast<uint32_t>(min(max(127 + 14 - (e - 127), 1), 254)) << 23);
}
// |x|, or 0 for infinities and NaN: they stay what they are whatever the scale.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;
}
__device__ __forceinline__ uint32_t pack_f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 64 bytes of each of 32 rows, a row per lane in w, to rows `row_bytes` apart
// from `out` on, at byte `at` of each: through 2 KB of shared memory, so that
// four lanes store a row's 64 bytes (16 bytes to 32 rows at once, straight from
// the lanes, took 1.6 us a tile).  Stores rows below `rows`, bytes below
// row_bytes.  16-byte unit u of row r lies at u ^ (r / 2 % 4): no bank
// conflicts in either direction.
__device__ __forceinline__ void store_rows(uint8_t* stg, int lane, const uint4 (&w)[4], uint8_t* out,
                                           size_t row_bytes, size_t at, int rows) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(stg + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) = w[u];
  __syncwarp();
  const int u = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4*>(stg + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
    if (r < rows && at + 16 * u < row_bytes) *reinterpret_cast<uint4*>(out + r * row_bytes + at + 16 * u) = v;
  }
  __syncwarp();
}

// One row of a tile from its sums, by a warp: a lane has columns 4 * lane .. + 3
// of the first (v0) and of the second weight block (v1).
template <int EPI>
__device__ __forceinline__ void finish_row(const Params& p, const Tile& tl, int r, int lane, float4 v0,
                                           float4 v1) {
  const size_t grow = static_cast<size_t>(tl.row0 + r) * p.n_out;
  if constexpr (EPI == kSiluQuant) {
    const int col = tl.n_blk * 128 + 4 * lane;
    const bool in = col < p.n_out;               // n_out is a multiple of 16
    float4 h;
    h.x = in ? silu_bf16_epilogue(v0.x) * v1.x : 0.f;
    h.y = in ? silu_bf16_epilogue(v0.y) * v1.y : 0.f;
    h.z = in ? silu_bf16_epilogue(v0.z) * v1.z : 0.f;
    h.w = in ? silu_bf16_epilogue(v0.w) * v1.w : 0.f;
    const float m = warp_max(fmaxf(fmaxf(fabsf(h.x), fabsf(h.y)), fmaxf(fabsf(h.z), fabsf(h.w))));
    const float s = fp8_scale(m);
    const Fp8Divisor over(m, s);
    if (in)
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + grow + col) =
          fp8_pack4(over(h.x), over(h.y), over(h.z), over(h.w));
    if (lane == 0) p.out_scales[static_cast<size_t>(tl.row0 + r) * ((p.n_out + 127) / 128) + tl.n_blk] = s;
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = tl.n_blk * 256 + c * 128 + 4 * lane;
      const float4 v = c ? v1 : v0;
      if constexpr (EPI == kOutF16) {
        const bool in = col < p.n_out;           // columns past it: another expert's, not to be looked at
        float m = in ? fmaxf(fmaxf(finite_abs(v.x), finite_abs(v.y)),
                             fmaxf(finite_abs(v.z), finite_abs(v.w))) : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = f16_scale(m);
        if (in)
          *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + grow + col) =
              make_uint2(pack_f16x2(v.x * s, v.y * s), pack_f16x2(v.z * s, v.w * s));
        if (in && (lane & 15) == 0)
          p.out_scales[static_cast<size_t>(tl.row0 + r) * ((p.n_out + 63) / 64) + col / 64] = 1.f / s;
        continue;
      }
      if (col >= p.n_out) continue;              // n_out is a multiple of 8
      if constexpr (EPI == kOutBf16) {
        uint2 w;
        reinterpret_cast<__nv_bfloat162*>(&w)[0] = __floats2bfloat162_rn(v.x, v.y);
        reinterpret_cast<__nv_bfloat162*>(&w)[1] = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + grow + col) = w;
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + grow + col) = v;
      }
    }
  }
}

template <int EPI, int MODE>
__global__ void __launch_bounds__(THREADS, 1)
    gemm_fp8_kernel(const __grid_constant__ AMaps tmA, const __grid_constant__ CUtensorMap tmB,
                    const Params p) {
  using C = Cfg<MODE>;
  constexpr bool PAIR = MODE == kPair;
  constexpr int STAGES = C::STAGES, A_BYTES = C::A_BYTES;
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned by its address in the shared window: the same offset in
  // both CTAs of a pair
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = MODE == kFew ? smem + STAGES * C::B_BYTES : smem;
  uint8_t* sB = MODE == kFew ? smem : smem + STAGES * A_BYTES;
  Tail<MODE>* st = reinterpret_cast<Tail<MODE>*>(smem + STAGES * C::STAGE_BYTES);

  constexpr int BN_OUT = EPI == kSiluQuant ? 128 : 256;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  // this CTA (or pair, or cluster) takes tiles worker, worker + workers, ...;
  // with split blocks one tile only: the grid covers every possible one
  const int split = MODE == kFew ? p.split : 1;
  const int share = MODE == kFew && split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int most = PAIR ? gridDim.x >> 1 : split > 1 ? 1 << 30 : gridDim.x;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x / split;
  const int kb_lo = share * p.num_kb / split, kb_hi = (share + 1) * p.num_kb / split;
  const int E = p.E;
  const int n_tiles = (p.n_out + BN_OUT - 1) / BN_OUT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&st->full[s], 1);
      mbar_init(&st->empty[s], 2);
    }
    for (int a = 0; a < 2; ++a) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&st->tfull[a][b], 1);
        mbar_init(&st->tempty[a][b], (PAIR ? 2 : 1) * C::READERS);
      }
      mbar_init(&st->xfull[a], 2 * C::READERS);
      if (a == 0) mbar_init(&st->xempty, EPI_WARPS);
      mbar_init(&st->sfull[a], 1);
      mbar_init(&st->sempty[a], 2 * C::READERS);
      mbar_init(&st->mma_done[a], 1);
    }
    st->abort = 0;
    mbar_fence_init();
  }
  // A small batch's slots are sorted by expert here, a thread per slot, by every
  // CTA for itself (stable: by slot): one launch less, 4 us.
  constexpr bool kSorts = EPI == kSiluQuant && MODE == kFew;
  const bool sorts = kSorts && p.selected != nullptr;
  int* count = reinterpret_cast<int*>(st->part);                   // an expert's slots
  int* warp_count = count + kMaxExperts;                           // of a warp's 32, [warp][expert]
  int expert = -1, rank_in = 0;
  if constexpr (kSorts) {
    if (sorts) {
      const int64_t v = threadIdx.x < p.M ? __ldg(p.selected + threadIdx.x) : -1;
      if (v >= 0 && v < E) expert = static_cast<int>(v);
      for (int i = threadIdx.x; i < (1 + THREADS / 32) * kMaxExperts; i += THREADS) count[i] = 0;
      __syncthreads();
      const unsigned int same = __match_any_sync(0xffffffffu, expert);
      rank_in = __popc(same & ((1u << lane) - 1u));
      if (expert >= 0 && rank_in == 0) {
        warp_count[warp * kMaxExperts + expert] = __popc(same);
        atomicAdd(&count[expert], __popc(same));                   // integers: the order is free
      }
      __syncthreads();
    }
  }
  if (warp == 2) {
    // The tile table, a lane for eight experts.
    int o[9];
    if (sorts) {
      int sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += count[lane * 8 + i];
      int incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      o[0] = incl - sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i + 1] = o[i] + count[lane * 8 + i];
    } else {
      // Offsets are device data: kept within [0, M] and in order (a running
      // maximum), so that no address below depends on their being right.
#pragma unroll
      for (int i = 0; i < 9; ++i) {
        const int e = lane * 8 + i;
        o[i] = p.offsets && e <= E ? min(max(__ldg(p.offsets + e), 0), p.M) : (e == 0 ? 0 : p.M);
        if (i > 0) o[i] = max(o[i], o[i - 1]);
      }
      int high = o[8];                           // over the lanes before
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, high, d);
        if (lane >= d) high = max(high, v);
      }
      high = __shfl_up_sync(0xffffffffu, high, 1);
      if (lane == 0) high = 0;
#pragma unroll
      for (int i = 0; i < 9; ++i) o[i] = max(o[i], high);
    }
    int tiles[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      tiles[i] = lane * 8 + i < E ? (o[i + 1] - o[i] + C::TILE_M - 1) / C::TILE_M * n_tiles : 0;
      sum += tiles[i];
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
      if (e <= E) {
        st->off[e] = o[i];
        st->tile_start[e] = at;
      }
      at += tiles[i];
    }
    if (lane == 31) {
      // With as many waves as all workers would need, as few of them as get the
      // same number of tiles each: the rest would only share the first waves'
      // bandwidth (a decode step over 64 experts: 97 us, with all of them 99).
      const int waves = max(1, (at + most - 1) / most);
      const int workers = split > 1 ? most : max(1, (at + waves - 1) / waves);
      st->workers = workers;
      st->total_tiles = worker < workers ? at : 0;         // 0: none for this CTA
      if (E == kMaxExperts) {
        st->off[E] = o[8];
        st->tile_start[E] = at;
      }
    }
  }
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tmB);
  if (warp == 1) tmem_get<PAIR>(&st->tmem_base);
  if constexpr (kSorts) {
    if (sorts) {
      __syncthreads();
      int row = -1;
      if (expert >= 0) {
        row = st->off[expert] + rank_in;
        for (int w = 0; w < warp; ++w) row += warp_count[w * kMaxExperts + expert];
        st->perm[row] = threadIdx.x;
      }
      if (blockIdx.x == 0) {
        if (threadIdx.x < p.M) p.pos_out[threadIdx.x] = row;
        if (threadIdx.x <= E) p.offsets_out[threadIdx.x] = st->off[threadIdx.x];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();      // the leader's barriers exist before the peer uses them
  tc_fence_after();

  const uint32_t tmem = st->tmem_base;
  const int total = st->total_tiles, workers = st->workers;
  volatile int* abort = &st->abort;
  auto slot_of = [&](int row) { return sorts ? st->perm[row] : __ldg(p.perm + row); };
  auto tile_of = [&](int t) { return decode_tile(st->tile_start, st->off, E, n_tiles, C::TILE_M, t); };

  // (each register split dominates its warps' code, so that the compiler
  // allots their registers by it)
  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // One elected lane, as in the MMA warps; gathered rows are fetched by all.
    int stage = 0;
    uint32_t phase = 0, used = 0, last_parity = 0;
    auto step = [&] {
      used |= 1u << stage;
      last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == STAGES) { stage = 0; phase ^= 1u; }
    };
    // The stage's weight rows.  Alone, a CTA holds rows 0..63 of both weight
    // blocks, then rows 64..127 (the halves; the map's box has 64 rows); of a
    // pair, each CTA holds one block.
    auto load_b = [&](const Tile& tl, int kb, uint32_t bar) {
      const int row_b0 = tl.e * p.w_rows + tl.n_blk * BN_OUT;
      const int row_b1 = EPI == kSiluQuant ? row_b0 + p.up_row : row_b0 + 128;
      uint8_t* b = sB + stage * C::B_BYTES;
      if constexpr (PAIR) {
        load_box<PAIR>(&tmB, bar, b, kb * BK, rank == 0 ? row_b0 : row_b1);
      } else {
        load_box<PAIR>(&tmB, bar, b, kb * BK, row_b0);
        load_box<PAIR>(&tmB, bar, b + 64 * BK, kb * BK, row_b1);
        load_box<PAIR>(&tmB, bar, b + 128 * BK, kb * BK, row_b0 + 64);
        load_box<PAIR>(&tmB, bar, b + 192 * BK, kb * BK, row_b1 + 64);
      }
    };
    bool ok = true;
    if (MODE == kFew && p.gather) {
      for (int t = worker; t < total && ok; t += workers) {
        const Tile tl = tile_of(t);
        const int rows = min(C::TILE_M, tl.rows);
        const int fetchers = (rows + 3) >> 2;    // lanes with rows, four each
        int tok[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)              // past the last row: that row again
          tok[i] = slot_of(tl.row0 + min(4 * lane + i, rows - 1)) / p.slots;
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if (!warp_wait(&st->empty[stage], phase ^ 1u, lane, abort, p.err, SITE_FP8_PRODUCER)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(&st->full[stage], fetchers * 512 + C::B_BYTES);
            load_b(tl, kb, smem_u32(&st->full[stage]));
          }
          __syncwarp();        // the bytes are expected before any row can land
          if (lane < fetchers)
            tma_gather4(&tmA.m[0], &st->full[stage], sA + stage * A_BYTES + lane * 512, kb * BK, tok[0],
                        tok[1], tok[2], tok[3]);
          step();
        }
      }
      used = lane == 0 ? used : 0u;
    } else if (elect_one()) {
      for (int t = worker; t < total && ok; t += workers) {
        const Tile tl = tile_of(t);
        int box = kBoxes - 1;
        if constexpr (!PAIR)
          for (box = 0; (8 << box) < min(C::TILE_M, tl.rows);) ++box;
        const uint32_t tx = PAIR ? 2 * C::STAGE_BYTES : (8 << box) * BK + C::B_BYTES;
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if (!wait(&st->empty[stage], phase ^ 1u, abort, p.err, SITE_FP8_PRODUCER)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&st->full[stage], tx);
          const uint32_t bar = PAIR ? map_to_rank0(&st->full[stage]) : smem_u32(&st->full[stage]);
          load_box<PAIR>(&tmA.m[box], bar, sA + stage * A_BYTES, kb * BK,
                         tl.row0 + static_cast<int>(rank) * BM);
          load_b(tl, kb, bar);
          step();
        }
      }
    }
    // Let every issued load land before the CTA can leave: the leader sees
    // them on its full barriers; a peer's complete on the leader's, so the
    // peer waits for the MMAs to have released its stages.
    for (int s = 0; s < STAGES; ++s)
      if (used & (1u << s))
        drain_wait(rank == 0 ? &st->full[s] : &st->empty[s], (last_parity >> s) & 1u, p.err,
                   SITE_FP8_PRODUCER);
  } else if (warp < 3) {
    // ----------------------------------------------------------------- MMA
    // One elected lane runs the loop: elect.sync tells the compiler that the
    // operands of tcgen05.mma are uniform (with `lane == 0` an issue takes
    // three times as long).
    const int half = warp - 1;
    constexpr uint32_t idesc = idesc_e4m3_f32(PAIR ? 2 * BM : BM, BH);
    if (rank == 0 && elect_one()) {
      // kFew: the second half's rows become accumulator rows 32..63, which other
      // warps can read
      const uint64_t da = sw128_kmajor_desc(smem_u32(sA) - (MODE == kFew ? half * 32 * BK : 0));
      const uint64_t db = sw128_kmajor_desc(smem_u32(sB) + half * (PAIR ? 64 : 128) * BK);
      const uint32_t d0 = tmem + half * 2 * BH;
      const uint32_t full0 = smem_u32(&st->full[0]), tempty0 = smem_u32(&st->tempty[half][0]);
      int stage = 0;
      uint32_t phase = 0, i = 0;                  // i: blocks issued so far
      bool ok = true;
      for (int t = worker; t < total && ok; t += workers) {
        for (int kb = kb_lo; kb < kb_hi; ++kb, ++i) {
          const uint32_t buf = i & 1u;
          const uint32_t tpar = ((i >> 1) & 1u) ^ 1u;
          if (!mbar_try_both(full0 + 8 * stage, phase, tempty0 + 8 * buf, tpar)) {
            if (!wait(&st->full[stage], phase, abort, p.err, SITE_FP8_MMA) ||
                !wait(&st->tempty[half][buf], tpar, abort, p.err, SITE_FP8_MMA)) {
              ok = false;
              break;
            }
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)      // 32 bytes further: +2 in 16-byte units
            umma_fp8<PAIR>(d0 + buf * BH, da + (stage * A_BYTES >> 4) + 2 * k,
                           db + (stage * C::B_BYTES >> 4) + 2 * k, idesc, k != 0 ? 1u : 0u);
          commit<PAIR>(&st->tfull[half][buf]);
          commit<PAIR>(&st->empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // All MMAs issued by this thread complete before TMEM / smem go away.  Of a
      // pair the leader alone is told: only it waits, and an arrival that the peer
      // does not wait for could reach it after it has left.
      commit<PAIR>(&st->mma_done[half], 1);
      drain_wait(&st->mma_done[half], 0, p.err, SITE_FP8_MMA);
    }
  } else if (warp == 3) {
    // -------------------------------------------------------- scale loader
    // A group's loads are issued before the wait for its place in shared
    // memory, so that their latency passes while the group before is used.
    const bool vec = ((p.num_kb | kb_lo) & 3) == 0;   // a row's scales start at 16 bytes
    const int k = lane & 7;                      // lanes 0..7: the first weight block's, 8..15: the second's
    const float* sw = nullptr;
    const float* sa[C::QUADS];
    float va[C::QUADS][SCALE_KB], vw = 0.f;
    auto point = [&](int t) {                    // at tile t
      const Tile tl = tile_of(t);
      const int b0 = EPI == kSiluQuant ? tl.n_blk : 2 * tl.n_blk;
      const int b1 = EPI == kSiluQuant ? p.up_block + tl.n_blk : min(b0 + 1, p.w_blocks - 1);
      sw = p.sw + (static_cast<size_t>(tl.e) * p.w_blocks + (lane & 8 ? b1 : b0)) * p.num_kb;
#pragma unroll
      for (int h = 0; h < C::QUADS; ++h) {       // past the last row: that row again
        const int grow = tl.row0 + min(static_cast<int>(rank) * BM + h * 32 + lane, tl.rows - 1);
        sa[h] = p.sa + static_cast<size_t>(p.perm ? slot_of(grow) / p.slots : grow) * p.num_kb;
      }
    };
    auto fetch = [&](int k0) {                   // past the last block: that block again
      if (vec) {
#pragma unroll
        for (int h = 0; h < C::QUADS; ++h)
#pragma unroll
          for (int q = 0; q < SCALE_KB / 4; ++q) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(sa[h] + min(k0 + 4 * q, p.num_kb - 4)));
            va[h][4 * q] = v.x;
            va[h][4 * q + 1] = v.y;
            va[h][4 * q + 2] = v.z;
            va[h][4 * q + 3] = v.w;
          }
      } else {
#pragma unroll
        for (int h = 0; h < C::QUADS; ++h)
#pragma unroll
          for (int q = 0; q < SCALE_KB; ++q) va[h][q] = __ldg(sa[h] + min(k0 + q, p.num_kb - 1));
      }
      vw = __ldg(sw + min(k0 + k, p.num_kb - 1));
    };
    int t = worker, k0 = kb_lo;
    if (t < total) {
      point(t);
      fetch(k0);
    }
    for (uint32_t g = 0; t < total; ++g) {       // g: groups stored so far
      const uint32_t buf = g & 1u;
      if (!warp_wait(&st->sempty[buf], ((g >> 1) & 1u) ^ 1u, lane, abort, p.err, SITE_FP8_SCALES)) break;
#pragma unroll
      for (int h = 0; h < C::QUADS; ++h)
#pragma unroll
        for (int q = 0; q < SCALE_KB; ++q) st->sa[buf][q][h * 32 + lane] = va[h][q];
      if (lane < 16) (lane & 8 ? st->sw[buf][k].y : st->sw[buf][k].x) = vw;
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->sfull[buf]);
      k0 += SCALE_KB;
      if (k0 >= kb_hi) {
        k0 = kb_lo;
        t += workers;
        if (t < total) point(t);
      }
      if (t < total) fetch(k0);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;                   // TMEM lanes this warp may access
    const int sub = (warp - EPI_WARP0) >> 2;
    // kFew: half h has its rows in lanes 32 h .. 32 h + 31, whose two warps take
    // the columns of a weight block each
    const int half = MODE == kFew ? quad : sub;
    const int r = MODE == kFew ? lane : quad * 32 + lane;     // row of this CTA's
    // the buffer to read next: its columns, its barriers (8 bytes apart at
    // multiples of 16) and the parity of its turn
    uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 2 * BH + (MODE == kFew ? 64 * sub : 0);
    uint32_t tfull = smem_u32(&st->tfull[half][0]);
    uint32_t tempty = PAIR ? map_to_rank0(&st->tempty[half][0]) : smem_u32(&st->tempty[half][0]);
    uint32_t par = 0;
    uint32_t g = 0;                              // groups of scales taken so far
    int n = 0;                                   // tiles begun before this one
    // kFew: the rows of tile tl that are this warp's, from the sums in part
    auto few_rows = [&](const Tile& tl, int n) {
      warp_wait(&st->xfull[0], n & 1u, lane, abort, p.err, SITE_FP8_EPILOGUE);
      const int rows = min(C::TILE_M, tl.rows);
      for (int r = warp - EPI_WARP0; r < rows; r += EPI_WARPS) {
        const float4* src = reinterpret_cast<const float4*>(st->part[r]) + lane;
        finish_row<EPI>(p, tl, r, lane, src[0], src[32]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->xempty);
    };
    const bool reads = MODE != kFew || quad < 2;
    if (!reads && split == 1)
      for (int t = worker, m = 0; t < total; t += workers, ++m) few_rows(tile_of(t), m);
    for (int t = reads ? worker : total; t < total; t += workers, ++n) {
      const Tile tl = tile_of(t);
      const int rows = min(tl.rows - static_cast<int>(rank) * BM, MODE == kFew ? C::TILE_M : BM);
      const bool live = MODE == kFew || quad * 32 < rows;      // warp-uniform
      const bool rvalid = r < rows;
      const int grow = tl.row0 + static_cast<int>(rank) * BM + (rvalid ? r : 0);
      constexpr int WB = MODE == kFew ? 1 : 2;
      f32x2 acc[WB][32];                         // 64 columns of each weight block, in pairs
#pragma unroll
      for (int c = 0; c < WB; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c][j] = 0ull;
      // Each block's accumulator, times a * w, onto the sums.  A scheduler has
      // two such warps, so what counts is the length of this chain: few
      // branches, one lane's arrivals as predicated instructions, the next
      // block's scales read ahead, addresses that flip by one xor.
      for (int k0 = kb_lo; k0 < kb_hi; k0 += SCALE_KB, ++g) {
        const uint32_t sbuf = g & 1u;
        warp_wait(&st->sfull[sbuf], (g >> 1) & 1u, lane, abort, p.err, SITE_FP8_EPILOGUE);
        const float* sa = &st->sa[sbuf][0][r];
        constexpr int kRows = 32 * C::QUADS;
        const float2* sw = st->sw[sbuf];
        const int nk = min(SCALE_KB, kb_hi - k0);
        float a = sa[0];
        float2 w = sw[0];
#pragma unroll 1
        for (int k = 0; k < nk; ++k) {
          if (__any_sync(0xffffffffu, !mbar_try(tfull, par)))
            warp_wait(&st->tfull[half][(src >> 7) & 1u], par, lane, abort, p.err, SITE_FP8_EPILOGUE);
          tc_fence_after();
          uint32_t v0[32], v1[32];
          if (live) {
            tmem_ld32(src, v0);
            tmem_ld32(src + 32, v1);
          }
          const f32x2 s0 = both(a * (MODE == kFew && sub ? w.y : w.x)), s1 = both(a * w.y);
          const int kn = min(k + 1, SCALE_KB - 1);
          a = sa[kn * kRows];
          w = sw[kn];
          if (live) {
            tmem_ld_wait();
            if constexpr (MODE != kFew) {
#pragma unroll
              for (int j = 0; j < 16; ++j) fma2(acc[0][j], v0[2 * j], v0[2 * j + 1], s0);
              tmem_ld32(src + 64, v0);
#pragma unroll
              for (int j = 0; j < 16; ++j) fma2(acc[0][16 + j], v1[2 * j], v1[2 * j + 1], s0);
              tmem_ld32(src + 96, v1);
              tmem_ld_wait();
            }
          }
          // all of it is in registers, of every lane: the buffer is free
          tc_fence_before();
          arrive_if<PAIR>(lane == 0, tempty);
          par ^= (src >> 7) & 1u;                // after the second buffer
          src ^= BH;
          tfull ^= 8u;
          tempty ^= 8u;
          if (live) {
            const f32x2 s = MODE == kFew ? s0 : s1;
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(acc[WB - 1][j], v0[2 * j], v0[2 * j + 1], s);
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(acc[WB - 1][16 + j], v1[2 * j], v1[2 * j + 1], s);
          }
        }
        __syncwarp();
        arrive_if<false>(lane == 0, smem_u32(&st->sempty[sbuf]));
      }

      if constexpr (MODE == kFew) {
        // The sums go through shared memory, from where all epilogue warps
        // finish them, a warp per row: on this warp alone, 64 lots of silu and
        // a row of stores took 4 us a tile.
        if (n > 0) warp_wait(&st->xempty, (n - 1) & 1u, lane, abort, p.err, SITE_FP8_EPILOGUE);
        float* dst = &st->part[r][sub * 128 + half * 64];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 x = unpack(acc[0][2 * j]), y = unpack(acc[0][2 * j + 1]);
          *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(x.x, x.y, y.x, y.y);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->xfull[0]);
        if (split == 1) few_rows(tl, n);
        continue;
      }
      uint8_t* stg = st->stage[warp - EPI_WARP0];
      const int row_in = quad * 32 + static_cast<int>(rank) * BM;      // this warp's first row in the tile
      const int nrows = tl.rows - row_in;                              // (may be none, or more than 32)
      if constexpr (MODE != kFew && EPI == kSiluQuant) {
        // columns [half * 64, half * 64 + 64) of the tile's 128
        const int parity = n & 1;
        const int col0 = tl.n_blk * 128 + half * 64;
        float m = 0.f;
        if (live) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {          // n_out is a multiple of 16
            if (col0 + 16 * c < p.n_out) {
#pragma unroll
              for (int j = 8 * c; j < 8 * c + 8; ++j) {
                const float2 gt = unpack(acc[0][j]), up = unpack(acc[1][j]);
                const float2 h = make_float2(silu_bf16_epilogue(gt.x) * up.x, silu_bf16_epilogue(gt.y) * up.y);
                acc[0][j] = pack(h);
                m = fmaxf(m, fmaxf(fabsf(h.x), fabsf(h.y)));
              }
            } else {
#pragma unroll
              for (int j = 8 * c; j < 8 * c + 8; ++j) acc[0][j] = 0ull;
            }
          }
        }
        st->amax[parity][half][r] = m;
        // meet the other half's warps
        __syncwarp();
        if (lane == 0) mbar_arrive(&st->xfull[parity]);
        warp_wait(&st->xfull[parity], (n >> 1) & 1u, lane, abort, p.err, SITE_FP8_EPILOGUE);
        if (live) {
          m = fmaxf(st->amax[parity][0][r], st->amax[parity][1][r]);
          const float s = fp8_scale(m);
          const Fp8Divisor over(m, s);
          uint4 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 f = unpack(acc[0][8 * c + 2 * q]), g2 = unpack(acc[0][8 * c + 2 * q + 1]);
              x[q] = fp8_pack4(over(f.x), over(f.y), over(g2.x), over(g2.y));
            }
            w[c] = make_uint4(x[0], x[1], x[2], x[3]);
          }
          store_rows(stg, lane, w, static_cast<uint8_t*>(p.out) + static_cast<size_t>(tl.row0 + row_in) * p.n_out,
                     p.n_out, col0, nrows);
          if (half == 0 && rvalid)
            p.out_scales[static_cast<size_t>(grow) * ((p.n_out + 127) / 128) + tl.n_blk] = s;
        }
      } else if (MODE != kFew && live) {
        constexpr int kBytes = EPI == kOutF32 ? 4 : 2;
        uint8_t* out = static_cast<uint8_t*>(p.out) + static_cast<size_t>(tl.row0 + row_in) * p.n_out * kBytes;
#pragma unroll
        for (int c = 0; c < WB; ++c) {
          float s = 1.f;
          if constexpr (EPI == kOutF16) {        // 64 columns in this thread: a block
            const int col = tl.n_blk * 256 + c * 128 + half * 64;
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float2 f = unpack(acc[c][j]);
              if (col + 2 * j < p.n_out) m = fmaxf(m, fmaxf(finite_abs(f.x), finite_abs(f.y)));
            }
            s = f16_scale(m);
            if (rvalid && col < p.n_out)
              p.out_scales[static_cast<size_t>(grow) * ((p.n_out + 63) / 64) + col / 64] = 1.f / s;
          }
#pragma unroll
          for (int k = 0; k < kBytes; ++k) {     // 64 bytes of a row at a time
            const int col = tl.n_blk * 256 + c * 128 + half * 64 + k * (64 / kBytes);
            if (col >= p.n_out) continue;        // n_out is a multiple of 8: whole 16 bytes
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const f32x2* a = acc[c] + k * (32 / kBytes) + u * (8 / kBytes);
              uint32_t x[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if constexpr (EPI == kOutF16) {
                  const float2 f = unpack(a[q]);
                  x[q] = pack_f16x2(f.x * s, f.y * s);
                } else if constexpr (EPI == kOutBf16) {
                  const float2 f = unpack(a[q]);
                  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
                  x[q] = *reinterpret_cast<const uint32_t*>(&b);
                } else {
                  const float2 f = unpack(a[q / 2]);
                  x[q] = __float_as_uint(q & 1 ? f.y : f.x);
                }
              }
              w[u] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            store_rows(stg, lane, w, out, static_cast<size_t>(p.n_out) * kBytes,
                       static_cast<size_t>(col) * kBytes, nrows);
          }
        }
      }
      __syncwarp();
    }
  }

  if constexpr (MODE == kFew) {
    if (split > 1) {
      // Every CTA of the cluster adds the shares of some of the rows, in rank
      // order, and finishes them: a warp per row, a lane four columns of each
      // weight block.
      cluster_sync_all();
      if (warp >= EPI_WARP0 && worker < total) {
        const Tile tl = tile_of(worker);
        const int rows = min(C::TILE_M, tl.rows);
        for (int r = share + (warp - EPI_WARP0) * split; r < rows; r += EPI_WARPS * split) {
          float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
          const uint32_t at = smem_u32(&st->part[r][4 * lane]);
          for (int q = 0; q < split; ++q) {
            const float4 x = ld_cluster(at, q), y = ld_cluster(at + 512, q);
            s0.x += x.x; s0.y += x.y; s0.z += x.z; s0.w += x.w;
            s1.x += y.x; s1.y += y.y; s1.z += y.z; s1.w += y.w;
          }
          finish_row<EPI>(p, tl, r, lane, s0, s1);
        }
      }
      cluster_sync_all();                      // no CTA leaves while its share may be read
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();      // neither CTA frees TMEM while its peer may still use it
  if (warp == 1) {
    tc_fence_after();
    tmem_free<PAIR>(tmem);
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

// Clusters of `size` CTAs (1: single CTAs) that the device runs at once; sets
// the kernel's shared-memory opt-in on the way.  A cluster stays within a GPC,
// so of 8 CTAs some 15 fit on 148 SMs.  Asked once per device, kernel and size.
template <int EPI, int MODE>
cudaError_t resident_clusters(int size, int* out) {
  static std::mutex mu;
  static int known[64][9] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev][size] == 0) {
    constexpr int bytes = static_cast<int>(smem_bytes<MODE>());
    err = cudaFuncSetAttribute(gemm_fp8_kernel<EPI, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    int n = num_sms() / size;
    if (size > 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(n * size);
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = bytes;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = size;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int fit = 0;
      if (cudaOccupancyMaxActiveClusters(&fit, gemm_fp8_kernel<EPI, MODE>, &cfg) == cudaSuccess && fit > 0)
        n = fit < n ? fit : n;
      else
        cudaGetLastError();            // the query is advisory
    }
    known[dev][size] = n;
  }
  *out = known[dev][size];
  return cudaSuccess;
}

// The most tiles that M rows of E experts can make, whatever the offsets.
long long tile_bound(long long M, int E, int tile_m, long long n_tiles) {
  const long long touched = M < E ? M : E;
  if (E == 1) return (M + tile_m - 1) / tile_m * n_tiles;
  return (M <= tile_m ? touched : M / tile_m + touched) * n_tiles;
}

template <int EPI, int MODE>
cudaError_t launch_epi(const AMaps& a, const CUtensorMap& b, Params p, cudaStream_t s) {
  int workers = 0;
  cudaError_t err = resident_clusters<EPI, MODE>(MODE == kPair ? 2 : 1, &workers);
  if (err != cudaSuccess) return err;
  const int bn_out = EPI == kSiluQuant ? 128 : 256;
  const long long n_tiles = (p.n_out + bn_out - 1) / bn_out;
  constexpr int tile_m = Cfg<MODE>::TILE_M;
  const long long bound = tile_bound(p.M, p.E, tile_m, n_tiles);
  if (MODE == kPair) {
    const int pairs = static_cast<int>(bound < workers ? bound : workers);
    return launch_k(gemm_fp8_kernel<EPI, MODE>, dim3(2 * pairs), dim3(THREADS), smem_bytes<MODE>(), s, false,
                    2, a, b, p);
  }
  // At most half as many tiles as SMs: a cluster shares each one's blocks, of
  // the largest size of which all run at once and every CTA keeps four.
  p.split = 1;
  if (MODE == kFew && bound * 2 <= workers)
    for (int size = 8; size > 1 && p.split == 1; --size) {
      int fit = 0;
      if (bound * size > workers || p.num_kb < 4 * size) continue;
      if ((err = resident_clusters<EPI, MODE>(size, &fit)) != cudaSuccess) return err;
      if (bound <= fit) p.split = size;
    }
  if (p.split > 1)
    return launch_k(gemm_fp8_kernel<EPI, MODE>, dim3(static_cast<unsigned>(bound * p.split)), dim3(THREADS),
                    smem_bytes<MODE>(), s, false, p.split, a, b, p);
  const int grid = static_cast<int>(bound < workers ? bound : workers);
  return launch_k(gemm_fp8_kernel<EPI, MODE>, dim3(grid), dim3(THREADS), smem_bytes<MODE>(), s, false, 1, a,
                  b, p);
}

template <int MODE>
cudaError_t launch_mode(const GemmFp8Args& g, const AMaps& a, const CUtensorMap& b, const Params& p,
                        cudaStream_t s) {
  if (g.q_scales) return launch_epi<kSiluQuant, MODE>(a, b, p, s);
  if (g.f16_scales) return launch_epi<kOutF16, MODE>(a, b, p, s);
  if (g.out_f32) return launch_epi<kOutF32, MODE>(a, b, p, s);
  return launch_epi<kOutBf16, MODE>(a, b, p, s);
}

}  // namespace

bool gemm_fp8_sorts(int64_t slots, bool gather) { return gather && slots <= THREADS; }

cudaError_t launch_gemm_fp8(const GemmFp8Args& g, cudaStream_t s) {
  const bool gated = g.q_scales != nullptr;
  Params p{};
  p.offsets = g.offsets;
  p.perm = g.perm;
  p.slots = g.slots;
  p.selected = g.selected;
  p.offsets_out = g.offsets_out;
  p.pos_out = g.pos_out;
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
  p.out_scales = gated ? g.q_scales : g.f16_scales;
  p.err = g.err;
  // By the rows of an expert on average.  Us a product, 32 rows | one CTA | pair:
  // 16 experts of 2048 x 2048, 24 rows each: 19 | 19 | 27, 32 rows: 23 | 20 | 27,
  // 512 rows: 138 | 57 | 58; 64 experts of 2816 x 2048, 512 rows each: one CTA
  // 244, pair 257 (half a pair tile of padding per expert); 8192 rows of 4096 x
  // 14336: one CTA 470, pair 435.  Where even tiles of 32 rows leave half the
  // SMs idle, that form shares each one out: 64 rows of 4096 x 4096: 14 | 21 | 21,
  // 128 rows: 19 | 22 | 22, 2000 rows of 256 x 7168: 19 | 31 | 32.  The offsets
  // are device data, so experts that differ cannot be told from even ones; 64
  // experts of 1408 x 2048, 1500 rows, even: 36 | 39 | 57, 1400 of them one
  // expert's: 48 | 40 | 56; 60000 rows, 40000 of them one expert's: 624 | 254 | 256.
  const long long few_tiles = tile_bound(g.M, g.E, Cfg<kFew>::TILE_M, gated ? blocks : (g.N + 255) / 256);
  int mode = g.M >= 768LL * g.E ? kPair : kOne;
  if (g.M <= 24LL * g.E || few_tiles * 2 <= num_sms()) mode = kFew;
  if (g.gather) mode = kFew;                     // the only form that fetches rows by token
  AMaps ma;
  CUtensorMap mb;
  for (int i = 0; i < kBoxes; ++i)
    if (!make_map(&ma.m[i], g.a, static_cast<uint64_t>(g.a_rows), static_cast<uint64_t>(g.K),
                  g.gather ? 1u : 8u << i))
      return cudaErrorInvalidValue;
  if (!make_map(&mb, g.w, static_cast<uint64_t>(g.E) * p.w_rows, static_cast<uint64_t>(g.K),
                mode == kPair ? 128u : 64u))
    return cudaErrorInvalidValue;
  if (mode == kPair) return launch_mode<kPair>(g, ma, mb, p, s);
  if (mode == kFew) return launch_mode<kFew>(g, ma, mb, p, s);
  return launch_mode<kOne>(g, ma, mb, p, s);
}

}  // namespace moe
