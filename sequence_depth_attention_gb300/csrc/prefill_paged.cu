// MoDA attention of a chunk of new tokens per sequence over the paged KV cache:
// the tokens of a batch (pieces of prompts, drafts to verify) attend, under one
// softmax, to the rows of their sequence's pages up to their own and to the L depth
// slots of their own position.
//
// A tile is the G heads of one KV head x 2 P positions of one sequence, in two halves
// of 128 rows. Both halves see (nearly) the same keys, so a block of 128 keys is
// brought into shared memory once for both: S = Q K^T and O += P V on tcgen05, the halves
// in turn, so that the softmax of one half runs beside the products of the other. A
// softmax thread has one row, or (bf16 pages, d = 64) the keys of half a block for one row,
// with an O of its own: the two threads of a row go their own ways (reference, sum, O) until
// the end of a tile, where their states are merged. The work is cut into equal shares of a line of blocks
// (prefill_paged.cuh), so a draft of five tokens over a long context is spread over
// the SMs like a long prompt, and the lengths stay on the device.
//   * A block of 128 keys is up to 8 pages, each looked up and copied by a lane.
//   * Depth slots are gathered by TMA, a block of each half's own positions, under a
//     block-diagonal mask (a softmax warp has a 32-row word of it), and spread evenly
//     among the sequence blocks.
//   * 4-bit pages are unpacked into the bf16 tiles that the tensor core reads (exactly: a
//     code times a power of two), once for both halves; V in units of 2^26 (kUnitLog).
//   * A row that a query must not see does not count whatever it holds. Its weight is
//     0, but 0 times an infinity or a NaN in V is NaN: in the blocks that some row of a
//     tile sees in part (the causal border, the depth blocks), rows that no query of the
//     tile sees become 0, and an infinity or NaN among the others becomes 0 too and is
//     added at the end to the rows that do see it.
//
// Roles (16 warps; 20 for 4-bit pages; 24 with two softmax threads a row):
//   warp 0        TMA producer of Q and K     warp 1  issuer of all MMAs, TMEM
//   warp 2        TMA producer of V           warp 3  4-bit pages: of the depth blocks
//   warps 4-7     softmax and epilogue of the first half, one thread per row (TMEM lane)
//   warps 8-11    of the second half (two threads a row: 4-11 of the first, 12-19)
//   the last 4    partly seen V blocks made harmless
//         (8)     and 4-bit pages unpacked, by way of registers
// TMEM (512 columns): S of the halves [0,128) [128,256), each half's P (bf16 pairs) in the
// first 64 columns of its S, O of the halves at 256 and 256 + d. (Two threads a row: each P in
// the first 32 of its thread's 64 columns of S, O of the threads 64 columns each from 256 on.)
// P is rounded to bf16 once, as in the forward: the sum l keeps fp32 weights, and
// what o is off by that is about as much as its own rounding to bf16 (0.0023 of the norm in all
// against 0.0017 with exact weights). Two bf16 parts, which the decode takes, would make the
// products 3/2 of what they are: 841 us and not 561 in the first case below.
//
// What bounds it, measured (us; the floor is that of the products or of the rows):
//   d = 128, 2048 tokens at 65536 rows, G = 4    735 to 810 (561)   tensor pipe 73 % of cycles, then
//            the clock. What the pipe is not busy is the halves' hand-over of S and P.
//   d = 64, 7 prompts' pieces, G = 8            1350 (577)   no unit is full (tensor pipe 41 %,
//            exponentials 37 %, issue 58 %): the softmax warps wait for TMEM and barriers, 4.1 of an
//            instruction's 10.3 cycles, and TMEM has no room for another tile meanwhile. Where this
//            took 1330, one thread a row took 1410, S ahead in columns of its own 1418 to 1530.
//   4-bit, 1024 tokens at 32768, G = 4           285 (140)   issue 60 %: each CTA unpacks all of its
//            tiles' blocks, beside the softmax. d = 64, G = 8: 772 (281), bf16 562.
//   32 drafts of up to 8 tokens, to 16000 rows    97 (80)    HBM: 82 % of the copy rate. d = 64, G = 8
//            136 (80): 1.45 us a block for half the bytes.
//   the same over 4-bit rows                     150 (22), d = 64 195 (22): a block's unpacking and its
//            softmax one behind the other, 1.9 us; to 32768 rows 278 (44) and 369 (44).
//   5 tokens at 701 rows                          14 (0.3)   latencies one behind another: share
//            2, first rows 3, blocks 4, the join behind the last CTA 3.
// The softmax takes 32 scores at a time. At d = 64 with two threads a row (all before the halves had
// flags of their own, which cost 0.5 %) 1330; 16 at a time 1478, 16 with the next on their way 1467, 64
// 1563, 32 with 160 spilled bytes 1632 (some 50 are). At d = 128: 1024 tokens without a past 40.9, 128
// tokens at 2000 27.9, 2048 at 65536 720 to 770; 128 at a time 42.4, 28.8 and 705 to 764. Over 4-bit
// pages 16 at a time 3 % slower, 64 5 %.
//
// Every wait is bounded (2 s); on expiry the CTA stops issuing work, waits for its
// copies and MMAs in flight, frees TMEM and latches MODA_ERR_TIMEOUT.
#include "mx4.cuh"
#include "prefill_paged.cuh"
#include "softmax_block.cuh"
#include "tensor_map.h"

namespace moda {
namespace prefill {
namespace {

using namespace mx4;
using namespace sm103;
using paged::kLn2;
using paged::kLog2e;

constexpr int BM = 128, BN = 128;  // rows of a half tile, keys of a block
constexpr uint64_t kTimeoutNs = 2000000000ull;
// 4-bit pages: O is held in units of 2^26, V's values unpacked in these and the depth blocks' P
// times 2^-26. Values are up to 1.5 * 2^127, a block's weights add up to kSumBound at most, and 2^24
// rows are 2^17 blocks: their sums stay finite. (Powers of two: no other bit changes. bf16 pages'
// values are what the tensor core reads; their sums have fp32's range.)
constexpr int kUnitLog = 26;
constexpr float kSumBound = 256.0f;  // of a row's weights in a block, see the softmax warps
// Points that are worth a CTA. Measured (us) with 1, 2, 3, 4, 6: 5 tokens at 701 rows 14.4,
// 15.1, 15.2, 17.2, 18.9; 128 tokens at 2000 31.6, 27.9, 27.5, 28.4, 31.7; where there is more
// work than that, no difference.
constexpr int kLeast = 2;

template <int D, bool MX4>
struct Cfg {
  static constexpr int kTameWarps = MX4 ? 8 : 4;
  // Threads of a row. (Two take more registers than 4-bit pages leave, and at d = 128 more TMEM
  // than there is.)
  static constexpr int kCh = D == 64 && !MX4 ? 2 : 1;
  static constexpr int kTame0 = 4 + 8 * kCh, kWarps = kTame0 + kTameWarps, kThreads = kWarps * 32;
  // Registers of a thread of each group of four warps; they add up to no more than the block
  // is launched with (kRegsLaunch a thread).
  static constexpr int kRegsIssue = kCh == 2 || MX4 ? 64 : 96, kRegsSoftmax = kCh == 2 ? 88 : MX4 ? 120 : 152;
  static constexpr int kRegsTame = kCh == 2 ? 64 : MX4 ? 88 : 104, kRegsLaunch = kCh == 2 ? 80 : MX4 ? 96 : 128;
  static_assert(kRegsIssue + 2 * kCh * kRegsSoftmax + kTameWarps / 4 * kRegsTame <= kWarps / 4 * kRegsLaunch);
  static constexpr int kBoxes = D / 64;  // 64-column (128-byte) swizzle boxes per row
  static constexpr int kBoxBytes = BN * 128;
  static constexpr int kQBytes = BM * D * 2;  // of a half
  static constexpr int kTileBytes = BN * D * 2;
  static constexpr int kNK = D == 128 ? 2 : 4, kNV = D == 128 ? 3 : 5;  // stages of K and of V
  static constexpr int kOffK = 2 * kQBytes;
  static constexpr int kOffV = kOffK + kNK * kTileBytes;
  static constexpr int kOffBar = kOffV + kNV * kTileBytes;
  static constexpr int kOffMl = kOffBar + (kCh == 2 ? 4096 : 2048);  // m and l of a row's threads
  static constexpr int kSmemBytes = kOffMl + (kCh == 2 ? 4 * BM * 8 : 0) + 1024;  // alignment
  static constexpr uint32_t kColS = 0, kColO = 256;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

constexpr int kMaxStages = 5;

template <int WALKS>
struct alignas(16) Barriers {
  uint64_t q_full, q_free;  // Q of the current tile landed / its last S = Q K^T completed
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  // bf16 pages: a partly seen V block lands at v_check and not at v_full, and is v_ready
  // once it has been made harmless. (A barrier of its own, whose phases the warps that
  // do it wait for one by one: they skip the other blocks.) 4-bit pages: a depth block
  // lands at k_check and v_check, and is full once the unpacking warps have seen it.
  uint64_t k_check[kMaxStages], v_check[kMaxStages], v_ready[kMaxStages];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t ml_full[8];  // two threads a row: a pair of warps have left their m and l
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
  // Had a tile infinities or NaN taken out? [half][n % 8] = k (16 bits) for the n-th of the tiles that
  // the half has rows of, the k-th of all. (Its next tile's V stages are freed behind its P alone, so
  // that the warps which say so are never more than the stages ahead of it. With places counted over
  // all tiles, a run of tiles of one half could pass the second half by, and take the place of an
  // answer that it had not read.)
  int poison[2][8];
  uint32_t some[24];  // see Share
  Share share;
  union {
    ShareSmem find;    // before the roles begin
    Walk walk[WALKS];  // of warps 4 on, whose registers are full
  };
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait_bounded(bar, parity, abort, kTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}
// One arrival for the warp, behind what its lanes have done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(bar));
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 or 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st16(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) { tmem_st32(taddr, r); }

// Waits for tcgen05.ld and ties the registers to it: nothing that reads them moves up.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
#define MODA_RW8(i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), \
                    "+r"(r[i + 6]), "+r"(r[i + 7])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : MODA_RW8(0), MODA_RW8(8), MODA_RW8(16), MODA_RW8(24)::"memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : MODA_RW8(0), MODA_RW8(8)::"memory");
}
#undef MODA_RW8

// A warp's walk in shared memory on to its next tile; the warp has read what it wants of
// the one before.
__device__ __forceinline__ bool warp_next(Walk& w, const Params& p, const Share& sh, int lane, bool first) {
  bool any = false;
  __syncwarp();
  if (lane == 0) {
    if (first) w.begin(p, sh);
    any = w.next(p, sh);
  }
  any = __shfl_sync(0xffffffffu, any, 0);
  __syncwarp();  // what lane 0 has written is seen
  return any;
}

// Is block (depth, index) of the walk's tile one that some row sees in part?
__device__ __forceinline__ bool partly_seen(const Walk& w, const Sched& sch) {
  return sch.depth || sch.index * BN + BN - 1 > w.t0;
}

// Row r of a V tile in shared memory: zeros where it does not count, and zeros in
// place of infinities and NaN; true if there were any.
template <int D>
__device__ __forceinline__ bool tame_row(uint8_t* tile, int r, bool counts) {
  constexpr int kBoxBytes = BN * 128;
  uint32_t bad = 0;
#pragma unroll 1
  for (int c = 0; c < D / 64; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint4* at = reinterpret_cast<uint4*>(tile + c * kBoxBytes + r * 128 + ((i ^ (r & 7)) << 4));
      if (!counts) {
        *at = make_uint4(0u, 0u, 0u, 0u);
      } else {
        const uint4 x = *at;
        bad |= not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w);
      }
    }
  if (!bad) return false;
  uint32_t* row = reinterpret_cast<uint32_t*>(tile + r * 128);
#pragma unroll 1
  for (int i = 0; i < D / 2; ++i) {
    uint32_t& x = row[(i >> 5) * (kBoxBytes / 4) + (i & 31)];  // the swizzle moves 16-byte chunks within the row
    const uint32_t f = not_finite(x);
    x &= ~(((f & 0x8000u) ? 0xffffu : 0u) | ((f & 0x80000000u) ? 0xffff0000u : 0u));
  }
  return true;
}

// A lane's 4-bit blocks of a tile, from global memory by way of registers to bf16: D / 32
// lanes a row, a block of 32 elements a lane, four warps. The next tile's are on their way
// while this one's are unpacked. One loop for K and V, all turns and both halves of a block:
// beside the softmax's code, unrolled ones waited for their instructions (1.7 of a scheduler's
// 5 warps did). 1024 tokens at 32768 285 us; the halves unrolled 294, two turns as well 301,
// a chunk at a time 341.
template <int D>
struct Codes {
  static constexpr int BPR = D / 32;        // blocks, and lanes, of a row
  static constexpr int RPT = 4 * 32 / BPR;  // rows the warps take at once
  static constexpr int kTurns = BN / RPT;
  uint4 codes[kTurns];
  uint32_t scale[kTurns];  // bytes
  static __device__ __forceinline__ int row(int turn, int hw, int lane) {
    return turn * RPT + hw * (32 / BPR) + lane / BPR;
  }
  // Into a bf16 tile, zeros from row `rows` on; `tame`: and in place of infinities and NaN.
  // True if there were any. (Of NaN: in units no finite code is infinite.) unit: see scale_in_units.
  __device__ __forceinline__ bool unpack(uint32_t tile, int hw, int lane, int rows, bool tame, int unit) {
    const int qtr = lane % BPR;
    // A block is four 16-byte chunks of a 64-column box from 4 (qtr & 1) on; lanes of the
    // upper box take them in another order, so that eight lanes (two rows) meet different
    // banks.
    const bool upper = qtr >> 1;
    uint32_t found = 0;
#pragma unroll 1
    for (int t = 0; t < kTurns; ++t) {
      const int r = row(t, hw, lane);
      const uint32_t to = tile + (upper ? BN * 128 : 0) + r * 128;
      const uint32_t s = r < rows ? scale_in_units(scale[0], unit) : 0u;
#pragma unroll 1
      for (int j = 0; j < 4; j += 2) {
        uint32_t y[2][4];
        unpack8(upper == (j == 0) ? codes[0].z : codes[0].x, s, y[0]);
        unpack8(upper == (j == 0) ? codes[0].w : codes[0].y, s, y[1]);
        if (tame && scale[0] == 255u) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t f = not_finite(y[i >> 2][i & 3]);
            found |= f;
            y[i >> 2][i & 3] &= ~(((f & 0x8000u) ? 0xffffu : 0u) | ((f & 0x80000000u) ? 0xffff0000u : 0u));
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int chunk = 4 * (qtr & 1) + (upper ? (j ^ 2) + i : j + i);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((chunk ^ (r & 7)) << 4)), "r"(y[i][0]),
                       "r"(y[i][1]), "r"(y[i][2]), "r"(y[i][3])
                       : "memory");
        }
      }
#pragma unroll
      for (int i = 0; i + 1 < kTurns; ++i) {
        codes[i] = codes[i + 1];
        scale[i] = scale[i + 1];
      }
    }
    return found != 0;
  }
};

// p = 2^(s sl - m) of 32 scores as bf16 pairs, added up in acc.
__device__ __forceinline__ void weigh(const uint32_t* x, uint32_t* pk, float sl, float m, uint64_t (&acc)[4]) {
  const uint64_t sl2 = f2(sl, sl), nb2 = f2(-m, -m);
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    float u, w;
    f2_split(ffma2(f2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sl2, nb2), u, w);
    const float e0 = ex2_approx(u), e1 = ex2_approx(w);
    pk[c] = pack_bf16x2(e0, e1);
    acc[c & 3] = fadd2(acc[c & 3], f2(e0, e1));
  }
}
__device__ __forceinline__ float total_of(uint64_t (&acc)[4]) {
  float u, w;
  f2_split(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), u, w);
  return u + w;
}

template <int D, bool MX4>
__global__ void __launch_bounds__(Cfg<D, MX4>::kThreads, 1)
prefill_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKd,
                     const __grid_constant__ CUtensorMap tmVd, const __grid_constant__ Params p) {
  using C = Cfg<D, MX4>;
  constexpr int NK = C::kNK, NV = C::kNV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  using Bars = Barriers<C::kWarps - 4>;
  static_assert(sizeof(Bars) <= C::kOffMl - C::kOffBar, "barrier block");
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  const uint32_t sQ = smem_u32(smem), sK = smem_u32(smem + C::kOffK), sV = smem_u32(smem + C::kOffV);
  volatile int* abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = BM >> p.lgG;           // positions of a half
  const int PW = P >> 2, SP = 32 / PW;  // positions and slots of a softmax warp's word of a depth block

  if (tid == 0) {
    bars->abort = 0;
    for (int i = 0; i < 16; ++i) bars->poison[i >> 3][i & 7] = 0;
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_free), 1);
    for (int s = 0; s < kMaxStages; ++s) {
      // 4-bit pages: the unpacking warps, and warp 3, which sees every stage free
      mbar_init(smem_u32(&bars->k_full[s]), MX4 ? 5 : 1);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
      mbar_init(smem_u32(&bars->v_full[s]), MX4 ? 5 : 1);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
      mbar_init(smem_u32(&bars->k_check[s]), 1);
      mbar_init(smem_u32(&bars->v_check[s]), 1);
      mbar_init(smem_u32(&bars->v_ready[s]), 4);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&bars->s_full[x]), 1);
      mbar_init(smem_u32(&bars->p_full[x]), 4 * C::kCh);
      mbar_init(smem_u32(&bars->o_done[x]), 1);
    }
    for (uint64_t& x : bars->ml_full) mbar_init(smem_u32(&x), 2);
    mbar_init(smem_u32(&bars->mma_done), 1);
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmKd);
    tma_prefetch_desc(&tmVd);
    if (!MX4) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  paged::wait_for_stream();
  {
    const Share mine = share_of<C::kWarps, kLeast>(p, bars->find, bars->some);
    if (mine.from >= mine.to) {
      if (tid == 0) work_of(p.work, D).opened[blockIdx.x] = {0, 0, 0, 0};
      return;
    }
    if (tid == 0) bars->share = mine;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  const Share& sh = bars->share;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsIssue));
    if (warp == 0 || warp == 2) {
      // ------------------- TMA producers (4-bit pages: of Q alone)
      const bool is_k = warp == 0;
      const bool leader = elect_one();
      const uint64_t pol_once = l2_policy_evict_first();
      const int ns = is_k ? NK : NV;  // stages
      uint64_t* full = is_k ? bars->k_full : bars->v_full;
      uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
      const int page_rows = 1 << p.page_shift;  // at most 128
      // a lane copies 64 columns of one page's rows
      const int my_box = lane / C::kBoxes, my_part = lane % C::kBoxes;
      int e = 0, f = 0, fph = 0, nq = 0;  // entries; the next one's stage and phase; Q loads
      uint32_t checks = 0, wholes = 0;  // of V's stages: parities of what went to v_check, to v_full
      uint32_t any_check = 0, any_whole = 0;
      Walk w;
      w.begin(p, sh);
      bool ok = true;
      for (int k = 0; ok && w.next(p, sh); ++k) {
        const int halves = w.npos > P ? 2 : 1;
        if (is_k) {
          // Q, once the last S product of the tile before has completed
          if (k > 0 && !warp_wait(smem_u32(&bars->q_free), (k - 1) & 1, abort)) break;
          if (leader) {
            const uint32_t qb = smem_u32(&bars->q_full);
            mbar_arrive_expect_tx(qb, halves * C::kQBytes);
            for (int x = 0; x < halves; ++x)
              for (int c = 0; c < C::kBoxes; ++c)
                tma_load_3d_hint(sQ + x * C::kQBytes + c * C::kBoxBytes, &tmQ, qb, c * 64, w.hk * p.G,
                                 w.token + x * P, pol_once);
          }
          ++nq;
        }
        if constexpr (!MX4) {
          Sched sch(p.n_depth, w.nb, w.j0);
          const int* table = p.table + (int64_t)w.b * p.max_pages;
          // the lane's page of a sequence block, looked up one block ahead
          auto page_of = [&](int index) -> int {
            const int key = index * BN + (my_box << p.page_shift);
            return my_box << p.page_shift < BN && key <= w.t_last ? table[key >> p.page_shift] : -1;
          };
          int page = page_of(sch.sbk);
          for (int j = w.j0; ok && j < w.j1; ++j) {
            sch.next(p.n_depth, w.nb);
            int pg = page;
            if (!sch.depth) page = page_of(sch.index + 1);
            // a depth block of each half, or a sequence block for both
            for (int x = 0; x < (sch.depth ? halves : 1); ++x) {
              if (!warp_wait(smem_u32(&empty[f]), fph ^ 1, abort)) {
                ok = false;
                break;
              }
              uint32_t fb = smem_u32(&full[f]);
              if (!is_k) {
                if (partly_seen(w, sch)) {
                  fb = smem_u32(&bars->v_check[f]);
                  checks ^= 1u << f;
                  any_check |= 1u << f;
                } else {
                  wholes ^= 1u << f;
                  any_whole |= 1u << f;
                }
              }
              const uint32_t dst = (is_k ? sK : sV) + f * C::kTileBytes;
              if (sch.depth) {
                // the words of the softmax warps that have positions: slots [SP index, + SP)
                // of a warp's PW positions, row slot * PW + position
                if (leader) {
                  const int words = (min(w.npos - x * P, P) + PW - 1) / PW;
                  mbar_arrive_expect_tx(fb, words * 32 * D * 2);
                  for (int y = 0; y < words; ++y)
                    for (int c = 0; c < C::kBoxes; ++c)
                      tma_load_4d_hint(dst + c * C::kBoxBytes + y * 32 * 128, is_k ? &tmKd : &tmVd, fb, c * 64, w.hk,
                                       w.token + x * P + y * PW, sch.index * SP, pol_once);
                }
              } else {
                const int rows = min(BN, w.t_last + 1 - sch.index * BN);
                const int boxes = (rows + page_rows - 1) >> p.page_shift;
                if (leader) mbar_arrive_expect_tx(fb, boxes * page_rows * D * 2);
                __syncwarp();
                if (my_box < boxes) {
                  if (pg < 0 || pg >= p.num_pages) {
                    atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
                    pg = 0;
                  }
                  tma_load_3d(dst + my_part * C::kBoxBytes + my_box * page_rows * 128, is_k ? &tmK : &tmV, fb,
                              my_part * 64, 0, pg * p.Hk + w.hk);
                }
              }
              __syncwarp();
              ++e;
              if (++f == ns) {
                f = 0;
                fph ^= 1;
              }
            }
          }
        } else if (!is_k) {
          break;
        }
      }
      // every copy of this warp has landed before its shared memory is released
      if (leader) {
        int never = 0;
        if (!is_k) {
          for (int s = 0; s < NV; ++s) {
            if (any_whole >> s & 1)
              mbar_wait_bounded(smem_u32(&bars->v_full[s]), (wholes >> s & 1) ^ 1, &never, kTimeoutNs);
            if (any_check >> s & 1)
              mbar_wait_bounded(smem_u32(&bars->v_check[s]), (checks >> s & 1) ^ 1, &never, kTimeoutNs);
          }
        } else {
          for (int j = max(0, e - ns); j < e; ++j)
            mbar_wait_bounded(smem_u32(&full[j % ns]), (j / ns) & 1, &never, kTimeoutNs);
        }
        if (is_k && nq > 0) mbar_wait_bounded(smem_u32(&bars->q_full), (nq - 1) & 1, &never, kTimeoutNs);
      }
      __syncwarp();
    } else if (warp == 3) {
      if constexpr (MX4) {
        // ------------------------- depth blocks beside 4-bit pages, and every stage seen free
        // (a stage's next user waits for this warp too, so that it misses no phase)
        if (elect_one()) {
          const uint64_t pol_once = l2_policy_evict_first();
          uint32_t landed[2] = {0, 0}, any[2] = {0, 0};  // of K, of V: parities and use of k_check, v_check
          int e = 0;
          bool ok = true;
          Walk w;
          w.begin(p, sh);
          while (ok && w.next(p, sh)) {
            const int halves = w.npos > P ? 2 : 1;
            Sched sch(p.n_depth, w.nb, w.j0);
            for (int j = w.j0; ok && j < w.j1; ++j) {
              sch.next(p.n_depth, w.nb);
              for (int x = 0; ok && x < (sch.depth ? halves : 1); ++x, ++e) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                  const int ns = v ? NV : NK, s = e % ns;
                  if (!mbar_wait_bounded(smem_u32(v ? &bars->v_empty[s] : &bars->k_empty[s]), ((e / ns) & 1) ^ 1, abort,
                                         kTimeoutNs)) {
                    ok = false;
                    break;
                  }
                  if (sch.depth) {
                    const uint32_t fb = smem_u32(v ? &bars->v_check[s] : &bars->k_check[s]);
                    const int words = (min(w.npos - x * P, P) + PW - 1) / PW;
                    landed[v] ^= 1u << s;
                    any[v] |= 1u << s;
                    mbar_arrive_expect_tx(fb, words * 32 * D * 2);
                    const uint32_t dst = (v ? sV : sK) + s * C::kTileBytes;
                    for (int y = 0; y < words; ++y)
                      for (int c = 0; c < C::kBoxes; ++c)
                        tma_load_4d_hint(dst + c * C::kBoxBytes + y * 32 * 128, v ? &tmVd : &tmKd, fb, c * 64, w.hk,
                                         w.token + x * P + y * PW, sch.index * SP, pol_once);
                  }
                  mbar_arrive(smem_u32(v ? &bars->v_full[s] : &bars->k_full[s]));
                }
              }
            }
          }
          int never = 0;
          for (int v = 0; v < 2; ++v)
            for (int s = 0; s < (v ? NV : NK); ++s)
              if (any[v] >> s & 1)
                mbar_wait_bounded(smem_u32(v ? &bars->v_check[s] : &bars->k_check[s]), (landed[v] >> s & 1) ^ 1, &never,
                                  kTimeoutNs);
        }
        __syncwarp();
      }
    } else if (elect_one()) {
      // -------------------------------------------------------- MMA issuer
      // One thread issues everything, in the order S of the halves, then for each block
      // and half P V of the block before and S of this one: MMAs complete in order, so a
      // half's S may overwrite the P that the P V before it reads.
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_wait_bounded(smem_u32(bar), parity, abort, kTimeoutNs);
      };
      constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false), idPV = idesc_bf16_f32(BM, D, true);
      const uint64_t dq = sdesc_sw128(sQ, 16, 1024);
      const uint32_t hi = (uint32_t)(dq >> 32), q_lo = (uint32_t)dq;
      const uint32_t k_lo = (uint32_t)sdesc_sw128(sK, 16, 1024), v_lo = (uint32_t)sdesc_sw128(sV, C::kBoxBytes, 1024);
      // entries of K: stage and phase of the next; of V (one block later): the next, and
      // bf16 pages' parities of v_ready and v_full, a bit for each stage
      int ks = 0, kph = 0, vs = 0, vph = 0;
      uint32_t ready = 0, whole = 0, pph = 0;  // pph: parities of p_full
      auto wait_v = [&](bool part) -> bool {
        if (MX4) return wait(&bars->v_full[vs], vph);
        if (part) {
          if (!wait(&bars->v_ready[vs], ready >> vs & 1)) return false;
          ready ^= 1u << vs;
        } else {
          if (!wait(&bars->v_full[vs], whole >> vs & 1)) return false;
          whole ^= 1u << vs;
        }
        return true;
      };
      auto next_v = [&] {
        tc_commit(smem_u32(&bars->v_empty[vs]));
        if (++vs == NV) {
          vs = 0;
          vph ^= 1;
        }
      };
      // P V of half x with the V in stage vs
      auto pv = [&](int x, uint32_t accumulate) {
        const uint32_t vb = v_lo + ((uint32_t)(vs * C::kTileBytes) >> 4);
        constexpr int KC = BN / 16 / C::kCh;  // steps of a chain
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_ts(tbase + C::kColO + (x * C::kCh + kk / KC) * D,
                 tbase + C::kColS + x * 128 + kk / KC * (BN / C::kCh) + kk % KC * 8,
                 desc_join(vb + ((uint32_t)(kk * 2048) >> 4), hi), idPV, kk % KC > 0 ? 1u : accumulate);
      };
      bool ok = true;
      Walk w;
      w.begin(p, sh);
      for (int k = 0; ok && w.next(p, sh); ++k) {
        const int halves = w.npos > P ? 2 : 1;
        if (!wait(&bars->q_full, k & 1)) break;
        Sched sch(p.n_depth, w.nb, w.j0);
        bool depth = false, part = false;  // of the block before
        for (int j = w.j0; ok && j <= w.j1; ++j) {
          const bool was_depth = depth, was_part = part, last = j == w.j1;
          if (!last) {
            sch.next(p.n_depth, w.nb);
            depth = sch.depth;
            part = partly_seen(w, sch);
          }
          for (int x = 0; x < halves; ++x) {
            if (j > w.j0) {
              if (((x == 0 || was_depth) && !wait_v(was_part)) || !wait(&bars->p_full[x], pph >> x & 1)) {
                ok = false;
                break;
              }
              pph ^= 1u << x;
              tc_fence_after();
              // a tile's first P V overwrites O (the softmax warps have read the tile
              // before's O before they stored this P)
              pv(x, j - 1 > w.j0 ? 1u : 0u);
              if (last) tc_commit(smem_u32(&bars->o_done[x]));
              if (x == halves - 1 || was_depth) next_v();
            }
            if (!last) {
              if ((x == 0 || depth) && !wait(&bars->k_full[ks], kph)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t kb = k_lo + ((uint32_t)(ks * C::kTileBytes) >> 4);
              const uint32_t qb = q_lo + ((uint32_t)(x * C::kQBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
                mma_ss(tbase + C::kColS + x * 128, desc_join(qb + off, hi), desc_join(kb + off, hi), idS, kk > 0);
              }
              tc_commit(smem_u32(&bars->s_full[x]));
              if (x == halves - 1 || depth) {
                tc_commit(smem_u32(&bars->k_empty[ks]));
                if (++ks == NK) {
                  ks = 0;
                  kph ^= 1;
                }
              }
              if (j == w.j1 - 1 && x == halves - 1) tc_commit(smem_u32(&bars->q_free));
            }
          }
        }
      }
      // every MMA has completed before TMEM is freed
      int never = 0;
      tc_commit(smem_u32(&bars->mma_done));
      mbar_wait_bounded(smem_u32(&bars->mma_done), 0, &never, kTimeoutNs);
    }
    __syncwarp();
  } else if (warp < C::kTame0) {
    // ----------------------------------------------------- softmax, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    constexpr int CH = C::kCh, W = BN / CH;  // columns of a thread
    constexpr int NE = CH == 2 || MX4 ? 16 : 32;  // of O at a time: spilled registers cost more
    const int half = (warp - 4) / (4 * CH), ch = (warp - 4) / 4 % CH;  // ch: which of a row's threads
    const int row = tid & 127;  // row of the half == TMEM lane
    const uint32_t scol = tmem_addr(tbase, (uint32_t)(warp & 3) * 32, C::kColS + half * 128 + ch * W);
    const uint32_t ocol = tmem_addr(tbase, (uint32_t)(warp & 3) * 32, C::kColO + half * CH * D);
    const int wq = warp & 3;  // this warp's word of a depth block
    const int wl = wq % (4 / CH);  // and where it is among the thread's columns, if it is
    const bool word_here = wq / (4 / CH) == ch;
    const int lp = half * P + (row >> p.lgG), h_off = row & ((1 << p.lgG) - 1);
    const int lpw = (row & 31) >> p.lgG;  // the row's position among its warp's
    const uint32_t own_cols = PW >= 32 ? 1u << lpw : (0xffffffffu / ((1u << PW) - 1u)) << lpw;
    const float sl = p.scale_log2;
    uint32_t sph = 0, oph = 0, mph = 0;  // parities of s_full, o_done, ml_full
    Walk& w = bars->walk[warp - 4];
    auto advance = [&](bool first) -> bool { return warp_next(w, p, sh, lane, first); };
    bool opened = false, ok = true, more = advance(true);
    for (int k = 0; ok && more; ++k, more = advance(false)) {
      if (half && w.npos <= P) continue;
      // rows without a query go along: their scores are the next tokens' (or zeros), and
      // what they hold is not looked at
      const bool there = lp < w.npos && h_off < p.G;
      float m_ref = -INFINITY, l = 0.f;
      // Rescale O and l to a new reference where a block's raw max mx (log2 units) is
      // above it. O holds blocks j0 .. j - 1: their P V has
      // completed, since S of block j, issued behind it, has.
      auto rescale = [&](float mx, int j) {
        const bool need = mx > m_ref;
        if (__any_sync(0xffffffffu, need && there)) {
          const float m_new = need ? mx : m_ref;
          const float alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
          if (j > w.j0) {
#pragma unroll
            for (int c = 0; c < D / NE; ++c) {
              uint32_t r[NE];
              tmem_ld(ocol + ch * D + c * NE, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int i = 0; i < NE; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tmem_st(ocol + ch * D + c * NE, r);
            }
            tmem_st_wait();
          }
          l *= alpha;
          m_ref = m_new;
        }
      };
      // Every block: exponentiate against the running reference right away. Every p is
      // at most the block's sum, so a sum within kSumBound proves that no score rose more
      // than 8 (log2 units) above it, and the block needs no maximum at all. Else the
      // references of the warp's rows become their maxima, and the block is weighed again. (Of the
      // rows that ask for it alone, so that no row's rounding depends on another's: 2048 tokens at
      // 65536 1.2 % slower, 1024 over 4-bit pages 2.4 %, for each raises its own at another block.)
      const int nb = w.nb, j1 = w.j1, border0 = (w.t0 + 1) / BN;  // the first sequence block at the causal border
      bool unset = true;  // some row has no reference yet
      Sched sch(p.n_depth, nb, w.j0);
      for (int j = w.j0; j < j1; ++j) {
        sch.next(p.n_depth, nb);
        if (!warp_wait(smem_u32(&bars->s_full[half]), sph, abort)) {
          ok = false;
          break;
        }
        sph ^= 1;
        tc_fence_after();
        if (unset) unset = __any_sync(0xffffffffu, there && m_ref == -INFINITY);
        bool slow = unset;
        float sum = 0.f;
        if (sch.depth) {
          // only this warp's word of 32 columns can hold its rows' slots: column c is
          // slot index * SP + c / PW of the warp's position c % PW
          const int nbits = min(SP, p.L - sch.index * SP) * PW;
          const uint32_t word = lp < w.npos ? own_cols & (nbits >= 32 ? 0xffffffffu : (1u << nbits) - 1u) : 0u;
          const uint32_t zeros[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
          if (word_here) {
            uint32_t x[32], pk[16];
            tmem_ld32(scol + wl * 32, x);
            tmem_ld_wait(x);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = (word & (1u << i)) ? x[i] : 0xff800000u;  // -inf
            for (int pass = 0; pass < 2; ++pass) {
              if (slow) rescale(raw_max32(x) * sl, j);
              uint64_t acc[4] = {0, 0, 0, 0};
              weigh(x, pk, sl, m_ref == -INFINITY ? 0.f : m_ref, acc);
              sum = total_of(acc);
              if (slow) break;
              slow = __any_sync(0xffffffffu, there && !(sum <= kSumBound));
              if (!slow) break;
            }
            if constexpr (MX4) {
              constexpr uint32_t kInUnits = (127u - kUnitLog) << 7 | (127u - kUnitLog) << 23;
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = mul_bf16x2(pk[i], kInUnits);
            }
            tmem_st16(scol + wl * 16, pk);
          } else {
            tmem_st16(scol + wl * 16, zeros);
          }
          for (int kk = 1; kk < 4 / CH; ++kk) tmem_st16(scol + (wl + kk) % (4 / CH) * 16, zeros);
        } else {
          // columns that the row sees: all, but at the causal border
          const bool border = sch.index >= border0;
          const int end = border ? min(w.t0 + lp, w.t_last) - sch.index * BN + 1 - ch * W : W;
          {
            uint32_t pk[W / 2];
            for (int pass = 0; pass < 2; ++pass) {
              if (slow) {
                float mx = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < W / 32; ++c) {
                  uint32_t y[32];
                  tmem_ld32(scol + c * 32, y);
                  tmem_ld_wait(y);
#pragma unroll
                  for (int i = 0; i < 32; ++i) y[i] = c * 32 + i < end ? y[i] : 0xff800000u;  // -inf
                  mx = fmaxf(mx, raw_max32(y));
                }
                rescale(mx * sl, j);
              }
              const float m = m_ref == -INFINITY ? 0.f : m_ref;
              uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
              for (int c0 = 0; c0 < W; c0 += 32) {
                uint32_t x[32];
                tmem_ld32(scol + c0, x);
                tmem_ld_wait(x);
                if (border) {
#pragma unroll
                  for (int c = 0; c < 32; ++c) x[c] = c0 + c < end ? x[c] : 0xff800000u;  // -inf
                }
                weigh(x, pk + c0 / 2, sl, m, acc);
              }
              sum = total_of(acc);
              if (slow) break;
              slow = __any_sync(0xffffffffu, there && !(sum <= kSumBound));
              if (!slow) break;
            }
            tmem_st32(scol, pk);
            if constexpr (CH == 1) tmem_st32(scol + 32, pk + 32);
          }
        }
        l += sum;
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&bars->p_full[half], lane);
      }
      if (!ok) break;
      const bool cut = w.cut();
      if (cut && w.j0 == 0 && tid == 128)  // the tile's first block is here: the join begins at this CTA
        work_of(p.work, D).opened[blockIdx.x] = {w.token, w.hk, w.npos,
                                                 sh.owner_of(w.next_at - 1) - (int)blockIdx.x + 1};
      opened |= cut && w.j0 == 0;
      if (!warp_wait(smem_u32(&bars->o_done[half]), oph, abort)) {
        ok = false;
        break;
      }
      oph ^= 1;
      tc_fence_after();
      float own = 1.f, other = 0.f;  // what the O of each of a row's threads counts
      if constexpr (CH == 2) {
        // the state of the row's other thread, whose O is in the same TMEM lane
        float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl) + half * 2 * BM + row;
        ml[ch * BM] = make_float2(m_ref, l);
        warp_arrive(&bars->ml_full[half * 4 + wq], lane);
        if (!(ok = warp_wait(smem_u32(&bars->ml_full[half * 4 + wq]), mph, abort))) break;
        mph ^= 1;
        const float2 o = ml[(ch ^ 1) * BM];
        const float m = fmaxf(m_ref, o.x);
        own = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
        other = o.x == -INFINITY ? 0.f : ex2_approx(o.x - m);
        l = l * own + o.y * other;
        m_ref = m;
      }
      const int64_t out = (int64_t)(w.token + lp) * p.Hq + w.hk * p.G + h_off;  // the row of o and lse
      const Work wk = work_of(p.work, D);
      const int64_t part_row = (2 * (int64_t)blockIdx.x + (w.j0 > 0 ? 0 : 1)) * kRows + half * BM + row;
      const float inv = (MX4 ? (float)(1ull << kUnitLog) : 1.f) / l;
#pragma unroll 1
      for (int c = ch; c < D / NE; c += CH) {
        uint32_t x[NE];
        __syncwarp();
        tmem_ld(ocol + ch * D + c * NE, x);
        tmem_ld_wait(x);
        float r[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) r[i] = __uint_as_float(x[i]);
        if constexpr (CH == 2) {
          tmem_ld(ocol + (ch ^ 1) * D + c * NE, x);
          tmem_ld_wait(x);
#pragma unroll
          for (int i = 0; i < NE; ++i) r[i] = r[i] * own + __uint_as_float(x[i]) * other;
        }
        // (Any place will do, and the answer is looked up for each part of O: d = 64 1336 us beside
        // 1348 with it kept over them; from the half's own place 1366, by a count of its tiles 1372.)
        const bool poisoned =
            __any_sync(0xffffffffu, ((volatile int*)&bars->poison[0][0])[lane & 15] == ((k + 1) & 0xffff));
        if (poisoned && there) {
          // infinities or NaN were taken out of V rows that not all queries see: this
          // row's own are added, found again in global memory
          auto add = [&](int i0, const uint4& y) {  // elements i0 .. i0 + 7 of the NE
            const uint32_t q[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < NE; i += 2)
              if (i >> 3 == i0 >> 3) {
                const uint32_t v = q[(i & 7) >> 1], f = not_finite(v);
                if (f & 0x8000u) r[i] += __uint_as_float(v << 16);
                if (f & 0x80000000u) r[i + 1] += __uint_as_float(v & 0xffff0000u);
              }
          };
          Sched again(p.n_depth, w.nb, w.j0);
#pragma unroll 1
          for (int j = w.j0; j < w.j1; ++j) {
            again.next(p.n_depth, w.nb);
            if (again.depth) {
              const int l_end = min(p.L, (again.index + 1) * SP);
#pragma unroll 1
              for (int slot = again.index * SP; slot < l_end; ++slot) {
                const uint4* v = reinterpret_cast<const uint4*>(p.vd + (int64_t)(w.token + lp) * p.depth_tok +
                                                                (int64_t)w.hk * p.depth_hk +
                                                                (int64_t)slot * p.depth_slot + c * NE);
#pragma unroll 1
                for (int i = 0; i < NE / 8; ++i) add(i * 8, v[i]);
              }
            } else if (again.index * BN + BN - 1 > w.t0) {
              const int k_end = min(w.t0 + lp + 1, (again.index + 1) * BN);
#pragma unroll 1
              for (int key = again.index * BN; key < k_end; ++key) {
                int pg = p.table[(int64_t)w.b * p.max_pages + (key >> p.page_shift)];
                if (pg < 0 || pg >= p.num_pages) pg = 0;
                const int64_t vr = ((int64_t)(pg * p.Hk + w.hk) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
#pragma unroll 1
                for (int i = 0; i < NE / 8; ++i) {
                  uint4 y;
                  if constexpr (MX4) {
                    uint32_t z[4];
                    unpack8(*reinterpret_cast<const uint32_t*>(p.v + vr * (D / 2) + c * (NE / 2) + i * 4),
                            scale_in_units(p.v_scale[vr * (D / 32) + c * NE / 32], kUnitLog), z);
                    y = make_uint4(z[0], z[1], z[2], z[3]);
                  } else {
                    y = *reinterpret_cast<const uint4*>(p.v + (vr * D + c * NE + i * 8) * 2);
                  }
                  add(i * 8, y);
                }
              }
            }
          }
        }
        if (!there) continue;
        if (cut) {
          float4* po = reinterpret_cast<float4*>(wk.o + part_row * D + c * NE);
#pragma unroll
          for (int i = 0; i < NE / 4; ++i) po[i] = make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        } else {
          uint4* po = reinterpret_cast<uint4*>(p.o + out * D + c * NE);
#pragma unroll
          for (int i = 0; i < NE / 8; ++i)
            po[i] = make_uint4(pack_bf16x2(r[8 * i] * inv, r[8 * i + 1] * inv),
                               pack_bf16x2(r[8 * i + 2] * inv, r[8 * i + 3] * inv),
                               pack_bf16x2(r[8 * i + 4] * inv, r[8 * i + 5] * inv),
                               pack_bf16x2(r[8 * i + 6] * inv, r[8 * i + 7] * inv));
        }
      }
      if (there && ch == 0 && cut)
        *reinterpret_cast<float2*>(wk.ml + part_row * 2) = make_float2(m_ref, l);
      else if (there && ch == 0 && p.lse)
        p.lse[out] = (m_ref + log2f(l)) * kLn2;
      // (the next tile's first P V, which overwrites O, follows this warp's next p_full)
      tc_fence_before();
    }
    if (tid == 128 && !opened) work_of(p.work, D).opened[blockIdx.x] = {0, 0, 0, 0};
  } else {
    // ----------------------------- 4-bit pages unpacked, V blocks made harmless
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsTame));
    const bool is_v = warp < C::kTame0 + 4;
    const int hw = warp & 3, r = tid & 127;  // a row of a tile each
    const int ns = is_v ? NV : NK;
    const uint32_t full = smem_u32(is_v ? (MX4 ? bars->v_full : bars->v_ready) : bars->k_full);
    const uint32_t check = smem_u32(is_v ? bars->v_check : bars->k_check);
    int s = 0, ph = 0;    // the next entry's stage and phase
    uint32_t checks = 0;  // parities of `check`
    bool ok = true;
    Walk& w = bars->walk[warp - 4];
    for (bool first = true; ok && warp_next(w, p, sh, lane, first); first = false) {
      const int halves = w.npos > P ? 2 : 1;
      Sched sch(p.n_depth, w.nb, w.j0);
      using Cd = Codes<D>;
      Cd c;  // of the next sequence block
      const int* table = p.table + (int64_t)w.b * p.max_pages;
      // A sequence block's codes on their way (for rows that no query sees those of the last
      // that one does), and the pages of the one after into L1. Nothing here may wait for
      // what it loads: registers spilled or chosen between cost 2400 cycles a block.
      auto fetch = [&](int index) {
        uint32_t at[Cd::kTurns];
#pragma unroll
        for (int t = 0; t < Cd::kTurns; ++t) {
          const int key = min(index * BN + Cd::row(t, hw, lane), w.t_last);
          at[t] = (uint32_t)table[key >> p.page_shift];
          asm volatile("prefetch.global.L1 [%0];" ::"l"(table + (min(key + BN, w.t_last) >> p.page_shift)));
        }
        bool bad = false;
#pragma unroll
        for (int t = 0; t < Cd::kTurns; ++t) {
          const int key = min(index * BN + Cd::row(t, hw, lane), w.t_last);
          bad |= at[t] >= (uint32_t)p.num_pages;
          at[t] = ((min(at[t], (uint32_t)p.num_pages - 1) * p.Hk + w.hk) << p.page_shift) +
                  (key & ((1 << p.page_shift) - 1));
        }
        if (bad) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
        const uint8_t *codes = is_v ? p.v : p.k, *scales = is_v ? p.v_scale : p.k_scale;
#pragma unroll
        for (int t = 0; t < Cd::kTurns; ++t) {
          c.codes[t] = *reinterpret_cast<const uint4*>(codes + (uint64_t)at[t] * (D / 2) + lane % Cd::BPR * 16);
          c.scale[t] = scales[(uint64_t)at[t] * Cd::BPR + lane % Cd::BPR];
        }
      };
      if constexpr (MX4) fetch(sch.sbk);
      for (int j = w.j0; ok && j < w.j1; ++j) {
        sch.next(p.n_depth, w.nb);
        const bool part = partly_seen(w, sch);
        for (int x = 0; ok && x < (sch.depth ? halves : 1); ++x) {
          uint8_t* tile = smem + (is_v ? C::kOffV : C::kOffK) + s * C::kTileBytes;
          if (MX4 || part) {
            // rows that some query of the tile sees
            auto counts = [&](int y) -> bool {
              if (!sch.depth) return sch.index * BN + y <= w.t_last;
              return x * P + (y >> 5) * PW + (y & (PW - 1)) < w.npos && sch.index * SP + (y & 31) / PW < p.L;
            };
            bool found = false;
            // (4-bit pages: each stage's phases one by one; a depth block's are seen by warp 3 too)
            if (MX4 && !(ok = warp_wait(smem_u32(is_v ? &bars->v_empty[s] : &bars->k_empty[s]), ph ^ 1, abort))) break;
            if (!MX4 || sch.depth) {
              if (!(ok = warp_wait(check + s * 8, checks >> s & 1, abort))) break;
              checks ^= 1u << s;
              if (is_v) found = tame_row<D>(tile, r, counts(r));
            } else {
              found = c.unpack(smem_u32(tile), hw, lane, w.t_last + 1 - sch.index * BN, is_v && part,
                               is_v ? kUnitLog : 0);
              fetch(sch.index + 1);
            }
            if (found) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (h < halves) *(volatile int*)&bars->poison[h][w.nth[h] & 7] = w.nth[0];
              __threadfence_block();
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(full + s * 8);
          }
          if (++s == ns) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if (tid == 0 && bars->abort) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_TIMEOUT);
}

// The cut tiles' rows from their partials: a warp for each row of the tile that
// CTA blockIdx.x begins (if any), its partials' loads in flight at once.
constexpr int kJoinWarps = 8, kJoinParts = 16;  // warps of a CTA, CTAs of a tile

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
prefill_join_kernel(const __grid_constant__ Params p) {
  constexpr int E = D / 32, U = 4;
  const Work wk = work_of(p.work, D);
  const int lane = threadIdx.x & 31;
  paged::wait_for_stream();
  const Opened t = wk.opened[blockIdx.x];
  if (t.parts == 0) return;
  const int G2 = 1 << p.lgG;
  const int stride = kJoinWarps * kJoinParts;
  for (int row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); row < t.npos << p.lgG; row += stride) {
    const int h = row & (G2 - 1);
    if (h >= p.G) continue;
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < t.parts; i0 += U) {
      float pm[U], pl[U], po[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        pm[u] = -INFINITY;
        pl[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) po[u][e] = 0.f;
        if (i < t.parts) {
          const int64_t at = (int64_t)(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * kRows + row;
          pm[u] = wk.ml[at * 2];
          pl[u] = wk.ml[at * 2 + 1];
#pragma unroll
          for (int e = 0; e < E; ++e) po[u][e] = wk.o[at * D + lane * E + e];
        }
      }
      paged::add_partials<U, E>(M, L, acc, pm, pl, po);
    }
    const int64_t out = (int64_t)(t.token + (row >> p.lgG)) * p.Hq + t.hk * p.G + h;
    const float inv = p.unit / L;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(p.o + out * D + lane * E + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse) p.lse[out] = (M + log2f(L)) * kLn2;
  }
}

template <int D, bool MX4>
cudaError_t launch(const PrefillPagedArgs& a, cudaStream_t stream) {
  using C = Cfg<D, MX4>;
  const PagedKv& c = a.c;
  int lgG = 0;
  while (1 << lgG < a.G) ++lgG;
  const int P = BM >> lgG, PW = P / 4;
  const uint64_t row = (uint64_t)D * 2;
  CUtensorMap tq, tk, tv, tkd, tvd;
  {
    // (a stride that is never stepped: any valid one)
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.N};
    const uint64_t str[2] = {row, (uint64_t)a.q_stride * 2};
    const uint32_t box[3] = {64, 1u << lgG, (uint32_t)P};
    if (encode_bf16_sw128(&tq, a.q, 3, dims, str, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  }
  if (!MX4) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)c.page_size, (uint64_t)c.num_pages * c.Hk};
    const uint64_t str[2] = {row, row * c.page_size};
    const uint32_t box[3] = {64, (uint32_t)c.page_size, 1};
    if (encode_bf16_sw128(&tk, c.k, 3, dims, str, box) != CUDA_SUCCESS ||
        encode_bf16_sw128(&tv, c.v, 3, dims, str, box) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  } else {
    tk = tv = tq;  // not read
  }
  if (a.L > 0) {
    // a box is one softmax warp's word, PW positions x 32 / PW slots
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)c.Hk, (uint64_t)a.N, (uint64_t)a.L};
    const uint64_t str[3] = {(uint64_t)a.depth_hk_stride * 2, (uint64_t)a.depth_tok_stride * 2,
                             (uint64_t)a.depth_slot_stride * 2};
    const uint32_t box[4] = {64, 1, (uint32_t)PW, 32u / PW};
    if (encode_bf16_sw128(&tkd, a.kd, 4, dims, str, box) != CUDA_SUCCESS ||
        encode_bf16_sw128(&tvd, a.vd, 4, dims, str, box) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  } else {
    tkd = tvd = tq;  // not read
  }
  Params p;
  p.q_starts = a.q_starts; p.lens = a.seq_lens; p.table = c.table;
  p.N = a.N; p.num_pages = c.num_pages; p.page_shift = __builtin_ctz((unsigned)c.page_size);
  p.max_pages = c.max_pages; p.B = c.B; p.Hq = a.Hq; p.Hk = c.Hk; p.G = a.G; p.L = a.L;
  p.lgG = lgG;
  p.lg_per = 0;
  while ((int64_t)C::kThreads << p.lg_per < c.B) ++p.lg_per;
  p.n_depth = (PW * a.L + 31) / 32;
  p.scale_log2 = a.scale * kLog2e;
  p.unit = MX4 ? (float)(1ull << kUnitLog) : 1.f;
  p.o = (__nv_bfloat16*)a.o; p.lse = a.lse; p.work = a.work; p.err = c.err;
  p.k = (const uint8_t*)c.k; p.v = (const uint8_t*)c.v;
  p.k_scale = (const uint8_t*)c.k_scale; p.v_scale = (const uint8_t*)c.v_scale;
  p.vd = (const __nv_bfloat16*)a.vd;
  p.depth_tok = a.depth_tok_stride; p.depth_hk = a.depth_hk_stride; p.depth_slot = a.depth_slot_stride;
  const int grid = a.num_sms < kMaxCtas ? a.num_sms : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(prefill_paged_kernel<D, MX4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  e = paged::launch_dependent(prefill_paged_kernel<D, MX4>, dim3(grid), C::kThreads, C::kSmemBytes, stream, tq, tk, tv,
                              tkd, tvd, p);
  if (e != cudaSuccess) return e;
  return paged::launch_dependent(prefill_join_kernel<D>, dim3(grid, kJoinParts), kJoinWarps * 32, 0, stream, p);
}

}  // namespace
}  // namespace prefill

size_t prefill_paged_workspace_bytes(int d) {
  return ((size_t)4 * prefill::kMaxCtas + (size_t)2 * prefill::kMaxCtas * prefill::kRows * (d + 2)) * sizeof(float);
}

cudaError_t launch_prefill_paged(const PrefillPagedArgs& a, cudaStream_t stream) {
  const bool mx4 = a.c.format == MODA_KV_MX4;
  if (a.c.d == 128) return mx4 ? prefill::launch<128, true>(a, stream) : prefill::launch<128, false>(a, stream);
  return mx4 ? prefill::launch<64, true>(a, stream) : prefill::launch<64, false>(a, stream);
}

}  // namespace moda
