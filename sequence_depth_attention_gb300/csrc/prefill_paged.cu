// MoDA attention of a chunk of new tokens per sequence over the paged KV cache:
// the tokens of a batch (pieces of prompts, drafts to verify) attend, under one
// softmax, to the rows of their sequence's pages up to their own and to the L depth
// slots of their own position.
//
// The forward's organisation (fwd_tc.cu) over pages and ragged sequences: a tile
// is the G heads of one KV head x P positions of one sequence, 128 rows;
// S = Q K^T and O += P V on tcgen05 with S, P, Q and O in tensor memory, K and V
// through shared memory by TMA, one softmax thread per row, the depth slots
// gathered as blocks with a block-diagonal mask. What differs:
//   * the work is cut into equal shares of a line of blocks (prefill_paged.cuh):
//     a draft of five tokens over a long context is spread over the SMs like a
//     long prompt, and the lengths stay on the device;
//   * a block of 128 keys is up to 8 pages, each looked up and copied by a lane;
//   * 4-bit pages come as codes and scales; four warps unpack them into the bf16
//     tiles that the tensor core reads (exactly: a code times a power of two);
//   * those warps also see to it that a row that a query must not see has no
//     influence whatever it holds. Its weight is 0, but 0 times an infinity or a
//     NaN in V is NaN: in the blocks that some row of a tile sees in part (the
//     causal border, the depth blocks), rows that no query of the tile sees
//     become 0, and an infinity or NaN among the others becomes 0 too and is added
//     at the end to the rows that do see it.
//
// Roles (12 warps):
//   warp 0  TMA producer of Q and K     warp 1  issuer of S = Q K^T, TMEM
//   warp 2  TMA producer of V           warp 3  issuer of O += P V
//   warps 4-7   softmax, Q into TMEM, epilogue: one thread per row (TMEM lane)
//   warps 8-11  4-bit pages unpacked, partly seen V blocks made harmless
// TMEM (512 columns): S double buffer [0,128) [128,256), O [256, 256+d), P (bf16
// pairs) [384,448), Q (bf16 pairs) [448, 448+d/2).
// P is rounded to bf16 once, as in the forward: the sum l keeps fp32 weights, and
// what o is off by that is about as much as its own rounding to bf16.
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

constexpr int BM = kRows, BN = 128;
constexpr int kWarps = 12, kThreads = kWarps * 32;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kSumBound = 256.0f;        // 2^kRescaleThreshold
constexpr int kLeast = 2;                  // points that are worth a CTA
// Registers: 384 threads x 168 at launch; the softmax warps take 240 and the first
// four give theirs (128 x (96 + 240 + 168) <= 384 x 168).
constexpr int kRegsIssue = 96, kRegsSoftmax = 240;
static_assert(128 * (kRegsIssue + kRegsSoftmax + 168) <= kThreads * 168, "within the launch's registers");

template <int D, bool MX4>
struct Cfg {
  static constexpr int kBoxes = D / 64;  // 64-column (128-byte) swizzle boxes per row
  static constexpr int kBoxBytes = BN * 128;
  static constexpr int kQBytes = BM * D * 2;
  static constexpr int kTileBytes = BN * D * 2;
  static constexpr int kNS = MX4 ? (D == 128 ? 2 : 4) : (D == 128 ? 3 : 6);  // stages of K, and of V
  // 4-bit rows on their way: codes, then scales
  static constexpr int kRawCodes = BN * D / 2, kRawScales = BN * D / 32;
  static constexpr int kRawBytes = kRawCodes + kRawScales;
  // (at most kNS: a producer that finds an entry free then knows that the tile before the
  // last in its stage is done with, so it cannot take that one's phase for the last one's)
  static constexpr int kNR = MX4 ? (D == 128 ? 2 : 3) : 0;
  static_assert(kNR <= kNS);
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + kNS * kTileBytes;
  static constexpr int kOffRawK = kOffV + kNS * kTileBytes;
  static constexpr int kOffRawV = kOffRawK + kNR * kRawBytes;
  static constexpr int kOffBar = kOffRawV + kNR * kRawBytes;
  static constexpr int kSmemBytes = kOffBar + 1536 + 1024;  // barriers, alignment
  static constexpr uint32_t kColS = 0, kColO = 256, kColP = 384, kColQ = 448;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kOffBar % 16 == 0 && kRawBytes % 16 == 0);
};

struct alignas(16) Barriers {
  uint64_t q_full, q_tmem;  // Q of the current tile landed / copied into TMEM
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  // bf16 pages: a partly seen V block lands at v_check and not at v_full, and is v_ready
  // once it has been made harmless. (A barrier of its own, whose phases the warps that
  // do it wait for one by one: they skip the other blocks.)
  uint64_t v_check[6], v_ready[6];
  uint64_t raw_k_full[4], raw_k_empty[4], raw_v_full[4], raw_v_empty[4];
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t mma_done, mma_done_pv;
  uint32_t tmem_base;
  int abort;
  int poison[8];  // [k % 8] = k + 1: tile k had infinities or NaN taken out (at most kNS tiles are under way)
  ShareSmem<kWarps> find;
  Share share;
  Walk walk[4];  // of the softmax warps, whose registers are full
};
static_assert(sizeof(Barriers) <= 1536, "barrier block");

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait_bounded(bar, parity, abort, kTimeoutNs);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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
#pragma unroll
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

// A 4-bit tile (codes, then scales) into a bf16 tile, by four warps: lane group
// of D / 32 lanes a row, a block of 32 elements a lane. TAME: as tame_row, with
// counts(r) for the rows.
template <int D, bool TAME, class Counts>
__device__ __forceinline__ bool unpack_tile(const uint8_t* raw, uint8_t* tile, int warp, int lane, Counts counts) {
  constexpr int BPR = D / 32;          // blocks, and lanes, of a row
  constexpr int RPI = 32 / BPR;        // rows a warp takes at once
  constexpr int kBoxBytes = BN * 128;
  const int qtr = lane % BPR;
  bool found = false;
#pragma unroll
  for (int it = 0; it < BN / (4 * RPI); ++it) {
    const int r = (it * 4 + warp) * RPI + lane / BPR;
    const uint4 codes = *reinterpret_cast<const uint4*>(raw + r * (D / 2) + qtr * 16);
    const uint32_t b = raw[BN * D / 2 + r * BPR + qtr];
    uint32_t mul, mul2;
    factors(b, mul, mul2);
    const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
    // the block's four 16-byte chunks; in the order that the lanes of eight
    // (two rows) meet different banks
    uint8_t* row = tile + (qtr >> 1) * kBoxBytes + r * 128;
    uint32_t y[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack8(cw[j], mul, mul2, y[j]);
    if constexpr (TAME) {
      const bool c = counts(r);
      if (!c || b >= 253u) {
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f = not_finite(y[j][i]);
            bad |= f;
            y[j][i] &= c ? ~(((f & 0x8000u) ? 0xffffu : 0u) | ((f & 0x80000000u) ? 0xffff0000u : 0u)) : 0u;
          }
        found |= c && bad;
      }
    }
    const int turn = (qtr >> 1) << 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int jj = j;  // chunk 4 (qtr & 1) + j of the 64-column box
      const int chunk = 4 * (qtr & 1) + (jj ^ turn);
      // y is indexed by the chunk that is stored: a select between two, both static
      const uint32_t* lo = y[jj];
      const uint32_t* hi = y[jj ^ 2];
      const uint4 v = turn ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(row + ((chunk ^ (r & 7)) << 4)) = v;
    }
  }
  return found;
}

template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads, 1)
prefill_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKd,
                     const __grid_constant__ CUtensorMap tmVd, const __grid_constant__ Params p) {
  using C = Cfg<D, MX4>;
  constexpr int NS = C::kNS, NR = MX4 ? C::kNR : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Barriers* bars = reinterpret_cast<Barriers*>(smem + C::kOffBar);
  const uint32_t sQ = smem_u32(smem), sK = smem_u32(smem + C::kOffK), sV = smem_u32(smem + C::kOffV);
  volatile int* abort = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G2 = 1 << p.lgG, P = BM >> p.lgG;
  const int PW = P >> 2, SP = 32 / PW;  // positions and slots of a softmax warp's word of a depth block

  if (tid == 0) {
    bars->abort = 0;
    for (int& x : bars->poison) x = 0;
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_tmem), 128);
    for (int s = 0; s < 6; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), MX4 ? 128 : 1);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
      mbar_init(smem_u32(&bars->v_full[s]), MX4 ? 128 : 1);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
      mbar_init(smem_u32(&bars->v_check[s]), 1);
      mbar_init(smem_u32(&bars->v_ready[s]), 128);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(smem_u32(&bars->raw_k_full[s]), 1);
      mbar_init(smem_u32(&bars->raw_k_empty[s]), 128);
      mbar_init(smem_u32(&bars->raw_v_full[s]), 1);
      mbar_init(smem_u32(&bars->raw_v_empty[s]), 128);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars->s_full[b]), 1);
      mbar_init(smem_u32(&bars->s_free[b]), 128);
      mbar_init(smem_u32(&bars->p_full[b]), 128);
      mbar_init(smem_u32(&bars->pv_done[b]), 1);
    }
    mbar_init(smem_u32(&bars->mma_done), 1);
    mbar_init(smem_u32(&bars->mma_done_pv), 1);
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
    const Share mine = share_of<kWarps, kLeast>(p, bars->find);
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------- TMA producers
      const bool is_k = warp == 0;
      const bool leader = elect_one();
      const uint64_t pol_once = l2_policy_evict_first();
      const CUtensorMap* seq_map = is_k ? &tmK : &tmV;
      const CUtensorMap* dep_map = is_k ? &tmKd : &tmVd;
      uint64_t* full = MX4 ? (is_k ? bars->raw_k_full : bars->raw_v_full) : (is_k ? bars->k_full : bars->v_full);
      uint64_t* empty = MX4 ? (is_k ? bars->raw_k_empty : bars->raw_v_empty) : (is_k ? bars->k_empty : bars->v_empty);
      uint64_t* tile_empty = is_k ? bars->k_empty : bars->v_empty;
      constexpr int NF = MX4 ? NR : NS;  // entries of `full`
      const uint32_t tiles = is_k ? sK : sV;
      const uint32_t raws = smem_u32(smem + (is_k ? C::kOffRawK : C::kOffRawV));
      const int page_rows = 1 << p.page_shift;  // at most 128
      // a lane copies one page's rows (bf16: 64 columns of them)
      constexpr int kParts = MX4 ? 1 : C::kBoxes;
      const int my_box = lane / kParts, my_part = lane % kParts;
      int g = 0, nq = 0;
      uint32_t checks = 0, wholes = 0;  // of V's stages: parities of what went to v_check, to v_full
      uint32_t any_check = 0, any_whole = 0;
      Walk w;
      w.begin(p, sh);
      bool ok = true;
      for (int k = 0; ok && w.next(p, sh); ++k) {
        if (is_k) {
          // Q, once the softmax warps have copied the previous one into TMEM
          if (k > 0 && !warp_wait(smem_u32(&bars->q_tmem), (k - 1) & 1, abort)) break;
          if (leader) {
            const uint32_t qb = smem_u32(&bars->q_full);
            mbar_arrive_expect_tx(qb, C::kQBytes);
            for (int c = 0; c < C::kBoxes; ++c)
              tma_load_3d_hint(sQ + c * C::kBoxBytes, &tmQ, qb, c * 64, w.hk * p.G, w.token, pol_once);
          }
          ++nq;
        }
        Sched sch(p.n_depth, w.nb, w.j0);
        const int* table = p.table + (int64_t)w.b * p.max_pages;
        // the lane's page of the sequence block after this one, looked up ahead
        auto page_of = [&](int index) -> int {
          const int key = index * BN + (my_box << p.page_shift);
          return my_box << p.page_shift < BN && key <= w.t_last ? table[key >> p.page_shift] : -1;
        };
        int page = page_of(sch.sbk);
        for (int j = w.j0; j < w.j1; ++j, ++g) {
          sch.next(p.n_depth, w.nb);
          const int f = g % NF, s = g % NS;
          int pg = page;
          if (!sch.depth) page = page_of(sch.index + 1);
          if (!warp_wait(smem_u32(&empty[f]), ((g / NF) & 1) ^ 1, abort)) {
            ok = false;
            break;
          }
          uint32_t fb = smem_u32(&full[f]);
          if (!MX4 && !is_k) {
            if (partly_seen(w, sch)) {
              fb = smem_u32(&bars->v_check[s]);
              checks ^= 1u << s;
              any_check |= 1u << s;
            } else {
              wholes ^= 1u << s;
              any_whole |= 1u << s;
            }
          }
          if (sch.depth) {
            // the words of the softmax warps that have positions: slots [SP index, + SP)
            // of warp w's PW positions, row slot * PW + position (4-bit pages: straight
            // into the tile, whose consumers are done then)
            if (MX4 && !warp_wait(smem_u32(&tile_empty[s]), ((g / NS) & 1) ^ 1, abort)) {
              ok = false;
              break;
            }
            if (leader) {
              const int words = (w.npos + PW - 1) / PW;
              mbar_arrive_expect_tx(fb, words * 32 * D * 2);
              const uint32_t dst = tiles + s * C::kTileBytes;
              for (int x = 0; x < words; ++x)
                for (int c = 0; c < C::kBoxes; ++c)
                  tma_load_4d_hint(dst + c * C::kBoxBytes + x * 32 * 128, dep_map, fb, c * 64, w.hk,
                                   w.token + x * PW, sch.index * SP, pol_once);
            }
          } else {
            const int rows = min(BN, w.t_last + 1 - sch.index * BN);
            const int boxes = (rows + page_rows - 1) >> p.page_shift;
            if (leader) mbar_arrive_expect_tx(fb, boxes * page_rows * (MX4 ? D / 2 + D / 32 : D * 2));
            __syncwarp();
            if (my_box < boxes) {
              if (pg < 0 || pg >= p.num_pages) {
                atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
                pg = 0;
              }
              const int head = pg * p.Hk + w.hk;
              if constexpr (MX4) {
                const uint32_t dst = raws + f * C::kRawBytes;
                const int64_t row = (int64_t)head << p.page_shift;
                bulk_load(dst + my_box * page_rows * (D / 2), (is_k ? p.k : p.v) + row * (D / 2),
                          page_rows * (D / 2), fb);
                bulk_load(dst + C::kRawCodes + my_box * page_rows * (D / 32),
                          (is_k ? p.k_scale : p.v_scale) + row * (D / 32), page_rows * (D / 32), fb);
              } else {
                tma_load_3d(tiles + s * C::kTileBytes + my_part * C::kBoxBytes + my_box * page_rows * 128, seq_map,
                            fb, my_part * 64, 0, head);
              }
            }
          }
          __syncwarp();
        }
      }
      // every copy of this warp has landed before its shared memory is released
      if (leader) {
        int never = 0;
        if (!MX4 && !is_k) {
          for (int s = 0; s < NS; ++s) {
            if (any_whole >> s & 1)
              mbar_wait_bounded(smem_u32(&bars->v_full[s]), (wholes >> s & 1) ^ 1, &never, kTimeoutNs);
            if (any_check >> s & 1)
              mbar_wait_bounded(smem_u32(&bars->v_check[s]), (checks >> s & 1) ^ 1, &never, kTimeoutNs);
          }
        } else {
          for (int j = max(0, g - NF); j < g; ++j)
            mbar_wait_bounded(smem_u32(&full[j % NF]), (j / NF) & 1, &never, kTimeoutNs);
        }
        if (is_k && nq > 0) mbar_wait_bounded(smem_u32(&bars->q_full), (nq - 1) & 1, &never, kTimeoutNs);
      }
      __syncwarp();
    } else if (elect_one()) {
      // ------------------------------------------------------- MMA issuers
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return mbar_wait_bounded(smem_u32(bar), parity, abort, kTimeoutNs);
      };
      const uint64_t dk = sdesc_sw128(sK, 16, 1024);
      const uint32_t hi = (uint32_t)(dk >> 32);
      int g = 0;
      bool ok = true;
      Walk w;
      w.begin(p, sh);
      if (warp == 1) {
        constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false);
        const uint32_t k_lo = (uint32_t)dk;
        for (int k = 0; ok && w.next(p, sh); ++k) {
          if (!wait(&bars->q_tmem, k & 1)) break;
          for (int j = w.j0; j < w.j1; ++j, ++g) {
            const int ks = g % NS;
            if ((g >= 2 && !wait(&bars->s_free[g & 1], ((g - 2) >> 1) & 1)) ||
                !wait(&bars->k_full[ks], (g / NS) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t kb = k_lo + ((uint32_t)(ks * C::kTileBytes) >> 4);
            const uint32_t dcol = tbase + C::kColS + (g & 1) * 128;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
              mma_ts(dcol, tbase + C::kColQ + kk * 8, desc_join(kb + off, hi), idS, kk > 0);
            }
            tc_commit(smem_u32(&bars->k_empty[ks]));
            tc_commit(smem_u32(&bars->s_full[g & 1]));
          }
        }
      } else {
        constexpr uint32_t idPV = idesc_bf16_f32(BM, D, true);
        const uint32_t v_lo = (uint32_t)sdesc_sw128(sV, C::kBoxBytes, 1024);
        const uint32_t pcol = tbase + C::kColP;
        uint32_t ready = 0, whole = 0;  // bf16: parities of v_ready and v_full, a bit for each stage
        for (int k = 0; ok && w.next(p, sh); ++k) {
          Sched sch(p.n_depth, w.nb, w.j0);
          for (int j = w.j0; j < w.j1; ++j, ++g) {
            sch.next(p.n_depth, w.nb);
            const int sb = g & 1, vs = g % NS;
            bool there;
            if (MX4) {
              there = wait(&bars->v_full[vs], (g / NS) & 1);
            } else if (partly_seen(w, sch)) {
              there = wait(&bars->v_ready[vs], (ready >> vs) & 1);
              ready ^= 1u << vs;
            } else {
              there = wait(&bars->v_full[vs], (whole >> vs) & 1);
              whole ^= 1u << vs;
            }
            if (!there || !wait(&bars->p_full[sb], (g >> 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t vb = v_lo + ((uint32_t)(vs * C::kTileBytes) >> 4);
            // a tile's first P V overwrites O (the softmax warps have read the previous
            // tile's O before they stored this P)
            const uint32_t acc0 = j > w.j0 ? 1u : 0u;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              mma_ts(tbase + C::kColO, pcol + kk * 8, desc_join(vb + ((uint32_t)(kk * 2048) >> 4), hi), idPV,
                     kk > 0 ? 1u : acc0);
            tc_commit(smem_u32(&bars->v_empty[vs]));
            tc_commit(smem_u32(&bars->pv_done[sb]));
          }
        }
      }
      // every MMA issued by this thread has completed before TMEM is freed
      uint64_t* done = warp == 1 ? &bars->mma_done : &bars->mma_done_pv;
      int never = 0;
      tc_commit(smem_u32(done));
      mbar_wait_bounded(smem_u32(done), 0, &never, kTimeoutNs);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ----------------------------------------------------- softmax, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int row = tid - 128;  // tile row == TMEM lane
    const uint32_t lane_base = (uint32_t)(warp & 3) * 32;
    const int wq = warp & 3;  // this warp's word of a depth block
    const int lp = row >> p.lgG, h_off = row & (G2 - 1);
    const int lpw = (row & 31) >> p.lgG;  // the row's position among its warp's
    const uint32_t own_cols = PW >= 32 ? 1u << lpw : (0xffffffffu / ((1u << PW) - 1u)) << lpw;
    const float sl = p.scale_log2;
    const uint32_t zeros[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    bool p_zero = false;  // this warp's P columns outside its depth word hold zeros
    int g = 0;
    // Q of tile k -> TMEM as bf16 pairs, the A operand of S = Q K^T; rows that no
    // query has become 0. Called once every S product of the tile before has completed.
    auto copy_q = [&](int k, const Walk& t) -> bool {
      if (!warp_wait(smem_u32(&bars->q_full), k & 1, abort)) return false;
      const bool there = lp < t.npos && h_off < p.G;
      const uint8_t* qrow = smem + row * 128;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + c * C::kBoxBytes + ((i ^ (row & 7)) << 4));
          x[4 * i] = there ? v.x : 0u;
          x[4 * i + 1] = there ? v.y : 0u;
          x[4 * i + 2] = there ? v.z : 0u;
          x[4 * i + 3] = there ? v.w : 0u;
        }
        tmem_st32(tmem_addr(tbase, lane_base, C::kColQ + c * 32), x);
      }
      tmem_st_wait();
      tc_fence_before();
      fence_async();  // the Q region takes the next tile's Q (a TMA write): order these reads first
      mbar_arrive(smem_u32(&bars->q_tmem));
      return true;
    };
    Walk& w = bars->walk[wq];
    // to the next tile; the warp has read what it wants of the one before
    auto advance = [&](bool first) -> bool {
      bool any = false;
      __syncwarp();
      if (lane == 0) {
        if (first) w.begin(p, sh);
        any = w.next(p, sh);
      }
      any = __shfl_sync(0xffffffffu, any, 0);
      __syncwarp();  // what lane 0 has written is seen
      return any;
    };
    bool more = advance(true), ok = !more || copy_q(0, w);
    bool opened = false;
    for (int k = 0; ok && more; ++k) {
      float m_ref = -INFINITY, l = 0.f;
      // Rescale O and l to a new reference when a block's raw max mx (log2 units) rose
      // more than the threshold above it; false on a timeout. O holds blocks j0 .. j - 1.
      auto rescale = [&](float mx, int j) -> bool {
        const bool need = mx > m_ref + kRescaleThreshold;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? mx : m_ref;
          const float alpha = need ? ex2_approx(m_ref - m_new) : 1.f;
          if (j > w.j0) {
            if (!warp_wait(smem_u32(&bars->pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort)) return false;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t r[32];
              const uint32_t ta = tmem_addr(tbase, lane_base, C::kColO + c * 32);
              tmem_ld32(ta, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
              tmem_st32(ta, r);
            }
            tmem_st_wait();
          }
          l *= alpha;
          m_ref = m_new;
        }
        return true;
      };
      // Every block: exponentiate against the running reference right away. Every p is
      // at most the block's sum, so a sum within 2^threshold proves that no score rose
      // more than that above it, and the block needs no maximum at all.
      Sched sch(p.n_depth, w.nb, w.j0);
      for (int j = w.j0; j < w.j1; ++j, ++g) {
        sch.next(p.n_depth, w.nb);
        const int sb = g & 1;
        if (!warp_wait(smem_u32(&bars->s_full[sb]), (g >> 1) & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t pcol = tmem_addr(tbase, lane_base, C::kColP);
        float sum = 0.f;
        if (sch.depth) {
          // only this warp's word of 32 columns can hold its rows' slots: column c is
          // slot index * SP + c / PW of the warp's position c % PW
          uint32_t xs[32];
          tmem_ld32(tmem_addr(tbase, lane_base, C::kColS + sb * 128 + wq * 32), xs);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(smem_u32(&bars->s_free[sb]));
          const int nbits = min(SP, p.L - sch.index * SP) * PW;
          const uint32_t word =
              lp < w.npos ? own_cols & (nbits >= 32 ? 0xffffffffu : (1u << nbits) - 1u) : 0u;
#pragma unroll
          for (int i = 0; i < 32; ++i) xs[i] = (word & (1u << i)) ? xs[i] : 0xff800000u;  // -inf
          uint32_t pk[16];
          bool slow = __any_sync(0xffffffffu, m_ref == -INFINITY);
          if (!slow) {
            sum = exp_block<32>(xs, pk, sl, m_ref);
            slow = __any_sync(0xffffffffu, !(sum <= kSumBound));
          }
          if (slow) {
            if (!rescale(raw_max32(xs) * sl, j)) {
              ok = false;
              break;
            }
            sum = exp_block<32>(xs, pk, sl, m_ref);
          }
          l += sum;
          // P_g overwrites P_{g-1}: the tensor core must have consumed it
          if (g >= 1) {
            if (!warp_wait(smem_u32(&bars->pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          tmem_st16(pcol + wq * 16, pk);
          if (!p_zero) {
            for (int kk = 1; kk < 4; ++kk) tmem_st16(pcol + ((wq + kk) & 3) * 16, zeros);
          }
          p_zero = true;
        } else {
          uint32_t x[BN];
#pragma unroll
          for (int c = 0; c < BN / 32; ++c)
            tmem_ld32(tmem_addr(tbase, lane_base, C::kColS + sb * 128 + c * 32), x + c * 32);
          tmem_ld_wait();
          tc_fence_before();
          mbar_arrive(smem_u32(&bars->s_free[sb]));
          const int k0 = sch.index * BN;
          if (k0 + BN - 1 > w.t0) {
            const int end = min(w.t0 + lp, w.t_last) - k0 + 1;
#pragma unroll
            for (int c = 0; c < BN; ++c) x[c] = c < end ? x[c] : 0xff800000u;  // -inf
          }
          uint32_t pk[BN / 2];
          bool slow = __any_sync(0xffffffffu, m_ref == -INFINITY);
          if (!slow) {
            sum = exp_block<BN>(x, pk, sl, m_ref);
            slow = __any_sync(0xffffffffu, !(sum <= kSumBound));
          }
          if (slow) {
            if (!rescale(raw_max128(x) * sl, j)) {
              ok = false;
              break;
            }
            sum = exp_block<BN>(x, pk, sl, m_ref);
          }
          l += sum;
          if (g >= 1) {
            if (!warp_wait(smem_u32(&bars->pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < BN / 64; ++c) tmem_st32(pcol + c * 32, pk + c * 32);
          p_zero = false;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&bars->p_full[sb]));
      }
      if (!ok) break;
      const bool there = lp < w.npos && h_off < p.G;
      const int token = w.token + lp, head = w.hk * p.G + h_off;
      const int j0 = w.j0, j1 = w.j1, nb = w.nb;
      const bool cut = w.cut();
      if (cut && j0 == 0 && tid == 128)  // the tile's first block is here: the join begins at this CTA
        work_of(p.work, D).opened[blockIdx.x] = {w.token, w.hk, w.npos, sh.owner_of(w.next_at - 1) - (int)blockIdx.x + 1};
      opened |= cut && j0 == 0;
      const int64_t out = (int64_t)token * p.Hq + head;  // the row of o and lse
      const int b = w.b, hk = w.hk, t0 = w.t0;
      // The next tile's Q goes into TMEM now that every S product that used this one has
      // completed, so that its first products run during this tile's epilogue.
      more = advance(false);
      if (more && !copy_q(k + 1, w)) {
        ok = false;
        break;
      }
      if (!warp_wait(smem_u32(&bars->pv_done[(g - 1) & 1]), ((g - 1) >> 1) & 1, abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float r[D];
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        tmem_ld32(tmem_addr(tbase, lane_base, C::kColO + c * 32), reinterpret_cast<uint32_t*>(r) + c * 32);
      tmem_ld_wait();
      // (the next tile's first P V, which overwrites O, follows this warp's next p_full)
      tc_fence_before();
      if (*(volatile int*)&bars->poison[k & 7] == k + 1 && there) {
        // infinities or NaN were taken out of V rows that not all queries see: this
        // row's own are added, found again in global memory
        Sched again(p.n_depth, nb, j0);
        auto add = [&](int c0, uint4 y) {  // 8 elements of a row of V
          const uint32_t e[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int cc = 0; cc < D; cc += 8)
            if (cc == c0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t f = not_finite(e[i]);
                if (f & 0x8000u) r[cc + 2 * i] += __uint_as_float(e[i] << 16);
                if (f & 0x80000000u) r[cc + 2 * i + 1] += __uint_as_float(e[i] & 0xffff0000u);
              }
            }
        };
#pragma unroll 1
        for (int j = j0; j < j1; ++j) {
          again.next(p.n_depth, nb);
          if (again.depth) {
            const int l_end = min(p.L, (again.index + 1) * SP);
#pragma unroll 1
            for (int slot = again.index * SP; slot < l_end; ++slot) {
              const uint4* v = reinterpret_cast<const uint4*>(p.vd + (int64_t)token * p.depth_tok +
                                                              (int64_t)hk * p.depth_hk + (int64_t)slot * p.depth_slot);
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) add(c * 8, v[c]);
            }
          } else if (again.index * BN + BN - 1 > t0) {
            const int k_end = min(t0 + lp + 1, (again.index + 1) * BN);
#pragma unroll 1
            for (int key = again.index * BN; key < k_end; ++key) {
              int pg = p.table[(int64_t)b * p.max_pages + (key >> p.page_shift)];
              if (pg < 0 || pg >= p.num_pages) pg = 0;
              const int64_t vr = ((int64_t)(pg * p.Hk + hk) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) {
                uint4 y;
                if constexpr (MX4) {
                  uint32_t mul, mul2, z[4];
                  factors(p.v_scale[vr * (D / 32) + (c >> 2)], mul, mul2);
                  unpack8(*reinterpret_cast<const uint32_t*>(p.v + vr * (D / 2) + c * 4), mul, mul2, z);
                  y = make_uint4(z[0], z[1], z[2], z[3]);
                } else {
                  y = *reinterpret_cast<const uint4*>(p.v + (vr * D + c * 8) * 2);
                }
                add(c * 8, y);
              }
            }
          }
        }
      }
      if (cut) {
        const int64_t slot = 2 * (int64_t)blockIdx.x + (j0 > 0 ? 0 : 1);
        const Work wk = work_of(p.work, D);
        if (there) {
          float4* po = reinterpret_cast<float4*>(wk.o + (slot * kRows + row) * D);
#pragma unroll
          for (int i = 0; i < D / 4; ++i) po[i] = make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          *reinterpret_cast<float2*>(wk.ml + (slot * kRows + row) * 2) = make_float2(m_ref, l);
        }
      } else if (there) {
        const float inv = 1.f / l;
        uint4* po = reinterpret_cast<uint4*>(p.o + out * D);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          po[i] = make_uint4(pack_bf16x2(r[8 * i] * inv, r[8 * i + 1] * inv),
                             pack_bf16x2(r[8 * i + 2] * inv, r[8 * i + 3] * inv),
                             pack_bf16x2(r[8 * i + 4] * inv, r[8 * i + 5] * inv),
                             pack_bf16x2(r[8 * i + 6] * inv, r[8 * i + 7] * inv));
        if (p.lse) p.lse[out] = (m_ref + log2f(l)) * kLn2;
      }
    }
    if (tid == 128 && !opened) work_of(p.work, D).opened[blockIdx.x] = {0, 0, 0, 0};
  } else {
    // ----------------------------- 4-bit pages unpacked, V blocks made harmless
    const int hw = warp - 8, r = tid - 256;  // a row of the tile each
    int g = 0;
    uint32_t checks = 0;  // bf16: parities of v_check
    bool ok = true;
    Walk w;
    w.begin(p, sh);
    for (int k = 0; ok && w.next(p, sh); ++k) {
      Sched sch(p.n_depth, w.nb, w.j0);
      for (int j = w.j0; j < w.j1; ++j, ++g) {
        sch.next(p.n_depth, w.nb);
        const bool part = partly_seen(w, sch);
        if (!MX4 && !part) continue;
        const int s = g % NS, f = g % NR;
        uint8_t* vt = smem + C::kOffV + s * C::kTileBytes;
        // rows that some query of the tile sees
        auto counts = [&](int x) -> bool {
          if (!sch.depth) return sch.index * BN + x <= w.t_last;
          return (x >> 5) * PW + (x & (PW - 1)) < w.npos && sch.index * SP + (x & 31) / PW < p.L;
        };
        bool found = false;
        if constexpr (MX4) {
          const uint8_t* rk = smem + C::kOffRawK + f * C::kRawBytes;
          const uint8_t* rv = smem + C::kOffRawV + f * C::kRawBytes;
          if (!warp_wait(smem_u32(&bars->raw_k_full[f]), (g / NR) & 1, abort)) { ok = false; break; }
          if (!sch.depth) {
            if (!warp_wait(smem_u32(&bars->k_empty[s]), ((g / NS) & 1) ^ 1, abort)) { ok = false; break; }
            unpack_tile<D, false>(rk, smem + C::kOffK + s * C::kTileBytes, hw, lane, counts);
          }
          fence_async();
          mbar_arrive(smem_u32(&bars->k_full[s]));
          mbar_arrive(smem_u32(&bars->raw_k_empty[f]));
          if (!warp_wait(smem_u32(&bars->raw_v_full[f]), (g / NR) & 1, abort)) { ok = false; break; }
          if (sch.depth) {
            found = tame_row<D>(vt, r, counts(r));
          } else {
            if (!warp_wait(smem_u32(&bars->v_empty[s]), ((g / NS) & 1) ^ 1, abort)) { ok = false; break; }
            if (part)
              found = unpack_tile<D, true>(rv, vt, hw, lane, counts);
            else
              unpack_tile<D, false>(rv, vt, hw, lane, counts);
          }
        } else {
          if (!warp_wait(smem_u32(&bars->v_check[s]), (checks >> s) & 1, abort)) { ok = false; break; }
          checks ^= 1u << s;
          found = tame_row<D>(vt, r, counts(r));
        }
        if (found) {
          *(volatile int*)&bars->poison[k & 7] = k + 1;
          __threadfence_block();
        }
        fence_async();
        mbar_arrive(smem_u32(MX4 ? &bars->v_full[s] : &bars->v_ready[s]));
        if (MX4) mbar_arrive(smem_u32(&bars->raw_v_empty[f]));
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
constexpr int kJoinWarps = 8, kJoinParts = 4;  // warps of a CTA, CTAs of a tile

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
    const float inv = 1.f / L;
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
  p.n_depth = (PW * a.L + 31) / 32;
  p.scale_log2 = a.scale * kLog2e;
  p.o = (__nv_bfloat16*)a.o; p.lse = a.lse; p.work = a.work; p.err = c.err;
  p.k = (const uint8_t*)c.k; p.v = (const uint8_t*)c.v;
  p.k_scale = (const uint8_t*)c.k_scale; p.v_scale = (const uint8_t*)c.v_scale;
  p.vd = (const __nv_bfloat16*)a.vd;
  p.depth_tok = a.depth_tok_stride; p.depth_hk = a.depth_hk_stride; p.depth_slot = a.depth_slot_stride;
  const int grid = a.num_sms < kMaxCtas ? a.num_sms : kMaxCtas;
  cudaError_t e = cudaFuncSetAttribute(prefill_paged_kernel<D, MX4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmemBytes);
  if (e != cudaSuccess) return e;
  e = paged::launch_dependent(prefill_paged_kernel<D, MX4>, dim3(grid), kThreads, C::kSmemBytes, stream, tq, tk, tv,
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
