// MoDA decode for a batch over the paged KV cache in bf16: the new token of
// every sequence attends, under one softmax, to the rows of its pages and to
// its L depth slots. decode_paged.cuh has the division of the work;
// decode_paged_mx4.cu is the kernel for 4-bit pages.
//
// HBM-bound: every cached row is read once for the G query heads of its KV
// head. A CTA is a producer warp and four consumer warps around a ring of
// shared-memory stages of 64 rows (or depth slots), K and V: the producer
// looks up pages and issues TMA copies, each consumer warp scores 16 of a
// stage's keys. Products are transposed (S^T = K Q^T with the keys as the rows
// of the A tile, then O^T += V^T P^T), so that the G heads fill the 8 columns
// of a warp MMA's B tile; G > 8 takes two such tiles. Two CTAs an SM keep up to
// 192 KB on the way. Measured (d = 128): 48 ragged sequences of up to 16384
// rows, 803 MB, 121 us (99 % of the copy bandwidth); one context of 65536 rows
// 26.4 us, of which its 134 MB take 20, the look-ups before them 2.7, the join 3;
// one of 701 rows, in clusters of eight, 4.5 us.
#include "decode_paged.cuh"
#include "tensor_map.h"

namespace moda {
namespace paged {
namespace {

constexpr int kCW = 4;                // consumer warps
constexpr int kWarps = kCW + 1;       // and the producer
constexpr int kKeys = 64;             // cached rows, or depth slots, of a unit
constexpr int kCols = 64;             // columns of O merged at a time
template <int D, int NT>
constexpr int kCost = D == 128 && NT == 1 ? 1 : 2;  // entering and leaving a segment, in units
constexpr int kCtasPerSm = 2;
constexpr int kGroupUnits = 8, kClusterUnits = 3;  // see group_of
constexpr float kSlack = 8.f;  // weights up to 2^8 lose nothing in bf16
constexpr uint64_t kTimeoutNs = 2000000000ull;

template <int D>
struct Smem {
  static constexpr int kNS = D == 128 ? 3 : 6;      // stages
  static constexpr int kTile = kKeys * D * 2;
  uint8_t ring[kNS][2][kTile];  // [stage][K or V], 1024-byte aligned
  MergeSmem<kCW, kCols> merge;
  uint64_t full[kNS], empty[kNS];
  ShareSmem<kWarps> share;
  int abort;
};

// 16 bf16 keys (rows row0.. of a tile of ROWS rows, `there` of them exist)
// into the state.
template <int D, int NT, int ROWS>
__device__ __forceinline__ void tile_bf16(State<D, NT>& st, const uint32_t (&qb)[NT][D / 16][2],
                                          uint32_t kb, uint32_t vb, int row0, int there,
                                          float scale_log2, int lane) {
  const int r0 = lane >> 2, c = lane & 3, lr = lane & 7, lm = lane >> 3;
  float s[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    uint32_t a[4];
    wmma16::ldsm_x4(kb + at_bf16<ROWS>(row0 + (lm & 1) * 8 + lr, ks * 16 + (lm >> 1) * 8), a[0], a[1],
                    a[2], a[3]);
#pragma unroll
    for (int t = 0; t < NT; ++t) wmma16::mma_bf16(s[t], a, qb[t][ks][0], qb[t][ks][1]);
  }
  const bool k0 = r0 < there, k1 = r0 + 8 < there;
  // P^T rounded to bf16, and what that left: a second product that the wait
  // for memory hides, for an o that is right to its own rounding
  uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s[t][0] = k0 ? s[t][0] * scale_log2 : -INFINITY;
    s[t][1] = k0 ? s[t][1] * scale_log2 : -INFINITY;
    s[t][2] = k1 ? s[t][2] * scale_log2 : -INFINITY;
    s[t][3] = k1 ? s[t][3] * scale_log2 : -INFINITY;
    st.template raise<4>(t, s[t], kSlack);
    float p[4];
    st.weigh(t, s[t], p);
    // P^T (rows = keys, columns = heads) transposed into the B tile
#pragma unroll
    for (int i = 0; i < 2; ++i) weights_bf16(p[2 * i], p[2 * i + 1], pb[t][i], pl[t][i]);
  }
  // rows that do not exist weigh 0, but 0 times what they hold may be NaN
  uint32_t lo = 0xffffffffu, hi = 0xffffffffu;
  if (there < 16) {
    lo = (2 * c < there ? 0xffffu : 0u) | (2 * c + 1 < there ? 0xffff0000u : 0u);
    hi = (2 * c + 8 < there ? 0xffffu : 0u) | (2 * c + 9 < there ? 0xffff0000u : 0u);
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t a[4];
    wmma16::ldsm_x4_t(vb + at_bf16<ROWS>(row0 + (lm >> 1) * 8 + lr, i * 16 + (lm & 1) * 8), a[0], a[1],
                      a[2], a[3]);
    if (there < 16) {
      a[0] &= lo; a[1] &= lo; a[2] &= hi; a[3] &= hi;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wmma16::mma_bf16(st.o[t][i], a, pb[t][0], pb[t][1]);
      wmma16::mma_bf16(st.o[t][i], a, pl[t][0], pl[t][1]);
    }
  }
}

template <int D, int NT, Split SPLIT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
decode_paged_split(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmKd, const __grid_constant__ CUtensorMap tmVd,
                   const __grid_constant__ Params p, int box) {
  using S = Smem<D>;
  constexpr int NS = S::kNS;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int depth_units = (p.L + kKeys - 1) / kKeys;
  const Work wk = work_of(p.work, p.G, D);

  if (tid == 0) {
    sm.abort = 0;
    for (int s = 0; s < NS; ++s) {
      sm103::mbar_init(sm103::smem_u32(&sm.full[s]), 1);
      sm103::mbar_init(sm103::smem_u32(&sm.empty[s]), kCW);
    }
    sm103::fence_barrier_init();
  }
  wait_for_stream();
  constexpr bool GROUP = SPLIT == Split::kGroup;
  Share<kKeys> sh;
  __syncthreads();
  if constexpr (GROUP) {
    sh = share_of_segment<kKeys>(p, depth_units);
    if (sh.at.n == 0) return write_empty_segment<D>(p, sh.at.b, sh.at.hk);
  } else {
    if constexpr (SPLIT == Split::kOne)
      sh = share_of_one<kKeys, kCost<D, NT>, 1>(p, depth_units);
    else
      sh = share_of<kKeys, kWarps, kCost<D, NT>, 1>(p, depth_units, sm.share);
    if (depth_units == 0) write_empty<D>(p);
    if (sh.n == 0) {
      if (tid == 0) wk.opened[blockIdx.x] = make_int2(-1, 0);
      return;
    }
  }
  Place<kKeys> at = sh.at;
  GroupSmem<D, kCW>& last = *reinterpret_cast<GroupSmem<D, kCW>*>(sm.ring);  // when the ring is free
  static_assert(sizeof(GroupSmem<D, kCW>) <= sizeof(sm.ring));
  const int64_t first_row = ((int64_t)at.b * p.Hk + at.hk) * p.G;

  if (warp == kCW) {
    // ------------------------------------------------------------ producer
    // One page row block per lane; the next unit's pages are looked up before
    // the wait for a free stage.
    auto page_of = [&](const Place<kKeys>& x) -> int {
      if (x.off < depth_units) return 0;
      const int key = (x.off - depth_units) * kKeys + lane * box;
      if (lane * box >= kKeys || key >= x.len) return 0;
      return *(p.table + (int64_t)x.b * p.max_pages + (key >> p.page_shift));
    };
    const int n = sh.n;
    int page = page_of(at);
    for (int k = 0; k < n; ++k) {
      const Place<kKeys> cur = at;
      int pg = page;
      if (k + 1 < n) {
        if (++at.off == at.n) at.next_segment(p, depth_units);
        page = page_of(at);
      }
      const int s = k % NS;
      const uint32_t bar = sm103::smem_u32(&sm.full[s]);
      if (k >= NS)
        sm103::mbar_wait_bounded(sm103::smem_u32(&sm.empty[s]), (uint32_t)((k / NS - 1) & 1), &sm.abort,
                                 kTimeoutNs);
      if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) break;
      const uint32_t kt = sm103::smem_u32(&sm.ring[s][0][0]), vt = sm103::smem_u32(&sm.ring[s][1][0]);
      if (cur.off < depth_units) {
        if (lane == 0) {
          constexpr uint32_t kBox = kKeys * 128;  // 64 columns
          sm103::mbar_arrive_expect_tx(bar, 2 * (D / 64) * kBox);
          const int l = cur.off * kKeys;
          const int2 of = depth_of(p, cur.b, cur.hk);
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            sm103::tma_load_4d(kt + x * kBox, &tmKd, bar, x * 64, l, of.y, of.x);
            sm103::tma_load_4d(vt + x * kBox, &tmVd, bar, x * 64, l, of.y, of.x);
          }
        }
      } else {
        const int key0 = (cur.off - depth_units) * kKeys;
        const int boxes = (min(kKeys, cur.len - key0) + box - 1) / box;
        const uint32_t box_bytes = (uint32_t)box * (D * 4);  // K and V
        if (lane == 0) sm103::mbar_arrive_expect_tx(bar, boxes * box_bytes);
        __syncwarp();
        if (lane < boxes) {
          if (pg < 0 || pg >= p.num_pages) {
            atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
            pg = 0;
          }
          const int row = (key0 + lane * box) & ((1 << p.page_shift) - 1);
          const int head = pg * p.Hk + cur.hk;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            const uint32_t off = x * (kKeys * 128) + lane * box * 128;
            sm103::tma_load_3d(kt + off, &tmK, bar, x * 64, row, head);
            sm103::tma_load_3d(vt + off, &tmV, bar, x * 64, row, head);
          }
        }
      }
    }
    if (*(volatile int*)&sm.abort && lane == 0) {
      // a wait gave up: let every stage's copies land before the CTA goes
      for (int s = 0; s < NS && s < n; ++s)
        for (uint32_t ph = 0; ph < 2; ++ph) {
          int never = 0;
          sm103::mbar_wait_bounded(sm103::smem_u32(&sm.full[s]), ph, &never, kTimeoutNs / 100);
        }
      atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_TIMEOUT);
    }
    if constexpr (GROUP) {
      __syncwarp();
      if (p.group > 1) join_group<D, kCW>(p, last, first_row);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // After a wait that gave up the warps go through the same steps, without the
  // arithmetic, so that they meet at the same barriers.
  const int r0 = lane >> 2;
  State<D, NT> st;
  int k = 0, left = sh.n;
  bool opened = false;
  long long seg_end = sh.end;
  while (GROUP || left > 0) {  // (a group's CTA leaves a state even if it has no unit)
    const int cnt = min(left, at.n - at.off);
    const int end = at.off + cnt;
    const bool cut_before = at.off > 0, cut_after = end < at.n;
    const __nv_bfloat16* q = p.q + ((int64_t)at.b * p.Hk + at.hk) * p.G * D;
    st.clear();
    int off = at.off;
    auto take = [&](int s) {
      return __all_sync(0xffffffffu,
                        sm103::mbar_wait_bounded(sm103::smem_u32(&sm.full[s]), (uint32_t)((k / NS) & 1),
                                                 &sm.abort, kTimeoutNs));
    };
    auto give = [&](int s) {
      __syncwarp();
      if (lane == 0) sm103::mbar_arrive(sm103::smem_u32(&sm.empty[s]));
      ++k;
    };
    uint32_t qb[NT][D / 16][2];
    load_q_bf16<D, NT>(qb, q, p.G, lane);
    for (; off < end; ++off) {
      const int s = k % NS;
      const bool ok = take(s);
      const int there = (off < depth_units ? p.L - off * kKeys
                                           : at.len - (off - depth_units) * kKeys) - warp * 16;
      if (ok && there > 0)
        tile_bf16<D, NT, kKeys>(st, qb, sm103::smem_u32(&sm.ring[s][0][0]),
                                sm103::smem_u32(&sm.ring[s][1][0]), warp * 16, there, p.scale_log2,
                                lane);
      give(s);
    }
    const auto put = [&](float* m0, float* m1, int t, int part, const auto& buf) {
      constexpr int kTiles = std::remove_reference_t<decltype(buf)>::kCols / 16;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        const float(&x)[4] = st.o[t][part * kTiles + i];
        m0[i * 16 + r0] = x[0];
        m1[i * 16 + r0] = x[1];
        m0[i * 16 + r0 + 8] = x[2];
        m1[i * 16 + r0 + 8] = x[3];
      }
    };
    if constexpr (GROUP) {
      leave<D, NT>(p, last.merge, st, p.group > 1, &last.o[0][0], &last.ml[0][0], 0, first_row, put);
      break;
    }
    const int slot = 2 * blockIdx.x + (cut_before ? 0 : 1);
    const int64_t row0 = ((int64_t)at.b * p.Hk + at.hk) * p.G;
    if (left == cnt)  // the last: the ring is free
      leave<D, NT>(p, last.merge, st, cut_before || cut_after, wk.o, wk.ml, slot, row0, put);
    else
      leave<D, NT>(p, sm.merge, st, cut_before || cut_after, wk.o, wk.ml, slot, row0, put);
    if (cut_after && !cut_before) {
      opened = true;
      if (tid == 0)
        wk.opened[blockIdx.x] =
            make_int2(at.b * p.Hk + at.hk, sh.owner_of(seg_end - 1) - (int)blockIdx.x + 1);
    }
    left -= cnt;
    if (left > 0) {
      at.next_segment(p, depth_units);
      seg_end += kCost<D, NT> + at.n;
    }
  }
  if constexpr (GROUP) {
    if (p.group > 1) join_group<D, kCW>(p, last, first_row);
  }
  if (tid == 0) {
    if (!GROUP && !opened) wk.opened[blockIdx.x] = make_int2(-1, 0);
    if (sm.abort) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_TIMEOUT);
  }
}

// Joining the partials, where segments have few of them: a warp for each split
// CTA (the segment that it opened) and head, all of its partials' loads in
// flight at once, a lane D/32 columns. Few small CTAs, because they have to be
// brought up when the split kernel has ended.
constexpr int kFewWarps = 8;

template <int D>
__global__ void __launch_bounds__(kFewWarps * 32)
decode_paged_join_few(float* work, int G, int shares, float unit, __nv_bfloat16* o, float* lse) {
  constexpr int E = D / 32;
  constexpr int U = 4;
  const Work wk = work_of(work, G, D);
  const int lane = threadIdx.x & 31;
  const int stride = gridDim.x * kFewWarps;
  wait_for_stream();
  for (int item = blockIdx.x * kFewWarps + (threadIdx.x >> 5); item < shares * G; item += stride) {
    const int opener = item / G, g = item - opener * G;
    const int2 seg = wk.opened[opener];
    if (seg.x < 0) continue;
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < seg.y; i0 += U) {
      float pm[U], pl[U], po[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u;
        pm[u] = -INFINITY;
        pl[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) po[u][e] = 0.f;
        if (i < seg.y) {
          const int64_t row = (int64_t)(2 * (opener + i) + (i == 0 ? 1 : 0)) * G + g;
          pm[u] = wk.ml[row * 2];
          pl[u] = wk.ml[row * 2 + 1];
#pragma unroll
          for (int e = 0; e < E; ++e) po[u][e] = wk.o[row * D + lane * E + e];
        }
      }
      add_partials<U, E>(M, L, acc, pm, pl, po);
    }
    const int64_t r = (int64_t)seg.x * G + g;
    const float inv = 1.f / L * unit;
#pragma unroll
    for (int e = 0; e < E; ++e) o[r * D + lane * E + e] = __float2bfloat16_rn(acc[e] * inv);
    if (lane == 0 && lse) lse[r] = (M + log2f(L)) * kLn2;
  }
}

// And where they have many: a CTA for each segment (blockIdx.x) and head
// (blockIdx.y), which looks among the `shares` split CTAs for the one that
// opened the segment; its 16 warps take the partials in turn.
constexpr int kManyWarps = 16;

template <int D>
__global__ void __launch_bounds__(kManyWarps * 32)
decode_paged_join_many(float* work, int G, int shares, float unit, __nv_bfloat16* o, float* lse) {
  constexpr int E = D / 32;
  constexpr int U = 8;  // partials a warp loads before it adds the first
  __shared__ float sm_o[kManyWarps][D];
  __shared__ float sm_ml[kManyWarps][2];
  __shared__ int sm_opener, sm_parts;
  const Work wk = work_of(work, G, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y;
  if (threadIdx.x == 0) sm_opener = -1;
  __syncthreads();
  wait_for_stream();
  for (int i = threadIdx.x; i < shares; i += kManyWarps * 32) {
    const int2 x = wk.opened[i];
    if (x.x == (int)blockIdx.x) {
      sm_opener = i;
      sm_parts = x.y;
    }
  }
  __syncthreads();
  const int opener = sm_opener, parts = sm_parts;
  if (opener < 0) return;
  float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = warp; i0 < parts; i0 += kManyWarps * U) {
    float pm[U], pl[U], po[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kManyWarps;
      pm[u] = -INFINITY;
      pl[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) po[u][e] = 0.f;
      if (i < parts) {
        const int64_t row = (int64_t)(2 * (opener + i) + (i == 0 ? 1 : 0)) * G + g;
        pm[u] = wk.ml[row * 2];
        pl[u] = wk.ml[row * 2 + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) po[u][e] = wk.o[row * D + e * 32 + lane];
      }
    }
    add_partials<U, E>(M, L, acc, pm, pl, po);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][e * 32 + lane] = acc[e];
  if (lane == 0) {
    sm_ml[warp][0] = M;
    sm_ml[warp][1] = L;
  }
  __syncthreads();
  if (warp < E) {  // 32 columns a warp; each lane first weighs one state
    float m = lane < kManyWarps ? sm_ml[lane][0] : -INFINITY, l = lane < kManyWarps ? sm_ml[lane][1] : 0.f;
    float Mt = m;
#pragma unroll
    for (int sh = 1; sh < kManyWarps; sh <<= 1) Mt = fmaxf(Mt, __shfl_xor_sync(0xffffffffu, Mt, sh));
    Mt = __shfl_sync(0xffffffffu, Mt, 0);
    const float a = m == -INFINITY ? 1.f : sm103::ex2_approx(m - Mt);
    l *= a;
#pragma unroll
    for (int sh = 1; sh < kManyWarps; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
    l = __shfl_sync(0xffffffffu, l, 0);
    const int d = threadIdx.x;
    float ot = 0.f;
#pragma unroll
    for (int w = 0; w < kManyWarps; ++w) ot = fmaf(__shfl_sync(0xffffffffu, a, w), sm_o[w][d], ot);
    const int64_t r = (int64_t)blockIdx.x * G + g;
    o[r * D + d] = __float2bfloat16_rn(ot / l * unit);
    if (d == 0 && lse) lse[r] = (Mt + log2f(l)) * kLn2;
  }
}

template <int D, int NT>
cudaError_t launch(const DecodePagedArgs& a, cudaStream_t stream) {
  const PagedKv& c = a.c;
  const int box = c.page_size < kKeys ? c.page_size : kKeys;  // page rows of one copy
  // pages as [num_pages * Hk][page_size][D]; depth slots as [B][Hk][L][D]
  CUtensorMap tk, tv, tkd, tvd;
  {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)c.page_size, (uint64_t)c.num_pages * c.Hk};
    const uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)D * 2 * c.page_size};
    const uint32_t bx[3] = {64, (uint32_t)box, 1};
    if (encode_bf16_sw128(&tk, c.k, 3, dims, str, bx) != CUDA_SUCCESS ||
        encode_bf16_sw128(&tv, c.v, 3, dims, str, bx) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (a.L > 0) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.L, (uint64_t)c.Hk * a.fold, (uint64_t)c.B / a.fold};
    const uint64_t str[3] = {(uint64_t)a.depth_slot_stride * 2, (uint64_t)a.depth_hk_stride * 2,
                             (uint64_t)a.depth_b_stride * 2};
    const uint32_t bx[4] = {64, (uint32_t)kKeys, 1, 1};
    if (encode_bf16_sw128(&tkd, a.kd, 4, dims, str, bx) != CUDA_SUCCESS ||
        encode_bf16_sw128(&tvd, a.vd, 4, dims, str, bx) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  } else {
    tkd = tk;  // never read when L == 0
    tvd = tv;
  }
  const size_t smem = sizeof(Smem<D>) + 1024;
  int grid = a.num_sms * kCtasPerSm;
  grid = grid < kMaxCtas ? grid : kMaxCtas;
  const int max_units = (a.L + kKeys - 1) / kKeys + (c.max_pages * c.page_size + kKeys - 1) / kKeys;
  const int group = group_of(a, max_units, grid, kGroupUnits, kClusterUnits);
  const auto kernel = group        ? decode_paged_split<D, NT, Split::kGroup>
                      : c.B == 1 ? decode_paged_split<D, NT, Split::kOne>
                                 : decode_paged_split<D, NT, Split::kShares>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (group > 8) {  // beyond the portable size
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (group)
    return launch_dependent_clusters(kernel, dim3(c.B * c.Hk * group), group, kWarps * 32, smem, stream, tk, tv,
                                     tkd, tvd, params_of(a, group), box);
  e = launch_dependent(kernel, dim3(grid), kWarps * 32, smem, stream, tk, tv, tkd, tvd, params_of(a, 0), box);
  return e != cudaSuccess ? e : launch_join(a, grid, stream);
}

}  // namespace

cudaError_t launch_join(const DecodePagedArgs& a, int shares, cudaStream_t stream) {
  // Many partials: eight a segment and more, while a CTA for each segment and
  // head fits the SMs at once.
  const int64_t segments = (int64_t)a.c.B * a.c.Hk;
  __nv_bfloat16* o = (__nv_bfloat16*)a.o;
  if (segments * 8 <= shares && segments * a.G <= a.num_sms * 4)
    return launch_dependent(a.c.d == 128 ? decode_paged_join_many<128> : decode_paged_join_many<64>,
                            dim3((unsigned)segments, a.G), kManyWarps * 32, 0, stream, a.work, a.G, shares,
                            unit_of(a), o, a.lse);
  const int ctas = (shares * a.G + kFewWarps - 1) / kFewWarps;
  return launch_dependent(a.c.d == 128 ? decode_paged_join_few<128> : decode_paged_join_few<64>,
                          dim3(ctas < 4 * a.num_sms ? ctas : 4 * a.num_sms), kFewWarps * 32, 0, stream, a.work,
                          a.G, shares, unit_of(a), o, a.lse);
}

}  // namespace paged

size_t decode_paged_workspace_bytes(int Hq, int Hk, int d) {
  const int64_t G = Hq / Hk;
  return (size_t)(2 * paged::kMaxCtas + 2 * paged::kMaxCtas * G * (d + 2)) * sizeof(float);
}

cudaError_t launch_decode_paged(const DecodePagedArgs& a, cudaStream_t stream) {
  if (a.c.format == MODA_KV_MX4) return paged::launch_mx4(a, stream);
  if (a.c.d == 128)
    return a.G <= 8 ? paged::launch<128, 1>(a, stream) : paged::launch<128, 2>(a, stream);
  return a.G <= 8 ? paged::launch<64, 1>(a, stream) : paged::launch<64, 2>(a, stream);
}

}  // namespace moda
