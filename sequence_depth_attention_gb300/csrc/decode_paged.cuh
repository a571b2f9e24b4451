// What the two paged decode kernels (bf16 pages, 4-bit pages) share: the line
// of units and its division over the CTAs, a warp's softmax state, and the way
// a segment's result leaves a CTA.
//
// The batch is cut into units (some rows of one KV head of one sequence, or
// some of its depth slots), all units of the batch lie in one line, and CTA i
// of P takes the i-th P-th of them, whatever sequences it crosses: each CTA
// streams the same number of bytes, for one long context as for a ragged
// batch, and the lengths stay on the device. The units of one (sequence, KV
// head) are a segment. A segment inside one CTA's share is written out there;
// one that is cut leaves a partial state (m, l, unnormalised o) per CTA, and a
// dependent kernel joins them.
//
// A short batch needs none of that: each segment gets a group of 1 to 16 CTAs, a
// cluster, which looks up nothing but its own length and joins its partials
// from shared memory to shared memory, in one launch (group_of).
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "moda_internal.h"
#include "sm103.cuh"
#include "warp_mma.cuh"

namespace moda {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCtas = 608;  // four per SM of 152; sizes the workspace

// The workspace: for each CTA the segment that it opens and does not finish
// (-1: none) with the number of its partials, and the partials of CTA i: slot
// 2i for a segment opened by an earlier CTA, 2i + 1 for the one that it opens.
struct Work {
  int2* opened;
  float* o;   // [2 * kMaxCtas][G][D]
  float* ml;  // [2 * kMaxCtas][G][2]
};
__host__ __device__ inline Work work_of(float* w, int G, int D) {
  Work k;
  k.opened = reinterpret_cast<int2*>(w);
  k.o = w + 2 * kMaxCtas;
  k.ml = k.o + (int64_t)2 * kMaxCtas * G * D;
  return k;
}

// How a batch is divided: into equal shares of the line, that of one sequence,
// or a group of CTAs for each segment.
enum class Split { kShares, kOne, kGroup };

struct Params {
  const __nv_bfloat16* q;
  const int* lens;
  const int* table;
  int num_pages, page_shift, max_pages, B, Hk, G, L;  // pages of 1 << page_shift rows
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  float* work;
  unsigned int* err;
  int group;   // CTAs of a segment; 0: shares of the line
  float unit;  // of the sums O that warps merge and CTAs leave, see unit_of
};
// O of 4-bit rows leaves a warp in units of 2^32: values are up to 1.5 * 2^127, and
// sums of up to 2^24 of them, each times a weight of up to 2^8, stay finite; what
// fp32 drops at the low end is below 2^-117.
constexpr float kUnit4 = 0x1p32f;
inline float unit_of(const DecodePagedArgs& a) { return a.c.format == MODA_KV_MX4 ? kUnit4 : 1.f; }
inline Params params_of(const DecodePagedArgs& a, int group) {
  const PagedKv& c = a.c;
  return {(const __nv_bfloat16*)a.q, a.seq_lens, c.table, c.num_pages, __builtin_ctz((unsigned)c.page_size),
          c.max_pages, c.B, c.Hk, a.G, a.L, a.scale * kLog2e, (__nv_bfloat16*)a.o, a.lse, a.work, c.err, group,
          unit_of(a)};
}

// Sequence b's rows, within what its table can name.
__device__ __forceinline__ int rows_of(const Params& p, int b) {
  return min(max(p.lens[b], 0), p.max_pages << p.page_shift);
}

// A place in the line of units: depth units first, then units of KEYS rows.
template <int KEYS>
struct Place {
  int b, hk, off, n, len;  // unit off of the n units of segment (b, hk); len rows
  __device__ __forceinline__ void enter(const Params& p, int depth_units) {
    len = rows_of(p, b);
    n = depth_units + (len + KEYS - 1) / KEYS;
  }
  // the first unit of the next segment that has any; only where there is one
  __device__ __forceinline__ void next_segment(const Params& p, int depth_units) {
    off = 0;
    if (++hk < p.Hk) return;
    hk = 0;
    do {
      ++b;
      enter(p, depth_units);
    } while (n == 0);
  }
};

// a / b for what are almost always small numbers
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// A CTA's share of the line, and the place it begins at. Entering and leaving
// a segment costs about as much as `cost` of its units, so the line that is
// divided has that many more in front of each segment ("points"): the first
// `rem` of the `shares` CTAs that have any take base + 1 points, the others
// base, and a CTA works on the units among its points.
template <int KEYS>
struct Share {
  long long total, base;  // points
  int shares, rem;
  long long end;  // the point behind the segment that it begins in
  int n;          // units of this CTA
  Place<KEYS> at;

  // `total` points over the grid's CTAs, `least` for each at least
  __device__ __forceinline__ void divide_line(int least) {
    shares = (int)min((long long)gridDim.x, divide(total + least - 1, least));
    base = n = rem = 0;
    if (shares > 0) {
      base = divide(total, shares);
      rem = (int)(total - base * shares);
    }
  }
  __device__ __forceinline__ long long first_point(int cta) const {
    return base * cta + min(cta, rem);
  }
  // the CTA that owns a point
  __device__ __forceinline__ int owner_of(long long point) const {
    const long long wide = (base + 1) * rem;  // points of the CTAs with base + 1
    return point < wide ? (int)divide(point, base + 1) : rem + (int)divide(point - wide, base);
  }
};
template <int WARPS>
struct ShareSmem {
  unsigned long long warp_sum[WARPS];
  int start[4];       // sequence, KV head, point of the segment, units
  long long units[2]; // of the line before the share's begin and before its end
};
// COST: see above. LEAST: points that are worth a CTA.
template <int KEYS, int WARPS, int COST, int LEAST>
__device__ __forceinline__ Share<KEYS> share_of(const Params& p, int depth_units,
                                                ShareSmem<WARPS>& sm) {
  constexpr int THREADS = WARPS * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The block table is needed as soon as the lengths are known: the grid asks
  // for it meanwhile, a line of 128 bytes a thread. (In all up to 6.2 MB in bf16, 7.5 MB
  // in 4 bits at three CTAs an SM; the table's whole width, whatever the lengths are.)
  {
    const int64_t line = (int64_t)blockIdx.x * THREADS + tid;
    if (line * 32 < (int64_t)p.B * p.max_pages)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + line * 32));
  }
  // Points of one KV head before each thread's run of sequences and in all
  // (below 2^37), and sequences that have any (at most 2^24), side by side.
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  auto units_of = [&](int b) { return depth_units + (rows_of(p, b) + KEYS - 1) / KEYS; };
  unsigned long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int raw = p.lens[b];
    if (raw < 0 || raw > p.max_pages << p.page_shift)
      atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
    const int n = units_of(b);
    if (n > 0) mine += ((unsigned long long)(n + COST) << 25) + 1;
  }
  unsigned long long before = mine;  // inclusive scan of the warp
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += x;
  }
  if (lane == 31) sm.warp_sum[warp] = before;
  if (tid == 0) sm.units[0] = sm.units[1] = -1;
  __syncthreads();
  unsigned long long all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sm.warp_sum[w];
    all += sm.warp_sum[w];
  }
  before -= mine;
  Share<KEYS> s;
  s.total = (long long)(all >> 25) * p.Hk;
  s.divide_line(LEAST);
  const int cta = blockIdx.x;
  if (cta < s.shares) {
    // where the share begins and ends, by the threads whose sequences these are
    const long long from = (long long)(before >> 25) * p.Hk, to = from + (long long)(mine >> 25) * p.Hk;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long point = s.first_point(cta + e);
      if (point < from || point >= to) continue;
      long long at = from, segments = (long long)(before & 0x1ffffff) * p.Hk;
      for (int b = b0; b < b1; ++b) {
        const int n = units_of(b);
        if (n == 0) continue;
        const int len = n + COST;
        if (point < at + (long long)len * p.Hk) {
          // (point - at) / len is below Hk, at most 4096: a float's quotient is
          // at most one off
          int hk = (int)((float)(point - at) / (float)len);
          int off = (int)(point - at - (long long)hk * len);
          if (off < 0) {
            --hk;
            off += len;
          } else if (off >= len) {
            ++hk;
            off -= len;
          }
          sm.units[e] = point - (segments + hk) * COST - min(off, COST);
          if (e == 0) {
            sm.start[0] = b;
            sm.start[1] = hk;
            sm.start[2] = off;
            sm.start[3] = n;
          }
          break;
        }
        at += (long long)len * p.Hk;
        segments += p.Hk;
      }
    }
  }
  __syncthreads();
  if (cta < s.shares) {
    const long long all_units = s.total - (long long)(all & 0x1ffffff) * p.Hk * COST;
    s.n = (int)((sm.units[1] < 0 ? all_units : sm.units[1]) - sm.units[0]);
    s.at.b = sm.start[0];
    s.at.hk = sm.start[1];
    s.at.off = max(0, sm.start[2] - COST);
    s.at.n = sm.start[3];
    s.at.len = rows_of(p, s.at.b);
    s.end = s.first_point(cta) - sm.start[2] + COST + s.at.n;
  }
  return s;
}

// The same for a single sequence, whose segments are all alike: no scan, no
// barrier (65536 rows: bf16 26.4 us instead of 27.2, 4-bit 15.6 instead of 16.2;
// as a branch of share_of it cost the others 0.7 %).
template <int KEYS, int COST, int LEAST>
__device__ __forceinline__ Share<KEYS> share_of_one(const Params& p, int depth_units) {
  const int cta = blockIdx.x, raw = p.lens[0];
  Share<KEYS> s;
  s.at.b = 0;
  s.at.enter(p, depth_units);
  if (cta == 0 && threadIdx.x == 0 && (raw < 0 || raw > p.max_pages << p.page_shift))
    atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
  const int len = s.at.n + COST;
  s.total = s.at.n > 0 ? (long long)len * p.Hk : 0;
  s.divide_line(LEAST);
  if (cta < s.shares) {
    const long long from = s.first_point(cta), to = s.first_point(cta + 1);
    s.at.hk = (int)divide(from, len);
    const int hk_to = (int)divide(to, len);
    const int off = (int)(from - (long long)s.at.hk * len), off_to = (int)(to - (long long)hk_to * len);
    s.at.off = max(0, off - COST);
    s.n = (int)(to - from) - (hk_to - s.at.hk) * COST + min(off, COST) - min(off_to, COST);
    s.end = from - off + len;
  }
  return s;
}

// Short batches: `group` CTAs, a cluster, for each segment, and this one's part
// of its units (perhaps none; at.n == 0 when the segment has none).
template <int KEYS>
__device__ __forceinline__ Share<KEYS> share_of_segment(const Params& p, int depth_units) {
  const int segment = blockIdx.x / p.group, rank = blockIdx.x - segment * p.group;
  Share<KEYS> s;
  s.at.b = segment / p.Hk;
  s.at.hk = segment - s.at.b * p.Hk;
  s.at.enter(p, depth_units);
  const int raw = p.lens[s.at.b];
  if (rank == 0 && s.at.hk == 0 && threadIdx.x == 0 && (raw < 0 || raw > p.max_pages << p.page_shift))
    atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
  s.at.off = s.at.n * rank / p.group;
  s.n = s.at.n * (rank + 1) / p.group - s.at.off;
  return s;
}

// o = 0 and lse = -infinity for the sequences with nothing to attend to.
template <int D>
__device__ __forceinline__ void write_empty(const Params& p) {
  const int Hq = p.Hk * p.G;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (rows_of(p, b) != 0) continue;
    uint32_t* o = reinterpret_cast<uint32_t*>(p.o + (int64_t)b * Hq * D);
    for (int i = threadIdx.x; i < Hq * D / 2; i += blockDim.x) o[i] = 0u;
    if (p.lse)
      for (int i = threadIdx.x; i < Hq; i += blockDim.x) p.lse[(int64_t)b * Hq + i] = -INFINITY;
  }
}

// The same for one segment, by the first CTA of its group.
template <int D>
__device__ __forceinline__ void write_empty_segment(const Params& p, int b, int hk) {
  if (blockIdx.x % p.group != 0) return;
  const int64_t row = ((int64_t)b * p.Hk + hk) * p.G;
  uint32_t* o = reinterpret_cast<uint32_t*>(p.o + row * D);
  for (int i = threadIdx.x; i < p.G * D / 2; i += blockDim.x) o[i] = 0u;
  if (p.lse)
    for (int i = threadIdx.x; i < p.G; i += blockDim.x) p.lse[row + i] = -INFINITY;
}

// Byte offset of (row, col) in a bf16 tile of ROWS rows: 64-column boxes,
// 16-byte chunks XORed with the row's low bits (the 128-byte TMA swizzle).
template <int ROWS>
__device__ __forceinline__ uint32_t at_bf16(int row, int col) {
  return (uint32_t)((col >> 6) * (ROWS * 128) + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) +
                    ((col & 7) << 1));
}

// One warp's softmax state of a segment: for head pair (2c, 2c + 1) of each
// 8-head tile the running maximum m (log2 units), this lane's share of the
// sum l, and O^T.
template <int D, int NT>
struct State {
  float m[NT][2], l[NT][2];
  float o[NT][D / 16][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }
  }
  // Raises m of tile t to cover z, N scores of head 2c at even and 2c + 1 at odd
  // places, and brings l and o to it. Only when one of them is more than `slack`
  // above m, which most tiles' are not: one vote tells.
  template <int N>
  __device__ __forceinline__ void raise(int t, const float (&z)[N], float slack) {
    float x0 = z[0], x1 = z[1];
#pragma unroll
    for (int i = 2; i < N; i += 2) {
      x0 = fmaxf(x0, z[i]);
      x1 = fmaxf(x1, z[i + 1]);
    }
    if (!__any_sync(0xffffffffu, x0 > m[t][0] + slack || x1 > m[t][1] + slack)) return;
    x0 = fmaxf(x0, m[t][0]);
    x1 = fmaxf(x1, m[t][1]);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
    }
    const float a0 = m[t][0] == x0 ? 1.f : sm103::ex2_approx(m[t][0] - x0);
    const float a1 = m[t][1] == x1 ? 1.f : sm103::ex2_approx(m[t][1] - x1);
    m[t][0] = x0;
    m[t][1] = x1;
    l[t][0] *= a0;
    l[t][1] *= a1;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      o[t][i][0] *= a0; o[t][i][1] *= a1; o[t][i][2] *= a0; o[t][i][3] *= a1;
    }
  }
  // p = 2^(s - m), added to l
  __device__ __forceinline__ void weigh(int t, const float* s, float* p) {
    const float r0 = m[t][0] == -INFINITY ? 0.f : m[t][0], r1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
    p[0] = sm103::ex2_approx(s[0] - r0);
    p[1] = sm103::ex2_approx(s[1] - r1);
    p[2] = sm103::ex2_approx(s[2] - r0);
    p[3] = sm103::ex2_approx(s[3] - r1);
    l[t][0] += p[0] + p[2];
    l[t][1] += p[1] + p[3];
  }
};

// bf16 queries of KV head hk as B tiles of S^T = K Q^T: k = the head
// dimension, n = the head. Heads G and above are 0.
template <int D, int NT>
__device__ __forceinline__ void load_q_bf16(uint32_t (&qb)[NT][D / 16][2], const __nv_bfloat16* q,
                                            int G, int lane) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = t * 8 + (lane >> 2);
    const uint32_t* row = reinterpret_cast<const uint32_t*>(q + (int64_t)h * D) + (lane & 3);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qb[t][ks][0] = h < G ? row[ks * 8] : 0u;
      qb[t][ks][1] = h < G ? row[ks * 8 + 4] : 0u;
    }
  }
}

// Weights of two keys for heads 2c and 2c + 1 as a register of the B tile of
// O^T += V^T P^T: rounded to bf16, and what that left, for a second product.
__device__ __forceinline__ void weights_bf16(float p0, float p1, uint32_t& head, uint32_t& rest) {
  const uint32_t hi = wmma16::pack_bf16(p0, p1);
  const uint32_t lo =
      wmma16::pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
  head = wmma16::movmatrix_t(hi);
  rest = wmma16::movmatrix_t(lo);
}

// The merge buffer: O of COLS columns of 8 heads for each warp, and (m, l).
template <int WARPS, int COLS>
struct MergeSmem {
  static constexpr int kCols = COLS;
  float o[WARPS][8][COLS + 4];  // the lanes of a quad land in different banks
  float ml[WARPS][8][2];
};

// The state of WARPS warps (threads 0 .. 32 * WARPS - 1, which meet at named
// barrier 1) as the segment's result, or where the segment is cut as a partial
// in part_o [slot][G][D] and part_ml [slot][G][2]. put(m0, m1, t, part, sm)
// stores the warp's columns COLS * part .. of tile t for its heads 2c and 2c + 1,
// sums of 2^(score - m) times values, in p.unit. row0: the segment's first row
// of o and lse.
template <int D, int NT, int WARPS, int COLS, class Put>
__device__ __forceinline__ void leave(const Params& p, MergeSmem<WARPS, COLS>& sm, State<D, NT>& st,
                                      bool cut, float* part_o, float* part_ml, int64_t slot, int64_t row0,
                                      Put put) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane & 3;
  auto meet = [] {
    __syncwarp();  // the barrier wants whole warps, whose lanes leave the loops below at different times
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
  };
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
      st.l[t][0] += __shfl_xor_sync(0xffffffffu, st.l[t][0], sh);
      st.l[t][1] += __shfl_xor_sync(0xffffffffu, st.l[t][1], sh);
    }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int heads = min(8, p.G - t * 8);
#pragma unroll
    for (int part = 0; part < D / COLS; ++part) {
      meet();  // the buffer is free
      put(sm.o[warp][2 * c], sm.o[warp][2 * c + 1], t, part, sm);
      if (lane < 4) {
        sm.ml[warp][2 * c][0] = st.m[t][0];
        sm.ml[warp][2 * c][1] = st.l[t][0];
        sm.ml[warp][2 * c + 1][0] = st.m[t][1];
        sm.ml[warp][2 * c + 1][1] = st.l[t][1];
      }
      meet();
      // four columns of one head per thread
      for (int i = tid; i < heads * (COLS / 4); i += WARPS * 32) {
        const int h = i / (COLS / 4), d = (i % (COLS / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm.ml[w][h][0]);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float mw = sm.ml[w][h][0];
          // a state that has met no key is (-infinity, 0, 0), or has the least
          // float for m; one that has met only NaN scores has that too, and its
          // NaN must go on
          const float a = mw == -INFINITY ? 1.f : sm103::ex2_approx(mw - M);
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][h][d]);
          L = fmaf(a, sm.ml[w][h][1], L);
          acc.x = fmaf(a, x.x, acc.x); acc.y = fmaf(a, x.y, acc.y);
          acc.z = fmaf(a, x.z, acc.z); acc.w = fmaf(a, x.w, acc.w);
        }
        const int g = t * 8 + h, col = part * COLS + d;
        if (cut) {
          const int64_t r = slot * p.G + g;
          *reinterpret_cast<float4*>(part_o + r * D + col) = acc;
          if (col == 0) {
            part_ml[r * 2] = M;
            part_ml[r * 2 + 1] = L;
          }
        } else {
          const float inv = 1.f / L * p.unit;
          const int64_t r = row0 + g;
          *reinterpret_cast<uint2*>(p.o + r * D + col) =
              make_uint2(wmma16::pack_bf16(acc.x * inv, acc.y * inv),
                         wmma16::pack_bf16(acc.z * inv, acc.w * inv));
          if (col == 0 && p.lse) p.lse[r] = (M + log2f(L)) * kLn2;
        }
      }
    }
  }
}

// What the CTAs of a group leave in their shared memory, and the merge of the
// warps before it.
template <int D, int WARPS>
struct GroupSmem {
  MergeSmem<WARPS, D> merge;
  float o[16][D];
  float ml[16][2];
};

// U partial states (m, l, o) added to the state (M, L, acc). An empty one is
// (-infinity, 0, 0), or has the least float for m; one that has met only NaN
// scores has that too, and its NaN must go on.
template <int U, int E>
__device__ __forceinline__ void add_partials(float& M, float& L, float (&acc)[E], const float (&pm)[U],
                                             const float (&pl)[U], const float (&po)[U][E]) {
  float Mn = M;
#pragma unroll
  for (int u = 0; u < U; ++u) Mn = fmaxf(Mn, pm[u]);
  const float a = M == -INFINITY ? 1.f : sm103::ex2_approx(M - Mn);
  M = Mn;
  L *= a;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] *= a;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float b = pm[u] == -INFINITY ? 1.f : sm103::ex2_approx(pm[u] - M);
    L = fmaf(b, pl[u], L);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(b, po[u][e], acc[e]);
  }
}

__device__ __forceinline__ void cluster_meet() {
  __syncwarp();  // .aligned: whole warps, see meet in leave
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
  return a;
}

// The segment's result from the partials of its group, each CTA some columns of
// it. All threads of all the group's CTAs call it.
template <int D, int WARPS>
__device__ __forceinline__ void join_group(const Params& p, const GroupSmem<D, WARPS>& sm, int64_t row0) {
  cluster_meet();
  const int rank = blockIdx.x % p.group;
  for (int i = rank * blockDim.x + threadIdx.x; i < p.G * (D / 4); i += p.group * blockDim.x) {
    const int g = i / (D / 4), col = i % (D / 4) * 4;
    const uint32_t at_o = sm103::smem_u32(&sm.o[g][col]), at_ml = sm103::smem_u32(&sm.ml[g][0]);
    float M = -INFINITY, L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto add_eight = [&](int r0) {
      float m[8], l[8], o[8][4];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        m[u] = -INFINITY;
        l[u] = o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;
        if (r0 + u < p.group) {
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(m[u]), "=f"(l[u]) : "r"(cluster_addr(at_ml, r0 + u)) : "memory");
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(o[u][0]), "=f"(o[u][1]), "=f"(o[u][2]), "=f"(o[u][3])
                       : "r"(cluster_addr(at_o, r0 + u)) : "memory");
        }
      }
      add_partials<8, 4>(M, L, acc, m, l, o);
    };
    add_eight(0);
    if (p.group > 8) add_eight(8);
    const float inv = 1.f / L * p.unit;
    *reinterpret_cast<uint2*>(p.o + (row0 + g) * D + col) = make_uint2(
        wmma16::pack_bf16(acc[0] * inv, acc[1] * inv), wmma16::pack_bf16(acc[2] * inv, acc[3] * inv));
    if (col == 0 && p.lse) p.lse[row0 + g] = (M + log2f(L)) * kLn2;
  }
  cluster_meet();  // the others' shared memory stays until it has been read
}

// Every kernel of the paged cache starts as a programmatic dependent: its
// launch overlaps the end of the kernel before it in the stream, and it waits
// here, before it touches global memory, until that one has completed. (So
// what earlier kernels wrote changes while it is resident: it reads by plain
// loads, never through the non-coherent path.)
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch_dependent_clusters(void (*kernel)(P...), dim3 grid, int cluster, int threads,
                                      size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             A&&... args) {
  return launch_dependent_clusters(kernel, grid, 1, threads, smem, stream, static_cast<A&&>(args)...);
}

// CTAs for each segment of a short batch: a group, where no segment can have
// more than `most` units for each (for each two of 16); 0 where the batch is
// better cut into equal shares. What the host knows of the lengths is the
// table's width: with a table for a model's longest context every batch is cut
// into shares. Measured, GPU time in us, d = 128, G = 4, L = 24, groups of the
// given number of CTAs against the same calls with a wide table:
//   sequences x KV heads     rows      bf16 (most = 8)       4-bit (most = 21)
//                                      group     shares      group     shares
//           1 x 8             700     4.6 (8)     5.3       5.2 (8)     6.6
//           1 x 4            4000     6.1 (16)    6.4       6.4 (16)    7.1
//           1 x 4            8000     8.4 (16)    7.3       7.9 (16)    7.7
//           8 x 8       1 .. 1000     6.6 (4)     8.4       7.7 (6)    10.1
//           8 x 8       1 .. 4000    13.7 (4)    12.5      14.2 (4)    13.4
//          22 x 4       1 .. 1000     7.1 (3)     9.1       8.1 (4)    10.9
//          16 x 8       1 ..  700     7.3 (2)     9.3       8.2 (3)    11.3
//          32 x 8       1 ..  256     5.6 (1)     9.8       8.3 (1)    11.9
//          32 x 8       1 .. 1000    12.8 (1)    12.2      14.0 (1)    15.1
// More CTAs are better as long as all clusters fit the SMs at once (8 or 4 at
// 15/16 of the places did not: 6.5 -> 10), 16 where 8 would have many units each
// and there is an SM for each CTA. A cluster costs as much as `cluster_units`
// units of one CTA take; where it saves less, one CTA has the segment.
inline int group_of(const DecodePagedArgs& a, int max_units, int resident, int most, int cluster_units) {
  const int64_t segments = (int64_t)a.c.B * a.c.Hk;
  int group = (int)std::max<int64_t>(1, std::min<int64_t>(8, resident / 8 * 7 / segments));
  if ((int64_t)max_units * (group - 1) <= cluster_units * group) group = 1;
  if (segments * group > resident || max_units > most * group) return 0;
  return segments * 16 <= a.num_sms && max_units > most * 5 ? 16 : group;
}

cudaError_t launch_join(const DecodePagedArgs& a, int shares, cudaStream_t stream);
cudaError_t launch_mx4(const DecodePagedArgs& a, cudaStream_t stream);

}  // namespace paged
}  // namespace moda
