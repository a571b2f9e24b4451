// The division of a chunked prefill's work over the CTAs, see prefill_paged.cu.
//
// A tile is 2 P positions of one sequence (P a power of two) and one KV head, two halves
// of 128 rows that share its keys, and has as many blocks of 128 keys as its last
// position sees, and its depth blocks.
// All tiles lie in one line, by sequence, KV head and position, each with
// kTileCost points in front of its blocks (what entering and leaving a tile
// costs), and CTA i of n takes the i-th n-th of the line, whatever tiles it
// crosses: long chunks and short ones, over long contexts and short ones, keep
// every SM busy to the end. A tile that is cut leaves a partial state (m, l,
// unnormalised o) per CTA, and a dependent kernel joins them. The lengths stay on
// the device: each CTA finds its share by itself, a scan over the sequences and
// then closed forms.
#pragma once

#include "decode_paged.cuh"

namespace moda {
namespace prefill {

constexpr int kMaxCtas = 160;  // one per SM of 152; sizes the workspace
constexpr int kRows = 256;     // rows of a tile: positions times heads
// Points in front of a tile's blocks. Measured (us) with 2, 3, 4, 6: 16 drafts over 4-bit rows
// 37.7, 37.8, 39.7, 41.8; 32 drafts over bf16 ones 97.1, 97.8, 99.0, 101.2; 7 pieces at d = 64 1372,
// 1350, 1354, 1367; 1024 tokens without a past 41.6, 41.4, 40.9, 42.3. (Blocks of a tile of one
// half, which take 3/4 of the time, at 3 points of 4: no faster.)
constexpr int kTileCost = 3;

// The workspace: for each CTA the cut tile whose first block is its own (parts 0:
// none), and its partials: slot 2i of CTA i for a tile begun by an earlier CTA,
// 2i + 1 for the one that it begins.
struct Opened {
  int token, hk, npos, parts;  // first token, KV head, positions, partials
};
struct Work {
  Opened* opened;
  float* o;   // [2 * kMaxCtas][kRows][D]
  float* ml;  // [2 * kMaxCtas][kRows][2]
};
__host__ __device__ inline Work work_of(float* w, int D) {
  Work k;
  k.opened = reinterpret_cast<Opened*>(w);
  k.o = w + 4 * kMaxCtas;
  k.ml = k.o + (int64_t)2 * kMaxCtas * kRows * D;
  return k;
}

struct Params {
  const int *q_starts, *lens, *table;
  int N, num_pages, page_shift, max_pages, B, Hq, Hk, G, L;
  int lg_per;   // log2 of a thread's sequences in share_of
  int lgG;      // log2 of G rounded up to a power of two: rows of a position in a tile
  int n_depth;  // depth blocks of a tile
  float scale_log2;
  float unit;  // of the partials' o
  __nv_bfloat16* o;
  float* lse;
  float* work;
  unsigned int* err;
  // what the copies do not read: 4-bit pages, and values looked up one by one
  const uint8_t *k, *v, *k_scale, *v_scale;
  const __nv_bfloat16* vd;
  int64_t depth_tok, depth_hk, depth_slot;  // elements
};

// A sequence's tokens: n of them from token q0 on, the last rows of `len`.
struct Seq {
  int q0, n, len;
};
// Where starts and length make no sense the sequence has no tokens.
__device__ __forceinline__ bool read_seq(const Params& p, int b, Seq& s) {
  const int a = p.q_starts[b], e = p.q_starts[b + 1];
  s.len = p.lens[b];
  s.q0 = a;
  const bool fine = a >= 0 && e >= a && e <= p.N && s.len >= e - a && s.len <= p.max_pages << p.page_shift;
  s.n = fine ? e - a : 0;
  return fine;
}

// Points of a sequence's tiles for one KV head.
struct SeqLine {
  int nt, q, u, base, lgP, lgR, last;
  __device__ __forceinline__ SeqLine(const Params& p, const Seq& s) {
    lgP = 8 - p.lgG;     // positions of a tile
    lgR = p.lgG - 1;     // tiles of 128 positions, 2^lgR; -1: a tile has 256
    nt = (s.n + (1 << lgP) - 1) >> lgP;
    const int first_end = s.len - s.n + (1 << lgP) - 1;  // last position of tile 0, were it whole
    q = first_end >> 7;
    u = (first_end & 127) >> lgP;
    base = kTileCost + p.n_depth + 1;
    last = kTileCost + p.n_depth + ((s.len - 1) >> 7) + 1;
  }
  // points of the first m tiles, m < nt: tile i's last position is first_end + i P,
  // and the sum of floor((u + i) / R) over i below m, u below R, is one over y below u + m
  __device__ __forceinline__ long long before(int m) const {
    if (lgR < 0) return (long long)m * (base + q) + (long long)m * (m - 1);
    const int x = u + m, a = x >> lgR, r = x & ((1 << lgR) - 1);
    return (long long)m * (base + q) + (((long long)a * (a - 1)) >> 1 << lgR) + (long long)a * r;
  }
  __device__ __forceinline__ long long all() const { return nt > 0 ? before(nt - 1) + last : 0; }
};

// A CTA's share: points [from, to) of the line, and the tile that `from` lies in.
struct Share {
  long long from, to, base;
  int shares, rem;
  int b, hk, tile;
  long long tile_at;  // the tile's first point
  const uint32_t* some;  // of each warp: a bit for each thread some of whose sequences have tokens
  // The next sequence that may have tokens, where the line goes on behind sequence b: of the
  // same thread's in share_of, or the first of the next thread that found any. (One by one a
  // sequence without tokens costs 94 ns; a table of 65536 with two in use took 6.2 ms.)
  __device__ __forceinline__ int behind(const Params& p, int b) const {
    ++b;
    if (b & ((1 << p.lg_per) - 1)) return b;
    const int thread = b >> p.lg_per;
    int w = thread >> 5;
    uint32_t set = some[w] >> (thread & 31) << (thread & 31);
    while (set == 0) set = some[++w];
    return (w * 32 + __ffs(set) - 1) << p.lg_per;
  }
  __device__ __forceinline__ int owner_of(long long point) const {
    const long long wide = (base + 1) * rem;  // points of the CTAs with base + 1
    return point < wide ? (int)paged::divide(point, base + 1) : rem + (int)paged::divide(point - wide, base);
  }
};
struct ShareSmem {
  unsigned long long warp_sum[24];
  long long tile_at;
  int b, hk, tile;
};

// All threads of the CTA call it. LEAST: points that are worth a CTA.
template <int WARPS, int LEAST>
__device__ __forceinline__ Share share_of(const Params& p, ShareSmem& sm, uint32_t (&some)[24]) {
  static_assert(WARPS <= 24);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (at most 2^32 - 1: half as many a thread would be fewer than B, below 2^31)
  const int b0 = (int)min((unsigned)p.B, (unsigned)tid << p.lg_per);
  const int b1 = (int)min((unsigned)p.B, (unsigned)(tid + 1) << p.lg_per);
  unsigned long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    Seq s;
    if (!read_seq(p, b, s) && blockIdx.x == 0) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
    mine += (unsigned long long)SeqLine(p, s).all() * p.Hk;
  }
  unsigned long long before = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += x;
  }
  const uint32_t have = __ballot_sync(0xffffffffu, mine > 0);
  if (lane == 31) {
    sm.warp_sum[warp] = before;
    some[warp] = have;
  }
  __syncthreads();
  unsigned long long total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  before -= mine;
  Share s;
  const long long all = (long long)total;
  s.shares = (int)min((long long)gridDim.x, paged::divide(all + LEAST - 1, LEAST));
  s.some = some;
  s.base = s.rem = 0;
  s.from = s.to = 0;
  const int cta = blockIdx.x;
  if (s.shares > 0) {
    s.base = paged::divide(all, s.shares);
    s.rem = (int)(all - s.base * s.shares);
  }
  if (cta < s.shares) {
    s.from = s.base * cta + min(cta, s.rem);
    s.to = s.from + s.base + (cta < s.rem ? 1 : 0);
    if (s.from >= (long long)before && s.from < (long long)(before + mine)) {
      // this thread's sequences hold the first point
      long long at = (long long)before;
      for (int b = b0; b < b1; ++b) {
        Seq q;
        read_seq(p, b, q);
        const SeqLine line(p, q);
        const long long one = line.all();
        if (s.from < at + one * p.Hk) {
          const int hk = (int)paged::divide(s.from - at, one);
          at += hk * one;
          int lo = 0, hi = line.nt;  // the last tile that begins at or before the point
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (line.before(mid) <= s.from - at) lo = mid;
            else hi = mid;
          }
          sm.b = b;
          sm.hk = hk;
          sm.tile = lo;
          sm.tile_at = at + line.before(lo);
          break;
        }
        at += one * p.Hk;
      }
    }
  }
  __syncthreads();
  if (cta < s.shares) {
    s.b = sm.b;
    s.hk = sm.hk;
    s.tile = sm.tile;
    s.tile_at = sm.tile_at;
  }
  return s;
}

// The tiles of a share (in shared memory) that it has blocks of, in order; each role
// of a CTA walks them by itself.
struct Walk {
  int b, hk, tile;
  long long at, next_at;  // the tile's first point, and the next one's
  Seq seq;
  // of the current tile
  int token, npos, t0, t_last;  // first token, positions, first and last position
  int nb, j0, j1;               // blocks, and those of this share: j0 .. j1 - 1
  uint16_t nth[2];              // the how-manieth of this share it is, of all and of those of two halves
  __device__ __forceinline__ void begin(const Params& p, const Share& s) {
    b = s.b;
    hk = s.hk;
    tile = s.tile - 1;
    next_at = s.tile_at;
    nth[0] = nth[1] = 0;
    read_seq(p, b, seq);
  }
  __device__ __forceinline__ bool next(const Params& p, const Share& s) {
    const int lgP = 8 - p.lgG, P = 1 << lgP;
    while (true) {
      if (next_at >= s.to) return false;
      at = next_at;
      if (++tile << lgP >= seq.n) {
        tile = 0;
        if (++hk == p.Hk) {
          hk = 0;
          do {
            b = s.behind(p, b);
            read_seq(p, b, seq);
          } while (seq.n == 0);  // there is another: the line goes on
        }
      }
      const int first = tile << lgP;
      token = seq.q0 + first;
      npos = min(P, seq.n - first);
      t0 = seq.len - seq.n + first;
      t_last = t0 + npos - 1;
      nb = p.n_depth + (t_last >> 7) + 1;
      next_at = at + kTileCost + nb;
      const long long begin = at + kTileCost;
      j0 = s.from > begin ? (int)(s.from - begin) : 0;
      j1 = s.to < next_at ? (int)max(s.to - begin, 0LL) : nb;
      if (j1 > j0) {
        ++nth[0];
        nth[1] += npos > P >> 1;
        return true;
      }
    }
  }
  __device__ __forceinline__ bool cut() const { return j1 - j0 < nb; }
};

// Block schedule of a tile: its depth blocks are spread evenly among the sequence
// blocks (block j is a depth block iff floor((j+1) n_depth / nb) > floor(j n_depth / nb)).
struct Sched {
  int acc, db, sbk;
  bool depth = false;
  int index = 0;  // of the current block among those of its kind
  __device__ __forceinline__ Sched(int n_depth, int nb, int j0) {
    const long long x = (long long)j0 * n_depth;
    db = (int)paged::divide(x, nb);
    acc = (int)(x - (long long)db * nb);
    sbk = j0 - db;
  }
  __device__ __forceinline__ void next(int n_depth, int nb) {
    acc += n_depth;
    depth = acc >= nb;
    if (depth) {
      acc -= nb;
      index = db++;
    } else {
      index = sbk++;
    }
  }
};

}  // namespace prefill
}  // namespace moda
