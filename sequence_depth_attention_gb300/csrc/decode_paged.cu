// MoDA decode for a batch over the paged KV cache: the new token of every
// sequence attends, under one softmax, to the rows of its pages and to its L
// depth slots. Pages in bf16 or in microscaled 4-bit (include/moda.h).
//
// HBM-bound: every cached row is read once for the G query heads of its KV
// head. The batch is cut into units (64 rows of one KV head of one sequence,
// or a block of its depth slots), all units of the batch lie in one line, and
// CTA i of P takes the i-th P-th of them, whatever sequences it crosses: each
// CTA streams the same number of bytes, for one long context as for a ragged
// batch, and the lengths stay on the device. The units of one (sequence, KV
// head) are a segment. A segment inside one CTA's share is written out there;
// one that is cut leaves a partial state (m, l, unnormalised o) per CTA, and a
// dependent kernel joins them.
//
// A CTA is a producer warp and four consumer warps around a ring of
// shared-memory stages, one unit each: the producer looks up pages and issues
// TMA copies, each consumer warp scores 16 of a unit's 64 keys. Products are
// transposed (S^T = K Q^T with the keys as the rows of the A tile, then
// O^T += V^T P^T), so that the G heads fill the 8 columns of a warp MMA's B
// tile; G > 8 takes two such tiles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moda_internal.h"
#include "sm103.cuh"
#include "tensor_map.h"
#include "warp_mma.cuh"

namespace moda {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kCW = 4;                    // consumer warps
constexpr int kThreads = (kCW + 1) * 32;  // and the producer
constexpr int kKeys = 64;                 // cached rows of a unit
constexpr int kMaxCtas = 608;             // four per SM of 152; sizes the workspace
constexpr uint64_t kTimeoutNs = 2000000000ull;

// Sizes of one variant. A stage holds a unit's K and V rows (kTile bytes
// each); 4-bit units are a quarter of bf16 units, and their depth slots
// (always bf16) come 16 to a unit so that they fit the same stage.
template <int D, int NT, bool MX4>
struct Cfg {
  static constexpr int kDepthKeys = MX4 ? 16 : 64;
  static constexpr int kTile = MX4 ? kKeys * D / 2 : kKeys * D * 2;
  static constexpr int kScaleTile = MX4 ? kKeys * D / 32 : 0;
  static constexpr int kCtasPerSm = MX4 ? (NT == 1 ? 3 : 2) : 2;
  static constexpr int kNS = MX4 ? (D == 128 ? 6 : 8) : (D == 128 ? 3 : 6);
  static constexpr int kCols = 64;            // columns of O merged at a time
  static constexpr int kRowPad = kCols + 4;  // floats; lanes of a quad land in different banks
};

template <int D, int NT, bool MX4>
struct Smem {
  using C = Cfg<D, NT, MX4>;
  uint8_t ring[C::kNS][2][C::kTile];  // [stage][K or V], 1024-byte aligned
  uint8_t scales[C::kNS][2][MX4 ? C::kScaleTile : 16];
  float mo[kCW][8][C::kRowPad];  // the warps' states, for the merge
  float ml[kCW][8][2];
  uint64_t full[C::kNS], empty[C::kNS];
  long long warp_sum[kThreads / 32];
  int start[3];  // sequence, KV head, unit that the CTA's share begins with
  int abort;
};

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

struct Params {
  const __nv_bfloat16* q;
  const int* lens;
  const int* table;
  const uint8_t *k_scale, *v_scale;
  int num_pages, page_size, max_pages, B, Hk, G, L;
  int box;     // page rows of one copy: min(page_size, 64)
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  float* work;
  unsigned int* err;
};

// Sequence b's rows, within what its table can name.
__device__ __forceinline__ int rows_of(const Params& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.max_pages * p.page_size);
}

// A place in the line of units.
struct Place {
  int b, hk, off, n, len;  // unit off of the n units of segment (b, hk); len rows
  __device__ __forceinline__ void enter(const Params& p, int depth_units) {
    len = rows_of(p, b);
    n = depth_units + (len + kKeys - 1) / kKeys;
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kCW * 32) : "memory");
}

// Byte offset of (row, col) in a bf16 tile of `rows` rows: 64-column boxes,
// 16-byte chunks XORed with the row's low bits (the 128-byte TMA swizzle).
template <int ROWS>
__device__ __forceinline__ uint32_t at_bf16(int row, int col) {
  return (uint32_t)((col >> 6) * (ROWS * 128) + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4) +
                    ((col & 7) << 1));
}
// Byte offset of 16-byte chunk `chunk` of a 4-bit row: rows of D/2 bytes under
// the 64-byte (D = 128) or 32-byte (D = 64) TMA swizzle.
template <int D>
__device__ __forceinline__ uint32_t at_mx4(int row, int chunk) {
  return D == 128 ? (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4))
                  : (uint32_t)(row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4));
}
// The key that MMA index i (a row of K, a column of V^T) of a 16-key tile
// stands for in the 4-bit path: bits 0 and 1 change places, so that the four
// rows that the lanes of a quad read V from at once lie in different banks.
__device__ __forceinline__ int key_of(int i) { return (i & 12) | ((i & 1) << 1) | ((i >> 1) & 1); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The eight e2m1 codes of w as fp16 pairs: byte i gives r[i], low half first.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                             uint32_t& r3) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(w));
}
// Two scale bytes as powers of two (255: NaN).
__device__ __forceinline__ void scales_to_f32(uint32_t two, float& a, float& b) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.bf16x2.ue8m0x2 %0, t;\n}\n"
      : "=r"(r)
      : "r"(two));
  a = __uint_as_float(r << 16);
  b = __uint_as_float(r & 0xffff0000u);
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
  // Raises m of tile t to cover z (the scores plus the exponents that their
  // values carry), and brings l and o to it. z: rows r0 and r0 + 8, heads 2c
  // and 2c + 1. Most tiles bring no new maximum: one vote tells.
  __device__ __forceinline__ void raise(int t, const float* z) {
    const bool up = z[0] > m[t][0] || z[2] > m[t][0] || z[1] > m[t][1] || z[3] > m[t][1];
    if (!__any_sync(0xffffffffu, up)) return;
    float x0 = fmaxf(fmaxf(z[0], z[2]), m[t][0]), x1 = fmaxf(fmaxf(z[1], z[3]), m[t][1]);
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
      qb[t][ks][0] = h < G ? __ldg(row + ks * 8) : 0u;
      qb[t][ks][1] = h < G ? __ldg(row + ks * 8 + 4) : 0u;
    }
  }
}

// fp16 queries for the 4-bit path, times a power of two per head that brings
// the head's largest element to [2^14, 2^15): bf16's 8 bits stay whole down to
// 2^-24 of it. Lane (r0, c) holds elements 32 g + 8 c .. + 7 of head r0, the
// elements whose codes it holds of K. back: scale * log2(e) over that power,
// for the lane's heads 2c and 2c + 1.
template <int D, int NT>
__device__ __forceinline__ void load_q_f16(uint32_t (&qb)[NT][D / 32][4], float (&back)[NT][2],
                                           const __nv_bfloat16* q, int G, float scale_log2,
                                           int lane) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = t * 8 + (lane >> 2), c = lane & 3;
    uint4 raw[D / 32];
    uint32_t big = 0;
#pragma unroll
    for (int g = 0; g < D / 32; ++g) {
      raw[g] = make_uint4(0u, 0u, 0u, 0u);
      if (h < G) raw[g] = __ldg(reinterpret_cast<const uint4*>(q + (int64_t)h * D + g * 32) + c);
      const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) big = max(big, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
    }
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // exponent of the largest element, from -100 (so that the factor is a
    // normal number); infinities and NaN stay what they are under any factor
    const int e = max((int)(big >> 23) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll
    for (int g = 0; g < D / 32; ++g) {
      const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qb[t][g][i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
    }
    // heads 2c and 2c + 1 of this tile belong to lanes 8c and 8c + 4
    const float mine = scale_log2 * __uint_as_float((uint32_t)(127 - 14 + max(e, -112)) << 23);
    back[t][0] = __shfl_sync(0xffffffffu, mine, c * 8);
    back[t][1] = __shfl_sync(0xffffffffu, mine, c * 8 + 4);
  }
}

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
  uint32_t pb[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s[t][0] = k0 ? s[t][0] * scale_log2 : -INFINITY;
    s[t][1] = k0 ? s[t][1] * scale_log2 : -INFINITY;
    s[t][2] = k1 ? s[t][2] * scale_log2 : -INFINITY;
    s[t][3] = k1 ? s[t][3] * scale_log2 : -INFINITY;
    st.raise(t, s[t]);
    float p[4];
    st.weigh(t, s[t], p);
    // P^T (rows = keys, columns = heads) transposed into the B tile
    pb[t][0] = wmma16::movmatrix_t(wmma16::pack_bf16(p[0], p[1]));
    pb[t][1] = wmma16::movmatrix_t(wmma16::pack_bf16(p[2], p[3]));
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
    for (int t = 0; t < NT; ++t) wmma16::mma_bf16(st.o[t][i], a, pb[t][0], pb[t][1]);
  }
}

// In the 4-bit path O is kept 2^15 times too large, so that a weight of the
// largest row (at most 1 with its block scale) is 2^15 in fp16 and weights
// keep their 11 bits down to 2^-29 of it.
constexpr float kBias = 32768.f;

// The 16 depth slots of a unit in the 4-bit path: bf16 rows with the 4-bit
// path's order of keys and of O's rows. Columns of V^T's tiles: tile 2g + t of
// block g holds d = 32 g + 4 r0 + 2 t in row r0 and the next one in r0 + 8.
template <int D, int NT>
__device__ __forceinline__ void tile_depth_mx4(State<D, NT>& st, const uint32_t (&qb)[NT][D / 16][2],
                                               uint32_t kb, uint32_t vb, int there, float scale_log2,
                                               int lane) {
  const int r0 = lane >> 2, c = lane & 3, lr = lane & 7, lm = lane >> 3;
  float s[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    uint32_t a[4];
    wmma16::ldsm_x4(kb + at_bf16<16>((lm & 1) * 8 + key_of(lr), ks * 16 + (lm >> 1) * 8), a[0], a[1],
                    a[2], a[3]);
#pragma unroll
    for (int t = 0; t < NT; ++t) wmma16::mma_bf16(s[t], a, qb[t][ks][0], qb[t][ks][1]);
  }
  const int ka = key_of(r0);
  const bool k0 = ka < there, k1 = ka + 8 < there;
  uint32_t pb[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s[t][0] = k0 ? s[t][0] * scale_log2 : -INFINITY;
    s[t][1] = k0 ? s[t][1] * scale_log2 : -INFINITY;
    s[t][2] = k1 ? s[t][2] * scale_log2 : -INFINITY;
    s[t][3] = k1 ? s[t][3] * scale_log2 : -INFINITY;
    st.raise(t, s[t]);
    float p[4];
    st.weigh(t, s[t], p);
    pb[t][0] = wmma16::movmatrix_t(wmma16::pack_bf16(p[0] * kBias, p[1] * kBias));
    pb[t][1] = wmma16::movmatrix_t(wmma16::pack_bf16(p[2] * kBias, p[3] * kBias));
  }
  // rows past L were filled with zeros by the copy
  const int v0 = key_of(2 * c);
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {
    const int col = g * 32 + r0 * 4;
    const uint2 x0 = lds64(vb + at_bf16<16>(v0, col)), x1 = lds64(vb + at_bf16<16>(v0 + 2, col));
    const uint2 x2 = lds64(vb + at_bf16<16>(v0 + 8, col)), x3 = lds64(vb + at_bf16<16>(v0 + 10, col));
    const uint32_t a[4] = {__byte_perm(x0.x, x1.x, 0x5410), __byte_perm(x0.x, x1.x, 0x7632),
                           __byte_perm(x2.x, x3.x, 0x5410), __byte_perm(x2.x, x3.x, 0x7632)};
    const uint32_t b[4] = {__byte_perm(x0.y, x1.y, 0x5410), __byte_perm(x0.y, x1.y, 0x7632),
                           __byte_perm(x2.y, x3.y, 0x5410), __byte_perm(x2.y, x3.y, 0x7632)};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wmma16::mma_bf16(st.o[t][2 * g], a, pb[t][0], pb[t][1]);
      wmma16::mma_bf16(st.o[t][2 * g + 1], b, pb[t][0], pb[t][1]);
    }
  }
}

// 16 4-bit keys (rows row0.. of a unit, `there` of them exist) into the state.
// K's codes are exact in fp16; a block's products are summed by two MMAs and
// then multiplied by its scale. V's block scales go into P, one P^T per block:
// m covers score + exponent of the row's largest scale, so that no product of
// weight and scale passes 1.
template <int D, int NT>
__device__ __forceinline__ void tile_mx4(State<D, NT>& st, const uint32_t (&qb)[NT][D / 32][4],
                                         const float (&back)[NT][2], uint32_t kb, uint32_t vb,
                                         uint32_t ksb, uint32_t vsb, int row0, int there, int lane) {
  constexpr int NB = D / 32;  // blocks of a row
  const int r0 = lane >> 2, c = lane & 3;
  const int ka = key_of(r0);  // this lane's keys: ka and ka + 8 of the tile
  const bool k0 = ka < there, k1 = ka + 8 < there;
  uint32_t ks0, ks1, vs0, vs1;
  const uint32_t so = (uint32_t)(row0 + ka) * NB;
  if constexpr (NB == 4) {
    ks0 = lds32(ksb + so); ks1 = lds32(ksb + so + 8 * NB);
    vs0 = lds32(vsb + so); vs1 = lds32(vsb + so + 8 * NB);
  } else {
    ks0 = lds16(ksb + so); ks1 = lds16(ksb + so + 8 * NB);
    vs0 = lds16(vsb + so); vs1 = lds16(vsb + so + 8 * NB);
  }
  // what lies behind the last row may be any byte: weight 0 times a power of two
  if (!k0) vs0 = 0x7f7f7f7fu;
  if (!k1) vs1 = 0x7f7f7f7fu;

  float s[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
  float f0[NB], f1[NB];
#pragma unroll
  for (int g = 0; g < NB; g += 2) {
    scales_to_f32(ks0 >> (8 * g), f0[g], f0[g + 1]);
    scales_to_f32(ks1 >> (8 * g), f1[g], f1[g + 1]);
  }
#pragma unroll
  for (int g = 0; g < NB; ++g) {
    uint32_t a[4], b[4];  // two k-steps of 16
    codes_to_f16(lds32(kb + at_mx4<D>(row0 + ka, g) + c * 4), a[0], a[2], b[0], b[2]);
    codes_to_f16(lds32(kb + at_mx4<D>(row0 + ka + 8, g) + c * 4), a[1], a[3], b[1], b[3]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(x, a, qb[t][g][0], qb[t][g][1]);
      mma_f16(x, b, qb[t][g][2], qb[t][g][3]);
      s[t][0] = fmaf(x[0], f0[g], s[t][0]);
      s[t][1] = fmaf(x[1], f0[g], s[t][1]);
      s[t][2] = fmaf(x[2], f1[g], s[t][2]);
      s[t][3] = fmaf(x[3], f1[g], s[t][3]);
    }
  }
  // V's scales, and the exponent of each row's largest (NaN aside), from -96 so
  // that the sum of 2^(score - m) stays in range
#pragma unroll
  for (int g = 0; g < NB; g += 2) {
    scales_to_f32(vs0 >> (8 * g), f0[g], f0[g + 1]);
    scales_to_f32(vs1 >> (8 * g), f1[g], f1[g + 1]);
  }
  float b0 = 0x1p-96f, b1 = 0x1p-96f;
#pragma unroll
  for (int g = 0; g < NB; ++g) {
    b0 = fmaxf(b0, f0[g]);
    b1 = fmaxf(b1, f1[g]);
  }
  const float e0 = (float)((int)(__float_as_uint(b0) >> 23) - 127);
  const float e1 = (float)((int)(__float_as_uint(b1) >> 23) - 127);

  float p[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s[t][0] = k0 ? s[t][0] * back[t][0] : -INFINITY;
    s[t][1] = k0 ? s[t][1] * back[t][1] : -INFINITY;
    s[t][2] = k1 ? s[t][2] * back[t][0] : -INFINITY;
    s[t][3] = k1 ? s[t][3] * back[t][1] : -INFINITY;
    const float z[4] = {s[t][0] + e0, s[t][1] + e0, s[t][2] + e1, s[t][3] + e1};
    st.raise(t, z);
    st.weigh(t, s[t], p[t]);
  }
  const int v0 = row0 + key_of(2 * c);
#pragma unroll
  for (int g = 0; g < NB; ++g) {
    // 4 codes (d = 32 g + 4 r0 .. + 3) of each of the lane's 4 keys; the same
    // code of a pair of keys side by side in a byte
    const uint32_t r2 = r0 * 2;
    const uint32_t x = lds16(vb + at_mx4<D>(v0, g) + r2) | (lds16(vb + at_mx4<D>(v0 + 8, g) + r2) << 16);
    const uint32_t y =
        lds16(vb + at_mx4<D>(v0 + 2, g) + r2) | (lds16(vb + at_mx4<D>(v0 + 10, g) + r2) << 16);
    uint32_t a[4], b[4];
    codes_to_f16((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), a[0], b[0], a[2], b[2]);
    codes_to_f16(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), a[1], b[1], a[3], b[3]);
    const float w0 = f0[g] * kBias, w1 = f1[g] * kBias;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint32_t pb0 = wmma16::movmatrix_t(pack_f16(p[t][0] * w0, p[t][1] * w0));
      const uint32_t pb1 = wmma16::movmatrix_t(pack_f16(p[t][2] * w1, p[t][3] * w1));
      mma_f16(st.o[t][2 * g], a, pb0, pb1);
      mma_f16(st.o[t][2 * g + 1], b, pb0, pb1);
    }
  }
}

// ------------------------------------------------------------ the split kernel
template <int D, int NT, bool MX4>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, MX4>::kCtasPerSm)
decode_paged_split(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmKd, const __grid_constant__ CUtensorMap tmVd,
                   const __grid_constant__ Params p) {
  using C = Cfg<D, NT, MX4>;
  using S = Smem<D, NT, MX4>;
  constexpr int NS = C::kNS;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int depth_units = (p.L + C::kDepthKeys - 1) / C::kDepthKeys;
  const Work wk = work_of(p.work, p.G, D);

  if (tid == 0) {
    sm.abort = 0;
    for (int s = 0; s < NS; ++s) {
      sm103::mbar_init(sm103::smem_u32(&sm.full[s]), 1);
      sm103::mbar_init(sm103::smem_u32(&sm.empty[s]), kCW);
    }
    sm103::fence_barrier_init();
  }
  // the joining kernel may be scheduled now; it waits for this grid to finish
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Units before each thread's run of sequences, and in all.
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int raw = __ldg(p.lens + b);
    if (raw < 0 || raw > p.max_pages * p.page_size)
      atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
    mine += depth_units + (rows_of(p, b) + kKeys - 1) / kKeys;
  }
  long long before = mine;  // inclusive scan of the warp
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += x;
  }
  if (lane == 31) sm.warp_sum[warp] = before;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  before = (before - mine) * p.Hk;
  total *= p.Hk;
  const int shares = (int)min((long long)gridDim.x, total);
  const int cta = blockIdx.x;
  const long long u0 = cta < shares ? total * cta / shares : 0;
  const long long u1 = cta < shares ? total * (cta + 1) / shares : 0;
  if (u0 < u1 && u0 >= before && u0 < before + mine * p.Hk) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const int n = depth_units + (rows_of(p, b) + kKeys - 1) / kKeys;
      if (u0 < at + (long long)n * p.Hk) {
        sm.start[0] = b;
        sm.start[1] = (int)((u0 - at) / n);
        sm.start[2] = (int)((u0 - at) % n);
        break;
      }
      at += (long long)n * p.Hk;
    }
  }
  // sequences with nothing to attend to
  if (depth_units == 0) {
    const int Hq = p.Hk * p.G;
    for (int b = cta; b < p.B; b += gridDim.x) {
      if (rows_of(p, b) != 0) continue;
      uint32_t* o = reinterpret_cast<uint32_t*>(p.o + (int64_t)b * Hq * D);
      for (int i = tid; i < Hq * D / 2; i += kThreads) o[i] = 0u;
      if (p.lse)
        for (int i = tid; i < Hq; i += kThreads) p.lse[(int64_t)b * Hq + i] = -INFINITY;
    }
  }
  __syncthreads();
  if (u0 >= u1) {
    if (tid == 0) wk.opened[cta] = make_int2(-1, 0);
    return;
  }
  Place at{sm.start[0], sm.start[1], sm.start[2], 0, 0};
  at.enter(p, depth_units);

  if (warp == kCW) {
    // ------------------------------------------------------------ producer
    // One page row block per lane; the next unit's pages are looked up before
    // the wait for a free stage.
    auto page_of = [&](const Place& x) -> int {
      if (x.off < depth_units) return 0;
      const int key = (x.off - depth_units) * kKeys + lane * p.box;
      if (lane * p.box >= kKeys || key >= x.len) return 0;
      return __ldg(p.table + (int64_t)x.b * p.max_pages + key / p.page_size);
    };
    const long long n = u1 - u0;
    int page = page_of(at);
    for (long long k = 0; k < n; ++k) {
      const Place cur = at;
      int pg = page;
      if (k + 1 < n) {
        if (++at.off == at.n) at.next_segment(p, depth_units);
        page = page_of(at);
      }
      const int s = (int)(k % NS);
      const uint32_t bar = sm103::smem_u32(&sm.full[s]);
      if (k >= NS)
        sm103::mbar_wait_bounded(sm103::smem_u32(&sm.empty[s]), (uint32_t)((k / NS - 1) & 1), &sm.abort,
                                 kTimeoutNs);
      if (__any_sync(0xffffffffu, *(volatile int*)&sm.abort)) break;
      const uint32_t kt = sm103::smem_u32(&sm.ring[s][0][0]), vt = sm103::smem_u32(&sm.ring[s][1][0]);
      if (cur.off < depth_units) {
        if (lane == 0) {
          constexpr uint32_t kBox = C::kDepthKeys * 128;  // 64 columns
          sm103::mbar_arrive_expect_tx(bar, 2 * (D / 64) * kBox);
          const int l = cur.off * C::kDepthKeys;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            sm103::tma_load_4d(kt + x * kBox, &tmKd, bar, x * 64, l, cur.hk, cur.b);
            sm103::tma_load_4d(vt + x * kBox, &tmVd, bar, x * 64, l, cur.hk, cur.b);
          }
        }
      } else {
        const int key0 = (cur.off - depth_units) * kKeys;
        const int boxes = (min(kKeys, cur.len - key0) + p.box - 1) / p.box;
        const uint32_t box_bytes = (uint32_t)p.box * (MX4 ? D + D / 16 : D * 4);  // K and V
        if (lane == 0) sm103::mbar_arrive_expect_tx(bar, boxes * box_bytes);
        __syncwarp();
        if (lane < boxes) {
          if (pg < 0 || pg >= p.num_pages) {
            atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
            pg = 0;
          }
          const int row = (key0 + lane * p.box) % p.page_size;
          const int head = pg * p.Hk + cur.hk;
          if constexpr (MX4) {
            sm103::tma_load_3d(kt + lane * p.box * (D / 2), &tmK, bar, 0, row, head);
            sm103::tma_load_3d(vt + lane * p.box * (D / 2), &tmV, bar, 0, row, head);
            const int64_t so = ((int64_t)head * p.page_size + row) * (D / 32);
            const uint32_t sd = lane * p.box * (D / 32), bytes = p.box * (D / 32);
            bulk_load(sm103::smem_u32(&sm.scales[s][0][0]) + sd, p.k_scale + so, bytes, bar);
            bulk_load(sm103::smem_u32(&sm.scales[s][1][0]) + sd, p.v_scale + so, bytes, bar);
          } else {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              const uint32_t off = x * (kKeys * 128) + lane * p.box * 128;
              sm103::tma_load_3d(kt + off, &tmK, bar, x * 64, row, head);
              sm103::tma_load_3d(vt + off, &tmV, bar, x * 64, row, head);
            }
          }
        }
      }
    }
    if (*(volatile int*)&sm.abort && lane == 0) {
      // a wait gave up: let every stage's copies land before the CTA goes
      int never = 0;
      for (int s = 0; s < NS && s < n; ++s)
        for (uint32_t ph = 0; ph < 2; ++ph)
          sm103::mbar_wait_bounded(sm103::smem_u32(&sm.full[s]), ph, &never, kTimeoutNs / 100);
      atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_TIMEOUT);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // After a wait that gave up the warps go through the same steps, without the
  // arithmetic, so that they meet at the same barriers.
  const int r0 = lane >> 2, c = lane & 3;
  State<D, NT> st;
  long long k = 0, left = u1 - u0;
  bool opened = false;
  while (left > 0) {
    const int cnt = (int)min(left, (long long)(at.n - at.off));
    const int end = at.off + cnt;
    const bool cut_before = at.off > 0, cut_after = end < at.n;
    const __nv_bfloat16* q = p.q + ((int64_t)at.b * p.Hk + at.hk) * p.G * D;
    st.clear();
    int off = at.off;
    auto take = [&](int s) {
      return sm103::mbar_wait_bounded(sm103::smem_u32(&sm.full[s]), (uint32_t)((k / NS) & 1), &sm.abort,
                                      kTimeoutNs);
    };
    auto give = [&](int s) {
      __syncwarp();
      if (lane == 0) sm103::mbar_arrive(sm103::smem_u32(&sm.empty[s]));
      ++k;
    };
    if constexpr (MX4) {
      if (off < depth_units) {
        uint32_t qb[NT][D / 16][2];
        load_q_bf16<D, NT>(qb, q, p.G, lane);
        for (; off < min(end, depth_units); ++off) {
          const int s = (int)(k % NS);
          const bool ok = take(s);
          if (ok && (off & (kCW - 1)) == warp)  // a warp each in turn
            tile_depth_mx4<D, NT>(st, qb, sm103::smem_u32(&sm.ring[s][0][0]),
                                  sm103::smem_u32(&sm.ring[s][1][0]), p.L - off * C::kDepthKeys,
                                  p.scale_log2, lane);
          give(s);
        }
      }
      if (off < end) {
        uint32_t qb[NT][D / 32][4];
        float back[NT][2];
        load_q_f16<D, NT>(qb, back, q, p.G, p.scale_log2, lane);
        for (; off < end; ++off) {
          const int s = (int)(k % NS);
          const bool ok = take(s);
          const int there = at.len - (off - depth_units) * kKeys - warp * 16;
          if (ok && there > 0)
            tile_mx4<D, NT>(st, qb, back, sm103::smem_u32(&sm.ring[s][0][0]),
                            sm103::smem_u32(&sm.ring[s][1][0]), sm103::smem_u32(&sm.scales[s][0][0]),
                            sm103::smem_u32(&sm.scales[s][1][0]), warp * 16, there, lane);
          give(s);
        }
      }
    } else {
      uint32_t qb[NT][D / 16][2];
      load_q_bf16<D, NT>(qb, q, p.G, lane);
      for (; off < end; ++off) {
        const int s = (int)(k % NS);
        const bool ok = take(s);
        const int there = (off < depth_units ? p.L - off * C::kDepthKeys
                                             : at.len - (off - depth_units) * kKeys) - warp * 16;
        if (ok && there > 0)
          tile_bf16<D, NT, kKeys>(st, qb, sm103::smem_u32(&sm.ring[s][0][0]),
                                  sm103::smem_u32(&sm.ring[s][1][0]), warp * 16, there, p.scale_log2,
                                  lane);
        give(s);
      }
    }

    // ---------------------------------------------- the segment's result
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) {
        st.l[t][0] += __shfl_xor_sync(0xffffffffu, st.l[t][0], sh);
        st.l[t][1] += __shfl_xor_sync(0xffffffffu, st.l[t][1], sh);
      }
    const int slot = 2 * cta + (cut_before ? 0 : 1);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int heads = min(8, p.G - t * 8);
#pragma unroll
      for (int half = 0; half < D / C::kCols; ++half) {
        consumers_sync();  // the buffer is free
        float* m0 = sm.mo[warp][2 * c];
        float* m1 = sm.mo[warp][2 * c + 1];
        if constexpr (MX4) {
#pragma unroll
          for (int g = 0; g < C::kCols / 32; ++g) {
            const float(&x)[4] = st.o[t][half * 4 + 2 * g];
            const float(&y)[4] = st.o[t][half * 4 + 2 * g + 1];
            const int d = g * 32 + r0 * 4;
            *reinterpret_cast<float4*>(m0 + d) = make_float4(x[0], x[2], y[0], y[2]);
            *reinterpret_cast<float4*>(m1 + d) = make_float4(x[1], x[3], y[1], y[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < C::kCols / 16; ++i) {
            const float(&x)[4] = st.o[t][half * 4 + i];
            m0[i * 16 + r0] = x[0];
            m1[i * 16 + r0] = x[1];
            m0[i * 16 + r0 + 8] = x[2];
            m1[i * 16 + r0 + 8] = x[3];
          }
        }
        if (r0 == 0) {
          sm.ml[warp][2 * c][0] = st.m[t][0];
          sm.ml[warp][2 * c][1] = st.l[t][0];
          sm.ml[warp][2 * c + 1][0] = st.m[t][1];
          sm.ml[warp][2 * c + 1][1] = st.l[t][1];
        }
        consumers_sync();
        // four columns of one head per thread
        const int h = tid / (C::kCols / 4), d = (tid % (C::kCols / 4)) * 4;
        if (h < heads) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kCW; ++w) M = fmaxf(M, sm.ml[w][h][0]);
          float L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kCW; ++w) {
            const float mw = sm.ml[w][h][0];
            // a state that has met no key is (-infinity, 0, 0); one that has met
            // only NaN scores has -infinity too, and its NaN must go on
            const float a = mw == -INFINITY ? 1.f : sm103::ex2_approx(mw - M);
            const float4 x = *reinterpret_cast<const float4*>(&sm.mo[w][h][d]);
            L = fmaf(a, sm.ml[w][h][1], L);
            acc.x = fmaf(a, x.x, acc.x); acc.y = fmaf(a, x.y, acc.y);
            acc.z = fmaf(a, x.z, acc.z); acc.w = fmaf(a, x.w, acc.w);
          }
          const int g = t * 8 + h, col = half * C::kCols + d;
          if (cut_before || cut_after) {
            *reinterpret_cast<float4*>(wk.o + ((int64_t)slot * p.G + g) * D + col) = acc;
            if (col == 0) {
              wk.ml[((int64_t)slot * p.G + g) * 2] = M;
              wk.ml[((int64_t)slot * p.G + g) * 2 + 1] = L;
            }
          } else {
            const float inv = 1.f / (MX4 ? L * kBias : L);
            const int64_t r = ((int64_t)at.b * p.Hk + at.hk) * p.G + g;
            *reinterpret_cast<uint2*>(p.o + r * D + col) =
                make_uint2(wmma16::pack_bf16(acc.x * inv, acc.y * inv),
                           wmma16::pack_bf16(acc.z * inv, acc.w * inv));
            if (col == 0 && p.lse) p.lse[r] = (M + log2f(L)) * kLn2;
          }
        }
      }
    }
    if (cut_after && !cut_before) {
      opened = true;
      if (tid == 0) {
        // the CTA that owns the segment's last unit, and so the partials' number
        const long long last = u0 + (k - cnt) + (at.n - at.off) - 1;
        const int j = (int)(((last + 1) * shares + total - 1) / total) - 1;
        wk.opened[cta] = make_int2(at.b * p.Hk + at.hk, j - cta + 1);
      }
    }
    left -= cnt;
    if (left > 0) at.next_segment(p, depth_units);
  }
  if (tid == 0) {
    if (!opened) wk.opened[cta] = make_int2(-1, 0);
    if (sm.abort) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_TIMEOUT);
  }
}

// Joins the partials of the segment that split CTA blockIdx.x opened, for head
// blockIdx.y: 8 warps take them in turn, each lane D/32 columns.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
decode_paged_join(float* work, int G, float bias, __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
  constexpr int E = D / 32;
  constexpr int U = 8;  // partials a warp loads before it adds the first
  __shared__ float sm_o[kJoinWarps][D];
  __shared__ float sm_ml[kJoinWarps][2];
  const Work wk = work_of(work, G, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y;
  // launched as a programmatic dependent of the split kernel: wait until that
  // grid has completed and what it wrote is visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 seg = wk.opened[blockIdx.x];
  if (seg.x < 0) return;
  float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = warp; i0 < seg.y; i0 += kJoinWarps * U) {
    float pm[U], pl[U], po[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kJoinWarps;
      pm[u] = -INFINITY;
      pl[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) po[u][e] = 0.f;
      if (i < seg.y) {
        const int64_t row = (int64_t)(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * G + g;
        pm[u] = wk.ml[row * 2];
        pl[u] = wk.ml[row * 2 + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) po[u][e] = wk.o[row * D + lane * E + e];
      }
    }
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
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    sm_ml[warp][0] = M;
    sm_ml[warp][1] = L;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    float Mt = -INFINITY, Lt = 0.f, ot = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) Mt = fmaxf(Mt, sm_ml[w][0]);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float a = sm_ml[w][0] == -INFINITY ? 1.f : sm103::ex2_approx(sm_ml[w][0] - Mt);
      Lt = fmaf(a, sm_ml[w][1], Lt);
      ot = fmaf(a, sm_o[w][d], ot);
    }
    const int64_t r = (int64_t)seg.x * G + g;
    o[r * D + d] = __float2bfloat16_rn(ot / (Lt * bias));
    if (d == 0 && lse) lse[r] = (Mt + log2f(Lt)) * kLn2;
  }
}

template <int D, int NT, bool MX4>
cudaError_t launch(const DecodePagedArgs& a, cudaStream_t stream) {
  using C = Cfg<D, NT, MX4>;
  const PagedKv& c = a.c;
  Params p{};
  p.q = (const __nv_bfloat16*)a.q;
  p.lens = a.seq_lens;
  p.table = c.table;
  p.k_scale = (const uint8_t*)c.k_scale;
  p.v_scale = (const uint8_t*)c.v_scale;
  p.num_pages = c.num_pages; p.page_size = c.page_size; p.max_pages = c.max_pages;
  p.B = c.B; p.Hk = c.Hk; p.G = a.G; p.L = a.L;
  p.box = c.page_size < kKeys ? c.page_size : kKeys;
  p.scale_log2 = a.scale * kLog2e;
  p.o = (__nv_bfloat16*)a.o;
  p.lse = a.lse;
  p.work = a.work;
  p.err = c.err;

  // pages as [num_pages * Hk][page_size][row]; depth slots as [B][Hk][L][D]
  CUtensorMap tk, tv, tkd, tvd;
  {
    const uint64_t row = MX4 ? D / 2 : D * 2;
    const uint64_t dims[3] = {(uint64_t)(MX4 ? D / 2 : D), (uint64_t)c.page_size,
                              (uint64_t)c.num_pages * c.Hk};
    const uint64_t str[2] = {row, row * c.page_size};
    const uint32_t box[3] = {MX4 ? D / 2 : 64, (uint32_t)p.box, 1};
    if (MX4) {
      if (encode_bytes_swizzled(&tk, c.k, 3, dims, str, box) != CUDA_SUCCESS ||
          encode_bytes_swizzled(&tv, c.v, 3, dims, str, box) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    } else {
      if (encode_bf16_sw128(&tk, c.k, 3, dims, str, box) != CUDA_SUCCESS ||
          encode_bf16_sw128(&tv, c.v, 3, dims, str, box) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
  }
  if (a.L > 0) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.L, (uint64_t)c.Hk, (uint64_t)c.B};
    const uint64_t str[3] = {(uint64_t)a.depth_slot_stride * 2, (uint64_t)a.depth_hk_stride * 2,
                             (uint64_t)a.depth_b_stride * 2};
    const uint32_t box[4] = {64, (uint32_t)C::kDepthKeys, 1, 1};
    if (encode_bf16_sw128(&tkd, a.kd, 4, dims, str, box) != CUDA_SUCCESS ||
        encode_bf16_sw128(&tvd, a.vd, 4, dims, str, box) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  } else {
    tkd = tk;  // never read when L == 0
    tvd = tv;
  }
  const size_t smem = sizeof(Smem<D, NT, MX4>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(decode_paged_split<D, NT, MX4>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int grid = a.num_sms * C::kCtasPerSm;
  grid = grid < kMaxCtas ? grid : kMaxCtas;
  decode_paged_split<D, NT, MX4><<<grid, kThreads, smem, stream>>>(tk, tv, tkd, tvd, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // programmatic dependent launch: the joining CTAs become resident while the
  // split kernel runs and start as soon as it completes
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, a.G);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_paged_join<D>, a.work, a.G, MX4 ? kBias : 1.f,
                         (__nv_bfloat16*)a.o, a.lse);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const DecodePagedArgs& a, cudaStream_t stream) {
  const bool mx4 = a.c.format == MODA_KV_MX4;
  if (a.G <= 8) return mx4 ? launch<D, 1, true>(a, stream) : launch<D, 1, false>(a, stream);
  return mx4 ? launch<D, 2, true>(a, stream) : launch<D, 2, false>(a, stream);
}

}  // namespace

size_t decode_paged_workspace_bytes(int Hq, int Hk, int d) {
  const int64_t G = Hq / Hk;
  return (size_t)(2 * kMaxCtas + 2 * kMaxCtas * G * (d + 2)) * sizeof(float);
}

cudaError_t launch_decode_paged(const DecodePagedArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace moda
