// MoDA decode for a batch over the paged KV cache in microscaled 4-bit (e2m1
// codes, a power-of-two scale for each block of 32; layout in include/moda.h).
// decode_paged.cuh has the division of the work.
//
// A row takes 4.25 bits an element, so at the memory's rate an SM has to
// unpack and multiply 43 elements a cycle: the kernel is bound by instruction
// issue as much as by HBM, and its arithmetic is laid out to need few.
//   S^T = K Q^T: a lane reads whole 32-bit words of codes of its keys (the
//     order of the head dimension in a product is free, so Q is loaded in the
//     same order), one conversion gives two fp16 values, two warp MMAs (fp16)
//     sum a block of 32, and the block's scale is applied to the fp32 sum.
//   O^T += V^T P^T: a lane pairs the codes of two keys in a byte, one
//     conversion gives their fp16 pair. V's block scales go into P, one P^T
//     per block of 32 columns.
// Each warp streams units of its own (32 rows, or 16 depth slots) through its
// own ring of shared-memory stages by asynchronous copies: no barrier between
// warps but at the end of a segment.
#include <cuda_fp16.h>

#include "decode_paged.cuh"

namespace moda {
namespace paged {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32;       // cached rows of a unit
constexpr int kDepthKeys = 16;  // depth slots of a unit; their K and V take a stage each
constexpr int kNS = 3;          // stages of a warp
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 3 : 2;

template <int D>
struct Smem {
  uint8_t codes[kWarps][kNS][2 * kKeys * D / 2];  // 1024-byte aligned stages
  uint8_t scales[kWarps][kNS][2][kKeys * D / 32];
  MergeSmem<kWarps> merge;
  ShareSmem<kWarps> share;
};

struct Mx4Pages {
  const uint8_t *k, *v, *k_scale, *v_scale;
  const uint8_t *kd, *vd;  // depth slots, bf16
  int64_t depth_b, depth_hk, depth_slot;  // bytes
};

// m is kept 15 below the largest score (with its values' exponent), so that
// the largest weight is 2^15: in fp16 weights then keep their 11 bits down to
// 2^-29 of it.
constexpr float kHeadroom = 15.f;

// Byte offset of 16-byte chunk `chunk` of a 4-bit row: rows of D/2 bytes whose
// chunks are XORed with bits of the row, so that neither the words that a warp
// reads of 8 keys of K nor the half words of 4 keys of V meet in a bank.
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

__device__ __forceinline__ void cp16(uint32_t dst, const uint8_t* src, bool there) {
  wmma16::cp_async16(dst, src, there ? 16u : 0u);
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Weights of 16 depth slots: p, as B tiles of O^T += V^T P^T.
template <int D, int NT>
__device__ __forceinline__ void depth_scores(State<D, NT>& st, const uint32_t (&qb)[NT][D / 16][2],
                                             uint32_t kb, int there, float scale_log2, int lane,
                                             uint32_t (&pb)[NT][2]) {
  const int lr = lane & 7, lm = lane >> 3;
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
  const int ka = key_of(lane >> 2);
  const bool k0 = ka < there, k1 = ka + 8 < there;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    s[t][0] = k0 ? s[t][0] * scale_log2 : -INFINITY;
    s[t][1] = k0 ? s[t][1] * scale_log2 : -INFINITY;
    s[t][2] = k1 ? s[t][2] * scale_log2 : -INFINITY;
    s[t][3] = k1 ? s[t][3] * scale_log2 : -INFINITY;
    const float z[4] = {s[t][0] - kHeadroom, s[t][1] - kHeadroom, s[t][2] - kHeadroom,
                        s[t][3] - kHeadroom};
    st.raise(t, z);
    float p[4];
    st.weigh(t, s[t], p);
    pb[t][0] = wmma16::movmatrix_t(wmma16::pack_bf16(p[0], p[1]));
    pb[t][1] = wmma16::movmatrix_t(wmma16::pack_bf16(p[2], p[3]));
  }
}

// Their values, in this kernel's order of O's rows: tile 2g + t of block g
// holds d = 32 g + 4 r0 + 2 t in row r0 and the next one in r0 + 8. Rows past
// L are zeros.
template <int D, int NT>
__device__ __forceinline__ void depth_values(State<D, NT>& st, const uint32_t (&pb)[NT][2], uint32_t vb,
                                             int lane) {
  const int r0 = lane >> 2, v0 = key_of(2 * (lane & 3));
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

// The 32 rows of a unit into the state, two tiles of 16 keys side by side.
// TAIL: only `there` of them exist.
template <int D, int NT, bool TAIL>
__device__ __forceinline__ void unit_mx4(State<D, NT>& st, const uint32_t (&qb)[NT][D / 32][4],
                                         const float (&back)[NT][2], uint32_t kb, uint32_t vb,
                                         uint32_t ksb, uint32_t vsb, int there, int lane) {
  constexpr int NB = D / 32;  // blocks of a row
  constexpr int ROW = D / 2;  // bytes
  const int r0 = lane >> 2, c = lane & 3;
  const int ka = key_of(r0);  // this lane's keys: ka + 8 i, i = 0 .. 3
  auto scale_word = [&](uint32_t base, int i) -> uint32_t {
    const uint32_t a = base + (ka + 8 * i) * NB;
    return NB == 4 ? lds32(a) : lds16(a);
  };
  float s[2][NT][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float f[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = scale_word(ksb, 2 * j + i);
#pragma unroll
      for (int g = 0; g < NB; g += 2) scales_to_f32(w >> (8 * g), f[i][g], f[i][g + 1]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) s[j][t][0] = s[j][t][1] = s[j][t][2] = s[j][t][3] = 0.f;
#pragma unroll
    for (int g = 0; g < NB; ++g) {
      uint32_t a[4], b[4];  // two k-steps of 16
      const uint32_t w = kb + at_mx4<D>(ka, g) + c * 4 + j * 16 * ROW;
      codes_to_f16(lds32(w), a[0], a[2], b[0], b[2]);
      codes_to_f16(lds32(w + 8 * ROW), a[1], a[3], b[1], b[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(x, a, qb[t][g][0], qb[t][g][1]);
        mma_f16(x, b, qb[t][g][2], qb[t][g][3]);
        s[j][t][0] = fmaf(x[0], f[0][g], s[j][t][0]);
        s[j][t][1] = fmaf(x[1], f[0][g], s[j][t][1]);
        s[j][t][2] = fmaf(x[2], f[1][g], s[j][t][2]);
        s[j][t][3] = fmaf(x[3], f[1][g], s[j][t][3]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // V's scales, and the exponent of each row's largest (NaN aside), from -80
    // so that the sum of 2^(score - m) stays in range
    float f[2][NB], e[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w = scale_word(vsb, 2 * j + i);
      // what lies behind the last row may be any byte: weight 0 times a power of two
      if (TAIL && ka + 8 * (2 * j + i) >= there) w = 0x7f7f7f7fu;
#pragma unroll
      for (int g = 0; g < NB; g += 2) scales_to_f32(w >> (8 * g), f[i][g], f[i][g + 1]);
      float big = 0x1p-80f;
#pragma unroll
      for (int g = 0; g < NB; ++g) big = fmaxf(big, f[i][g]);
      e[i] = (float)((int)(__float_as_uint(big) >> 23) - 127) - kHeadroom;
    }
    float p[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = s[j][t][i] * back[t][i & 1];
        if (TAIL && ka + 8 * (2 * j + (i >> 1)) >= there) x[i] = -INFINITY;
      }
      const float z[4] = {x[0] + e[0], x[1] + e[0], x[2] + e[1], x[3] + e[1]};
      st.raise(t, z);
      st.weigh(t, x, p[t]);
    }
    const int v0 = key_of(2 * c);
    const uint32_t r2 = r0 * 2 + j * 16 * ROW;
#pragma unroll
    for (int g = 0; g < NB; ++g) {
      // 4 codes (d = 32 g + 4 r0 .. + 3) of each of the lane's 4 keys; the same
      // code of a pair of keys side by side in a byte
      const uint32_t w0 = vb + at_mx4<D>(v0, g) + r2, w1 = vb + at_mx4<D>(v0 + 2, g) + r2;
      const uint32_t x = lds16(w0) | (lds16(w0 + 8 * ROW) << 16);
      const uint32_t y = lds16(w1) | (lds16(w1 + 8 * ROW) << 16);
      uint32_t a[4], b[4];
      codes_to_f16((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), a[0], b[0], a[2], b[2]);
      codes_to_f16(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), a[1], b[1], a[3], b[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t pb0 = wmma16::movmatrix_t(pack_f16(p[t][0] * f[0][g], p[t][1] * f[0][g]));
        const uint32_t pb1 = wmma16::movmatrix_t(pack_f16(p[t][2] * f[1][g], p[t][3] * f[1][g]));
        mma_f16(st.o[t][2 * g], a, pb0, pb1);
        mma_f16(st.o[t][2 * g + 1], b, pb0, pb1);
      }
    }
  }
}

// What a warp copies next: its units, W apart in the CTA's share; a depth unit
// is two entries of the ring (K, then V), a unit of rows one.
template <int D>
struct Feed {
  static constexpr int ROW = D / 2, NB = D / 32;
  Place<kKeys> at;
  long long left;  // units of the CTA's share from `at` on
  int part;        // of a depth unit
  int page0, page1;  // pages of the unit's first and second 16 rows

  __device__ __forceinline__ void look_up(const Params& p, int depth_units) {
    page0 = page1 = 0;
    if (left <= 0 || at.off < depth_units) return;
    const int key = (at.off - depth_units) * kKeys;
    const int* row = p.table + (int64_t)at.b * p.max_pages;
    page0 = __ldg(row + key / p.page_size);
    page1 = p.page_size > 16 ? page0 : key + 16 < at.len ? __ldg(row + key / p.page_size + 1) : 0;
  }
  // n units on
  __device__ __forceinline__ void skip(const Params& p, int depth_units, int n) {
    left -= n;
    if (left <= 0) return;
    int off = at.off + n;
    while (off >= at.n) {
      off -= at.n;
      at.next_segment(p, depth_units);
    }
    at.off = off;
  }
  // Starts the next entry's copies into a stage (or nothing at the end); one
  // group of asynchronous copies in any case.
  __device__ __forceinline__ void start(const Params& p, const Mx4Pages& pg, int depth_units,
                                        uint32_t codes, uint32_t scales, int lane) {
    if (left > 0) {
      if (at.off < depth_units) {
        const int l0 = at.off * kDepthKeys;
        const uint8_t* src = (part ? pg.vd : pg.kd) + at.b * pg.depth_b + at.hk * pg.depth_hk +
                             l0 * pg.depth_slot;
        constexpr int VPR = D / 8;  // 16-byte vectors of a row
#pragma unroll
        for (int i = 0; i < kDepthKeys * VPR / 32; ++i) {
          const int r = (i * 32 + lane) / VPR, v = lane % VPR;
          const bool there = l0 + r < p.L;
          cp16(codes + at_bf16<16>(r, v * 8), there ? src + r * pg.depth_slot + v * 16 : src, there);
        }
        if (part == 0) {
          part = 1;
        } else {
          part = 0;
          skip(p, depth_units, kWarps);
          look_up(p, depth_units);
        }
      } else {
        const int key = (at.off - depth_units) * kKeys, rows = at.len - key;
        if (page0 < 0 || page0 >= p.num_pages || page1 < 0 || page1 >= p.num_pages) {
          if (lane == 0) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
          page0 = min(max(page0, 0), p.num_pages - 1);
          page1 = min(max(page1, 0), p.num_pages - 1);
        }
        const int in0 = key % p.page_size;
        const int in1 = p.page_size > 16 ? in0 + 16 : 0;
        const int64_t row[2] = {((int64_t)page0 * p.Hk + at.hk) * p.page_size + in0,
                                ((int64_t)page1 * p.Hk + at.hk) * p.page_size + in1};
        constexpr int RPI = 512 / ROW;  // rows of one copy instruction of a warp
        const int r = lane / (ROW / 16), v = lane % (ROW / 16);
        const uint32_t dst = codes + at_mx4<D>(r, v);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int i = 0; i < 16 / RPI; ++i) {
            const bool there = half * 16 + i * RPI + r < rows;
            const int64_t from = there ? row[half] * ROW + i * 512 + lane * 16 : 0;
            const uint32_t to = dst + (half * 16 + i * RPI) * ROW;
            cp16(to, pg.k + from, there);
            cp16(to + kKeys * ROW, pg.v + from, there);
          }
        // scales: 16-byte vectors of 16 / NB rows
        constexpr int SV = kKeys * NB / 16;  // vectors of the unit, of K or of V
        if (lane < 2 * SV) {
          const int x = lane % SV, first = x * (16 / NB);
          const bool there = first < rows;
          const int64_t from = there ? (first < 16 ? row[0] + first : row[1] + first - 16) * NB : 0;
          cp16(scales + lane * 16, (lane < SV ? pg.k_scale : pg.v_scale) + from, there);
        }
        skip(p, depth_units, kWarps);
        look_up(p, depth_units);
      }
    }
    cp_commit();
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<NT>)
decode_paged_mx4_split(const __grid_constant__ Params p, const __grid_constant__ Mx4Pages pg) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int depth_units = (p.L + kDepthKeys - 1) / kDepthKeys;
  const Work wk = work_of(p.work, p.G, D);

  // the joining kernel may be scheduled now; it waits for this grid to finish
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Share<kKeys> sh = share_of<kKeys, kWarps>(p, depth_units, sm.share);
  if (depth_units == 0) write_empty<D>(p);
  if (sh.u0 >= sh.u1) {
    if (tid == 0) wk.opened[blockIdx.x] = make_int2(-1, 0);
    return;
  }
  const uint32_t codes0 = sm103::smem_u32(&sm.codes[warp][0][0]);
  const uint32_t scales0 = sm103::smem_u32(&sm.scales[warp][0][0][0]);
  constexpr uint32_t kCodes = 2 * kKeys * D / 2, kScales = 2 * kKeys * D / 32;

  Feed<D> feed;
  feed.at = sh.at;
  feed.left = sh.u1 - sh.u0;
  feed.part = 0;
  feed.skip(p, depth_units, warp);
  feed.look_up(p, depth_units);
  int in = 0, out = 0;  // stages to fill and to read next
  auto fill = [&] {
    feed.start(p, pg, depth_units, codes0 + in * kCodes, scales0 + in * kScales, lane);
    in = in + 1 == kNS ? 0 : in + 1;
  };
#pragma unroll
  for (int i = 0; i < kNS - 1; ++i) fill();
  // the oldest entry has landed, and the stage read before it is filled again
  auto next = [&]() -> int {
    cp_wait<kNS - 2>();
    __syncwarp();
    fill();
    const int s = out;
    out = out + 1 == kNS ? 0 : out + 1;
    return s;
  };

  Place<kKeys> at = sh.at;
  State<D, NT> st;
  long long left = sh.u1 - sh.u0;
  int turn = 0;  // the warp that takes the unit at `at`
  bool opened = false;
  while (left > 0) {
    const int cnt = (int)min(left, (long long)(at.n - at.off));
    const int end = at.off + cnt;
    const bool cut_before = at.off > 0, cut_after = end < at.n;
    const __nv_bfloat16* q = p.q + ((int64_t)at.b * p.Hk + at.hk) * p.G * D;
    st.clear();
    int off = at.off + ((warp - turn) & (kWarps - 1));
    if (off < min(end, depth_units)) {
      uint32_t qb[NT][D / 16][2], pb[NT][2];
      load_q_bf16<D, NT>(qb, q, p.G, lane);
      for (; off < min(end, depth_units); off += kWarps) {
        int s = next();
        depth_scores<D, NT>(st, qb, codes0 + s * kCodes, p.L - off * kDepthKeys, p.scale_log2, lane, pb);
        s = next();
        depth_values<D, NT>(st, pb, codes0 + s * kCodes, lane);
      }
    }
    if (off < end) {
      uint32_t qb[NT][D / 32][4];
      float back[NT][2];
      load_q_f16<D, NT>(qb, back, q, p.G, p.scale_log2, lane);
      for (; off < end; off += kWarps) {
        const int s = next();
        const int there = at.len - (off - depth_units) * kKeys;
        const uint32_t kb = codes0 + s * kCodes, ks = scales0 + s * kScales;
        if (there >= kKeys)
          unit_mx4<D, NT, false>(st, qb, back, kb, kb + kCodes / 2, ks, ks + kScales / 2, there, lane);
        else
          unit_mx4<D, NT, true>(st, qb, back, kb, kb + kCodes / 2, ks, ks + kScales / 2, there, lane);
      }
    }
    leave<D, NT, kWarps>(p, wk, sm.merge, st, cut_before || cut_after,
                         2 * blockIdx.x + (cut_before ? 0 : 1),
                         ((int64_t)at.b * p.Hk + at.hk) * p.G,
                         [&](float* m0, float* m1, int t, int half) {
#pragma unroll
                           for (int g = 0; g < kCols / 32; ++g) {
                             const float(&x)[4] = st.o[t][half * 4 + 2 * g];
                             const float(&y)[4] = st.o[t][half * 4 + 2 * g + 1];
                             const int d = g * 32 + (lane >> 2) * 4;
                             *reinterpret_cast<float4*>(m0 + d) = make_float4(x[0], x[2], y[0], y[2]);
                             *reinterpret_cast<float4*>(m1 + d) = make_float4(x[1], x[3], y[1], y[3]);
                           }
                         });
    if (cut_after && !cut_before) {
      opened = true;
      if (tid == 0) {
        const long long last = sh.u1 - left + (at.n - at.off) - 1;  // of the segment
        wk.opened[blockIdx.x] =
            make_int2(at.b * p.Hk + at.hk, owner_of(sh, last) - (int)blockIdx.x + 1);
      }
    }
    left -= cnt;
    turn = (turn + cnt) & (kWarps - 1);
    if (left > 0) at.next_segment(p, depth_units);
  }
  if (tid == 0 && !opened) wk.opened[blockIdx.x] = make_int2(-1, 0);
}

template <int D, int NT>
cudaError_t launch(const DecodePagedArgs& a, cudaStream_t stream) {
  const PagedKv& c = a.c;
  const Mx4Pages pg{(const uint8_t*)c.k,       (const uint8_t*)c.v,
                    (const uint8_t*)c.k_scale, (const uint8_t*)c.v_scale,
                    (const uint8_t*)a.kd,      (const uint8_t*)a.vd,
                    a.depth_b_stride * 2,      a.depth_hk_stride * 2,
                    a.depth_slot_stride * 2};
  cudaError_t e = cudaFuncSetAttribute(decode_paged_mx4_split<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  int grid = a.num_sms * kCtasPerSm<NT>;
  grid = grid < kMaxCtas ? grid : kMaxCtas;
  decode_paged_mx4_split<D, NT><<<grid, kWarps * 32, sizeof(Smem<D>), stream>>>(params_of(a), pg);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join(a, grid, stream);
}

}  // namespace

cudaError_t launch_mx4(const DecodePagedArgs& a, cudaStream_t stream) {
  if (a.c.d == 128) return a.G <= 8 ? launch<128, 1>(a, stream) : launch<128, 2>(a, stream);
  return a.G <= 8 ? launch<64, 1>(a, stream) : launch<64, 2>(a, stream);
}

}  // namespace paged
}  // namespace moda
