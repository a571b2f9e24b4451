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
//     conversion gives their fp16 pair. V's block scales go into P (in fp32, then
//     rounded to fp16, State4), one P^T per block of 32 columns.
// Measured (d = 128): 64 ragged sequences of up to 32768 rows at G = 8, 584 MB,
// 123 us, 675 instructions a unit; the same rows in TMA boxes with a producer
// warp and four codes to a load took 226. 16 sequences of
// up to 999 rows (d = 64, 8 KV heads, G = 8), in clusters of three, 7.3 us.
// Each warp streams units of its own (32 rows, or 16 depth slots) through its
// own ring of shared-memory stages by asynchronous copies: no barrier between
// warps but at the end of a segment.
#include <cuda_fp16.h>
#include <float.h>

#include "decode_paged.cuh"

namespace moda {
namespace paged {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32;       // cached rows of a unit
constexpr int kDepthKeys = 16;  // depth slots of a unit; their K and V take a stage each
constexpr int kNS = 3;          // stages of a warp
// Entering and leaving a segment, in units. (4 KV heads, 64 ragged sequences of up
// to 32768 rows, G = 8, at 6, 10, 14, 18: 123.6, 123.3, 123.9, 124.6 us; of up to
// 8000, G = 16, 139 MB: 67, 56.3, 55.1, 56.1.)
template <int D, int NT>
constexpr int kCost = NT == 1 ? (D == 128 ? 10 : 12) : 14;
// 168 registers (two head tiles: 255): four at 128 registers were 6 % slower
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
constexpr int kGroupUnits = 21, kClusterUnits = 8;  // see group_of

// A stage: codes of K and of V (or kDepthKeys bf16 rows of one of the two),
// then their scales.
template <int D>
struct Stage {
  static constexpr uint32_t kRow = D / 2, kBlocks = D / 32;  // bytes of a row
  static constexpr uint32_t kV = kKeys * kRow;
  static constexpr uint32_t kKs = 2 * kV, kVs = kKs + kKeys * kBlocks;
  static constexpr uint32_t kBytes = kVs + kKeys * kBlocks;
};
template <int D>
struct Smem {
  uint8_t ring[kWarps][kNS][Stage<D>::kBytes];
  MergeSmem<kWarps, D> merge;
  ShareSmem<kWarps> share;
};

struct Mx4Pages {
  const uint8_t *k, *v, *k_scale, *v_scale;
  const uint8_t *kd, *vd;  // depth slots, bf16
  int64_t depth_b, depth_hk, depth_slot;  // bytes
};

// Weights are held in fp32 as p = 2^(score - m), for the sum l, and as p c, which
// times a block scale of V goes into the products with fp16's range. m is the
// scores' alone: what a row weighs in l has nothing to do with its values. (One
// reference for both, the score's plus the values' exponent, lost rows of zeros
// from l beside values of 2^60.) c is a factor of the head that puts the
// largest product so far at 2^kTop when it is set, and is set again when a product
// passes 2^kMost: products stay in fp16's range, and as the largest is 2^kTop at
// least, keep their 11 bits down to 2^-21 of it and lose at most 2^-32 of it below
// (2^-31 beside values of 2^100 and more, where p c has few bits left in fp32).
// One rounding to fp16 is a choice: with what it leaves in a second part and two
// more products, 64 ragged sequences take 141 us instead of 123, and o, against 64
// bits, is off by 1.667e-3 of its norm instead of 1.670e-3 (o's own rounding to bf16).
// m is raised when a lane's four weights sum to more than kMostWeight.
constexpr float kTop = 7.f;
constexpr float kMost = 0x1p15f;
constexpr float kMostWeight = 0x1p8f;

template <int D, int NT>
struct State4 : State<D, NT> {
  using State<D, NT>::m;
  using State<D, NT>::l;
  using State<D, NT>::o;  // sums of p c times values
  float c[NT][2];
  // m from the least of all scores, for which the first key's weight is infinite.
  __device__ __forceinline__ void clear() {
    State<D, NT>::clear();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -FLT_MAX;
      c[t][0] = c[t][1] = 1.f;
    }
  }
  // x: N scores over `back`, of head 2c at even and 2c + 1 at odd places, two to
  // a key; v: the largest block scale of each key's values (a power of two).
  // Adds the keys to l and leaves p c in w.
  template <int N>
  __device__ __forceinline__ void weigh(int t, const float (&x)[N], const float (&back)[2],
                                        const float (&v)[N / 2], float (&w)[N]) {
    float sum[2], most[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int i = e; i < N; i += 2) w[i] = sm103::ex2_approx(fmaf(x[i], back[e], -m[t][e]));
      add_up<N>(t, e, v, w, sum[e], most[e]);
    }
    if (__any_sync(0xffffffffu, most[0] > kMost || most[1] > kMost || sum[0] > kMostWeight || sum[1] > kMostWeight)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rebase<N>(t, e, x, back[e], v, w);
        add_up<N>(t, e, v, w, sum[e], most[e]);
      }
    }
    l[t][0] += sum[0];
    l[t][1] += sum[1];
  }
  // The sum of head 2c + e's weights, then w = p c and the largest product.
  template <int N>
  __device__ __forceinline__ void add_up(int t, int e, const float (&v)[N / 2], float (&w)[N], float& sum,
                                         float& most) const {
    sum = w[e] + w[e + 2];
#pragma unroll
    for (int i = 4; i < N; i += 4) sum += w[i + e] + w[i + e + 2];
    most = 0.f;
#pragma unroll
    for (int i = e; i < N; i += 2) {
      w[i] *= c[t][e];
      most = fmaxf(most, w[i] * v[i >> 1]);
    }
  }
  // m to cover the scores and c the products, where these are more than before;
  // l and o follow. (m - log2(c) is what o is relative to.) As no row's values are
  // counted below 2^-80 or above 2^125, c is between 2^-118 and 2^95. Leaves p in w.
  // Works with scores rounded as m is and their differences: the fused product of
  // weigh keeps what m was rounded by, which is 2^7 at scores of 2^31.
  template <int N>
  __device__ __forceinline__ void rebase(int t, int e, const float (&x)[N], float back, const float (&v)[N / 2],
                                         float (&w)[N]) {
    auto most = [](float a) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
      return a;
    };
    float s = -INFINITY, z = -INFINITY;
#pragma unroll
    for (int i = e; i < N; i += 2) {
      w[i] = __fmul_rn(x[i], back);
      s = fmaxf(s, w[i]);
    }
    const float m1 = fmaxf(m[t][e], most(s)), raised = m[t][e] - m1;
#pragma unroll
    for (int i = e; i < N; i += 2) {
      w[i] -= m1;
      z = fmaxf(z, w[i] + (__uint_as_float(0x4b000000u | (__float_as_uint(v[i >> 1]) >> 23)) -
                           (8388608.f + 127.f + kTop)));  // v's exponent as a float, by way of 2^23
      w[i] = sm103::ex2_approx(w[i]);
    }
    const float r0 = raised - __log2f(c[t][e]), r1 = fmaxf(r0, most(z));
    const float a = sm103::ex2_approx(r0 - r1);
    l[t][e] *= sm103::ex2_approx(raised);
    c[t][e] = sm103::ex2_approx(-r1);
    m[t][e] = m1;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      o[t][i][e] *= a;
      o[t][i][e + 2] *= a;
    }
  }
};

// Byte offset of 16-byte vector `v` (block v of 32 codes) of row r, placed so
// that none of these meet in a bank: whole rows side by side (the copies), 8
// rows in a row (V's transposing loads), rows 4i and 4i + 1, or 4i + 2 and
// 4i + 3, of 16 (K's words).
template <int D>
__device__ __forceinline__ uint32_t at_mx4(int r, int v) {
  return D == 128 ? (uint32_t)(r * 64 + ((v ^ ((r >> 1) & 3) ^ ((r >> 3) & 1)) << 4))
                  : (uint32_t)((r ^ ((r >> 2) & 2)) * 32 + ((v ^ ((r >> 2) & 1)) << 4));
}
// The key that MMA index i (a row of K, a column of V^T) of a 16-key tile
// stands for: a lane's columns 2c, 2c + 1, 2c + 8, 2c + 9 of V^T are the four
// keys in a row that the transposing load gives it.
__device__ __forceinline__ int key_of(int i) {
  return ((i & 6) << 1) | ((i & 8) >> 2) | (i & 1);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// The bits of a where m has ones, of b elsewhere.
__device__ __forceinline__ uint32_t choose_bits(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(a), "r"(b), "r"(m));
  return r;
}
// Two 16x16 byte matrices (16 rows of 16 bytes at the addresses of lanes 0-15
// and 16-31) transposed: lane (r0, c) gets of each matrix the bytes of rows
// 4c .. 4c + 3 in column r0 (first register) and r0 + 8 (second).
__device__ __forceinline__ void ldsm_t_bytes(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
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
// Those of bytes 1 and 3 alone.
__device__ __forceinline__ void odd_codes_to_f16(uint32_t w, uint32_t& r1, uint32_t& r3) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %2;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b;\n cvt.rn.f16x2.e2m1x2 %1, d;\n}\n"
      : "=r"(r1), "=r"(r3)
      : "r"(w));
}
// The scale bytes of a row's blocks as powers of two (255: infinity). A byte
// at a time: the load unit and the multiplier have room, the ALU has not.
template <int NB>
__device__ __forceinline__ void load_scales(uint32_t addr, float (&f)[NB]) {
#pragma unroll
  for (int g = 0; g < NB; ++g) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr + g));
    f[g] = __uint_as_float(v * (1u << 23));
  }
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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
      if (h < G) raw[g] = *(reinterpret_cast<const uint4*>(q + (int64_t)h * D + g * 32) + c);
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
    // (never 0: the rows that do not exist carry -infinity times it)
    const float mine = fmaxf(scale_log2 * __uint_as_float((uint32_t)(127 - 14 + e) << 23), 0x1p-126f);
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

// Weights of 16 depth slots, as B tiles of O^T += V^T P^T: bf16 and the rest.
template <int D, int NT>
__device__ __forceinline__ void depth_scores(State4<D, NT>& st, const uint32_t (&qb)[NT][D / 16][2],
                                             uint32_t kb, int there, float scale_log2, int lane,
                                             uint32_t (&pb)[NT][2], uint32_t (&pl)[NT][2]) {
  const int lr = lane & 7, lm = lane >> 3;
  float s[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    uint32_t a[4];
    wmma16::ldsm_x4(kb + at_bf16<16>(key_of((lm & 1) * 8 + lr), ks * 16 + (lm >> 1) * 8), a[0], a[1],
                    a[2], a[3]);
#pragma unroll
    for (int t = 0; t < NT; ++t) wmma16::mma_bf16(s[t], a, qb[t][ks][0], qb[t][ks][1]);
  }
  const int ka = key_of(lane >> 2);
  const bool k0 = ka < there, k1 = ka + 2 < there;
  const float back[2] = {scale_log2, scale_log2}, v[2] = {1.f, 1.f};  // their values in bf16 have their own range
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (!k0) s[t][0] = s[t][1] = -INFINITY;
    if (!k1) s[t][2] = s[t][3] = -INFINITY;
    float w[4];
    st.template weigh<4>(t, s[t], back, v, w);
    weights_bf16(w[0], w[1], pb[t][0], pl[t][0]);
    weights_bf16(w[2], w[3], pb[t][1], pl[t][1]);
  }
}

// Their values, in this kernel's order of O's rows: of block g, tile 2g holds
// d = 32 g + 2 r0 in row r0 and 32 g + 16 + 2 r0 in r0 + 8, tile 2g + 1 the
// elements after them. Rows past L are zeros.
template <int D, int NT>
__device__ __forceinline__ void depth_values(State4<D, NT>& st, const uint32_t (&pb)[NT][2],
                                             const uint32_t (&pl)[NT][2], uint32_t vb, int lane) {
  const int r0 = lane >> 2, v0 = 4 * (lane & 3);
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = g * 32 + h * 16 + r0 * 2;
      const uint32_t x0 = lds32(vb + at_bf16<16>(v0, col)), x1 = lds32(vb + at_bf16<16>(v0 + 1, col));
      const uint32_t x2 = lds32(vb + at_bf16<16>(v0 + 2, col)), x3 = lds32(vb + at_bf16<16>(v0 + 3, col));
      a[h] = __byte_perm(x0, x1, 0x5410);
      a[h + 2] = __byte_perm(x2, x3, 0x5410);
      b[h] = __byte_perm(x0, x1, 0x7632);
      b[h + 2] = __byte_perm(x2, x3, 0x7632);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wmma16::mma_bf16(st.o[t][2 * g], a, pb[t][0], pb[t][1]);
      wmma16::mma_bf16(st.o[t][2 * g], a, pl[t][0], pl[t][1]);
      wmma16::mma_bf16(st.o[t][2 * g + 1], b, pb[t][0], pb[t][1]);
      wmma16::mma_bf16(st.o[t][2 * g + 1], b, pl[t][0], pl[t][1]);
    }
  }
}

// A lane's places in a stage, the same for every unit.
template <int D>
struct Lane {
  static constexpr int NB = D / 32;
  uint32_t k[2][NB];    // codes of block g of its keys in a tile's rows r0 and r0 + 8
  uint32_t v[NB / 2];   // row of V's transposing load of blocks 2g and 2g + 1
  uint32_t scale;       // of its first key
  uint32_t copy, copy8; // of its vector in 8 rows from row 0, and from row 8 (D = 128)
  __device__ __forceinline__ explicit Lane(int lane) {
    const int c = lane & 3, ka = key_of(lane >> 2);
#pragma unroll
    for (int g = 0; g < NB; ++g) {
      k[0][g] = at_mx4<D>(ka, g) + c * 4;
      k[1][g] = at_mx4<D>(ka + 2, g) + c * 4;
    }
#pragma unroll
    for (int g = 0; g < NB; g += 2)
      v[g / 2] = Stage<D>::kV + at_mx4<D>(lane & 15, g + (lane >> 4));
    scale = Stage<D>::kKs + ka * NB;
    copy = at_mx4<D>(lane / NB, lane % NB);
    copy8 = at_mx4<D>(lane / NB + 8, lane % NB);
  }
};

// The 32 rows of a unit (in the stage at `sb`) into the state, two tiles of 16
// keys side by side. TAIL: only `there` of them exist.
template <int D, int NT, bool TAIL>
__device__ __forceinline__ void unit_mx4(State4<D, NT>& st, const uint32_t (&qb)[NT][D / 32][4],
                                         const float (&back)[NT][2], const Lane<D>& at, uint32_t sb, int there,
                                         int lane) {
  using S = Stage<D>;
  constexpr int NB = S::kBlocks;
  // this lane's keys: ka + 16 j + 2 i, rows r0 + 8 i of tile j
  const int ka = key_of(lane >> 2);
  auto key = [&](int n) { return ka + 16 * (n >> 1) + 2 * (n & 1); };
  float s[2][NT][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float f[2][NB];
    load_scales<NB>(sb + at.scale + (16 * j) * NB, f[0]);
    load_scales<NB>(sb + at.scale + (16 * j + 2) * NB, f[1]);
#pragma unroll
    for (int g = 0; g < NB; ++g) {
      uint32_t a[4], b[4];  // two k-steps of 16
      const uint32_t tile = sb + j * 16 * S::kRow;
      codes_to_f16(lds32(tile + at.k[0][g]), a[0], a[2], b[0], b[2]);
      codes_to_f16(lds32(tile + at.k[1][g]), a[1], a[3], b[1], b[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4];
        mma_f16_first(x, a, qb[t][g][0], qb[t][g][1]);
        mma_f16(x, b, qb[t][g][2], qb[t][g][3]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[j][t][i] = g == 0 ? x[i] * f[i >> 1][g] : fmaf(x[i], f[i >> 1][g], s[j][t][i]);
      }
    }
  }
  // V's scales, and each row's largest, 2^-80 at least, so that c stays in range.
  // A block stored as NaN (its codes are 0, and 0 times infinity is NaN) leaves
  // the other blocks' alone.
  float f[4][NB], e[4];
  uint32_t dead = 0;  // bit n: this lane's key n does not exist
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    load_scales<NB>(sb + at.scale + kKeys * NB + (16 * (n >> 1) + 2 * (n & 1)) * NB, f[n]);
    if (TAIL && key(n) >= there) {
      dead |= 1u << n;
#pragma unroll
      for (int g = 0; g < NB; ++g) f[n][g] = 1.f;  // it may be any byte: weight 0 times 1
    }
    e[n] = 0x1p-80f;
#pragma unroll
    for (int g = 0; g < NB; ++g) e[n] = fmaxf(e[n], f[n][g]);
  }
  if (__any_sync(0xffffffffu, fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])) == INFINITY)) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      e[n] = 0x1p-80f;
#pragma unroll
      for (int g = 0; g < NB; ++g)
        if (f[n][g] < INFINITY) e[n] = fmaxf(e[n], f[n][g]);
    }
  }
  float w[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = s[i >> 2][t][i & 3];
      if (TAIL && (dead >> (i >> 1) & 1u)) x[i] = -INFINITY;
    }
    st.template weigh<8>(t, x, back[t], e, w[t]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int g2 = 0; g2 < NB; g2 += 2) {
      uint32_t raw[4];  // blocks g2 and g2 + 1: bytes of 4 keys, columns r0 and r0 + 8
      ldsm_t_bytes(sb + j * 16 * S::kRow + at.v[g2 / 2], raw);
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) {
        const int g = g2 + gi;
        // a byte holds elements 2r and 2r + 1 of one key: put the same element
        // of keys 0, 1 into byte 1 and of keys 2, 3 into byte 3 (left shifts
        // only, which the multiplier does)
        uint32_t a[4], b[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = raw[2 * gi + h], x4 = x * 16u, x8 = x * 256u;
          odd_codes_to_f16(choose_bits(x8, x4, 0x0f000f00u), a[h], a[h + 2]);
          odd_codes_to_f16(choose_bits(x4, x, 0x0f000f00u), b[h], b[h + 2]);
        }
        const float f0 = f[2 * j][g], f1 = f[2 * j + 1][g];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float* p = w[t] + 4 * j;
          const uint32_t pb0 = wmma16::movmatrix_t(pack_f16(p[0] * f0, p[1] * f0));
          const uint32_t pb1 = wmma16::movmatrix_t(pack_f16(p[2] * f1, p[3] * f1));
          mma_f16(st.o[t][2 * g], a, pb0, pb1);
          mma_f16(st.o[t][2 * g + 1], b, pb0, pb1);
        }
      }
    }
}

// What a warp copies next: its units, kWarps apart in the CTA's share; a depth
// unit is two entries of the ring (K, then V), a unit of rows one.
template <int D>
struct Feed {
  using S = Stage<D>;
  static constexpr int ROW = S::kRow, NB = S::kBlocks;
  static constexpr int kStep = kWarps * kKeys;  // rows from one unit of a warp to its next
  Place<kKeys> at;
  int left;  // units of the CTA's share from `at` on
  int part;  // of a depth unit
  int run;   // units of rows from `at` on, all whole, with another one of the segment after each
  const int* pages;   // the table's entry of the unit's first 16 rows
  uint32_t in_page;   // their place in the page: the same for all units of a segment,
                      // since page sizes divide kStep
  int page0, page1;   // pages of the unit's first and second 16 rows

  // The unit at `at`, from nothing.
  __device__ __forceinline__ void enter(const Params& p, int depth_units) {
    run = 0;
    page0 = page1 = 0;
    if (left <= 0 || at.off < depth_units) return;
    const int key = (at.off - depth_units) * kKeys;
    pages = p.table + (int64_t)at.b * p.max_pages + (key >> p.page_shift);
    in_page = key & ((1 << p.page_shift) - 1);
    page0 = pages[0];
    page1 = p.page_shift > 4 ? page0 : key + 16 < at.len ? pages[1] : 0;
    run = min((min(at.n, at.off + left) - 1 - at.off) / kWarps, (at.len - key) / kStep);
  }
  __device__ __forceinline__ void begin(const Params& p, int depth_units, const Share<kKeys>& sh,
                                        int first) {
    at = sh.at;
    left = sh.n;
    part = 0;
    skip(p, depth_units, first);
    enter(p, depth_units);
  }
  // n units on
  __device__ __forceinline__ void skip(const Params& p, int depth_units, int n) {
    left -= n;
    at.off += n;
    if (at.off < at.n || left <= 0) return;
    int off = at.off;
    do {
      off -= at.n;
      at.next_segment(p, depth_units);
    } while (off >= at.n);
    at.off = off;
  }
  // The rows of the unit at `at`; TAIL: only `rows` of them are read, the
  // others become zeros.
  template <bool TAIL>
  __device__ __forceinline__ void copy_rows(const Params& p, const Mx4Pages& pg, const Lane<D>& to,
                                            uint32_t stage, int rows, int lane) {
    if ((unsigned)page0 >= (unsigned)p.num_pages || (unsigned)page1 >= (unsigned)p.num_pages) {
      if (lane == 0) atomicCAS(p.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
      page0 = min(max(page0, 0), p.num_pages - 1);
      page1 = min(max(page1, 0), p.num_pages - 1);
    }
    // row numbers in the pool fit 31 bits
    const uint32_t row0 = (((uint32_t)page0 * p.Hk + at.hk) << p.page_shift) + in_page;
    const uint32_t row1 = p.page_shift > 4 ? row0 + 16 : ((uint32_t)page1 * p.Hk + at.hk) << 4;
    constexpr int RPI = 512 / ROW;  // rows of one copy instruction of a warp
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t from = (int64_t)(half ? row1 : row0) * ROW + lane * 16;
#pragma unroll
      for (int i = 0; i < 16 / RPI; ++i) {
        const bool there = !TAIL || half * 16 + i * RPI + lane / NB < rows;
        const int64_t src = there ? from + i * 512 : 0;
        const uint32_t dst = stage + half * 16 * ROW + (i ? to.copy8 : to.copy);
        cp16(dst, pg.k + src, there);
        cp16(dst + S::kV, pg.v + src, there);
      }
    }
    // scales: 16-byte vectors of 16 / NB rows
    constexpr int SV = kKeys * NB / 16;  // vectors of the unit, of K or of V
    if (lane < 2 * SV) {
      const int first = lane % SV * (16 / NB);
      const bool there = !TAIL || first < rows;
      const int64_t src = there ? (int64_t)(first < 16 ? row0 + first : row1 + first - 16) * NB : 0;
      cp16(stage + S::kKs + lane * 16, (lane < SV ? pg.k_scale : pg.v_scale) + src, there);
    }
  }
  // Starts the next entry's copies into a stage (or nothing at the end); one
  // group of asynchronous copies in any case.
  __device__ __forceinline__ void start(const Params& p, const Mx4Pages& pg, int depth_units,
                                        const Lane<D>& to, uint32_t stage, int lane) {
    if (run > 0) {
      copy_rows<false>(p, pg, to, stage, kKeys, lane);
      --run;
      at.off += kWarps;
      left -= kWarps;
      pages += kStep >> p.page_shift;
      page0 = pages[0];
      // past the sequence's end there is no page to look up
      page1 = p.page_shift > 4 ? page0
              : (at.off - depth_units) * kKeys + 16 < at.len ? pages[1] : 0;
    } else if (left > 0) {
      if (at.off < depth_units) {
        const int l0 = at.off * kDepthKeys;
        const uint8_t* src = (part ? pg.vd : pg.kd) + at.b * pg.depth_b + at.hk * pg.depth_hk +
                             l0 * pg.depth_slot;
        constexpr int VPR = D / 8;  // 16-byte vectors of a row
#pragma unroll
        for (int i = 0; i < kDepthKeys * VPR / 32; ++i) {
          const int r = (i * 32 + lane) / VPR, v = lane % VPR;
          const bool there = l0 + r < p.L;
          cp16(stage + at_bf16<16>(r, v * 8), there ? src + r * pg.depth_slot + v * 16 : src, there);
        }
        part ^= 1;
        if (part == 0) {
          skip(p, depth_units, kWarps);
          enter(p, depth_units);
        }
      } else {
        copy_rows<true>(p, pg, to, stage, at.len - (at.off - depth_units) * kKeys, lane);
        skip(p, depth_units, kWarps);
        enter(p, depth_units);
      }
    }
    cp_commit();
  }
};

template <int D, int NT, Split SPLIT>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<NT>)
decode_paged_mx4_split(const __grid_constant__ Params p, const __grid_constant__ Mx4Pages pg) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int depth_units = (p.L + kDepthKeys - 1) / kDepthKeys;
  const Work wk = work_of(p.work, p.G, D);

  wait_for_stream();
  constexpr bool GROUP = SPLIT == Split::kGroup;
  Share<kKeys> sh;
  if constexpr (GROUP) {
    sh = share_of_segment<kKeys>(p, depth_units);
    if (sh.at.n == 0) return write_empty_segment<D>(p, sh.at.b, sh.at.hk);
  } else {
    if constexpr (SPLIT == Split::kOne)
      sh = share_of_one<kKeys, kCost<D, NT>, kWarps>(p, depth_units);
    else
      sh = share_of<kKeys, kWarps, kCost<D, NT>, kWarps>(p, depth_units, sm.share);
    if (depth_units == 0) write_empty<D>(p);
    if (sh.n == 0) {
      if (tid == 0) wk.opened[blockIdx.x] = make_int2(-1, 0);
      return;
    }
  }
  const uint32_t ring = sm103::smem_u32(&sm.ring[warp][0][0]);
  constexpr uint32_t kRing = kNS * Stage<D>::kBytes;

  const Lane<D> to(lane);
  Feed<D> feed;
  feed.begin(p, depth_units, sh, warp);
  uint32_t in = 0, out = 0;  // stages to fill and to read next
  auto fill = [&] {
    feed.start(p, pg, depth_units, to, ring + in, lane);
    in = in + Stage<D>::kBytes == kRing ? 0 : in + Stage<D>::kBytes;
  };
#pragma unroll 1
  for (int i = 0; i < kNS - 1; ++i) fill();
  // the oldest entry has landed, and the stage read before it is filled again
  auto next = [&]() -> uint32_t {
    cp_wait<kNS - 2>();
    __syncwarp();
    fill();
    const uint32_t s = ring + out;
    out = out + Stage<D>::kBytes == kRing ? 0 : out + Stage<D>::kBytes;
    return s;
  };

  Place<kKeys> at = sh.at;
  GroupSmem<D, kWarps>& last = *reinterpret_cast<GroupSmem<D, kWarps>*>(sm.ring);  // when the rings are free
  static_assert(sizeof(GroupSmem<D, kWarps>) <= sizeof(sm.ring));
  const int64_t first_row = ((int64_t)at.b * p.Hk + at.hk) * p.G;
  State4<D, NT> st;
  int left = sh.n;
  int turn = 0;  // the warp that takes the unit at `at`
  bool opened = false;
  long long seg_end = sh.end;
  while (GROUP || left > 0) {  // (a group's CTA leaves a state even if it has no unit)
    const int cnt = min(left, at.n - at.off);
    const int end = at.off + cnt;
    const bool cut_before = at.off > 0, cut_after = end < at.n;
    const __nv_bfloat16* q = p.q + ((int64_t)at.b * p.Hk + at.hk) * p.G * D;
    st.clear();
    int off = at.off + ((warp - turn) & (kWarps - 1));
    if (off < min(end, depth_units)) {
      uint32_t qb[NT][D / 16][2], pb[NT][2], pl[NT][2];
      load_q_bf16<D, NT>(qb, q, p.G, lane);
      for (; off < min(end, depth_units); off += kWarps) {
        uint32_t s = next();
        depth_scores<D, NT>(st, qb, s, p.L - off * kDepthKeys, p.scale_log2, lane, pb, pl);
        s = next();
        depth_values<D, NT>(st, pb, pl, s, lane);
      }
    }
    if (off < end) {
      uint32_t qb[NT][D / 32][4];
      float back[NT][2];
      load_q_f16<D, NT>(qb, back, q, p.G, p.scale_log2, lane);
      // whole units, then the sequence's last one if it is not
      // (one place that asks for the next entry: with two the kernel was so long that
      // 100 sequences of up to 1000 rows took 39.3 us instead of 37.2)
      const int whole = min(end, depth_units + at.len / kKeys);
      for (; off < end; off += kWarps) {
        const uint32_t s = next();
        if (off < whole)
          unit_mx4<D, NT, false>(st, qb, back, to, s, kKeys, lane);
        else
          unit_mx4<D, NT, true>(st, qb, back, to, s, at.len % kKeys, lane);
      }
    }
    const auto put = [&](float* m0, float* m1, int t, int part, const auto& buf) {
      constexpr int kBlocks = std::remove_reference_t<decltype(buf)>::kCols / 32;
      const float u0 = __fdividef(1.f / kUnit4, st.c[t][0]), u1 = __fdividef(1.f / kUnit4, st.c[t][1]);
#pragma unroll
      for (int g = 0; g < kBlocks; ++g) {
        const float(&x)[4] = st.o[t][2 * (part * kBlocks + g)];
        const float(&y)[4] = st.o[t][2 * (part * kBlocks + g) + 1];
        const int d = g * 32 + (lane >> 2) * 2;
        *reinterpret_cast<float2*>(m0 + d) = make_float2(x[0] * u0, y[0] * u0);
        *reinterpret_cast<float2*>(m1 + d) = make_float2(x[1] * u1, y[1] * u1);
        *reinterpret_cast<float2*>(m0 + d + 16) = make_float2(x[2] * u0, y[2] * u0);
        *reinterpret_cast<float2*>(m1 + d + 16) = make_float2(x[3] * u1, y[3] * u1);
      }
    };
    if constexpr (GROUP) {
      leave<D, NT>(p, sm.merge, st, p.group > 1, &last.o[0][0], &last.ml[0][0], 0, first_row, put);
      if (p.group > 1) join_group<D, kWarps>(p, last, first_row);
      return;
    }
    const int slot = 2 * blockIdx.x + (cut_before ? 0 : 1);
    const int64_t row0 = ((int64_t)at.b * p.Hk + at.hk) * p.G;
    leave<D, NT>(p, sm.merge, st, cut_before || cut_after, wk.o, wk.ml, slot, row0, put);
    if (cut_after && !cut_before) {
      opened = true;
      if (tid == 0)
        wk.opened[blockIdx.x] =
            make_int2(at.b * p.Hk + at.hk, sh.owner_of(seg_end - 1) - (int)blockIdx.x + 1);
    }
    left -= cnt;
    turn = (turn + cnt) & (kWarps - 1);
    if (left > 0) {
      at.next_segment(p, depth_units);
      seg_end += kCost<D, NT> + at.n;
    }
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
  int grid = a.num_sms * kCtasPerSm<NT>;
  grid = grid < kMaxCtas ? grid : kMaxCtas;
  const int max_units =
      (a.L + kDepthKeys - 1) / kDepthKeys + (c.max_pages * c.page_size + kKeys - 1) / kKeys;
  const int group = group_of(a, max_units, grid, kGroupUnits, kClusterUnits);
  const auto kernel = group        ? decode_paged_mx4_split<D, NT, Split::kGroup>
                      : c.B == 1 ? decode_paged_mx4_split<D, NT, Split::kOne>
                                 : decode_paged_mx4_split<D, NT, Split::kShares>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  if (group > 8) {  // beyond the portable size
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  if (group)
    return launch_dependent_clusters(kernel, dim3(c.B * c.Hk * group), group, kWarps * 32, sizeof(Smem<D>),
                                     stream, params_of(a, group), pg);
  e = launch_dependent(kernel, dim3(grid), kWarps * 32, sizeof(Smem<D>), stream, params_of(a, 0), pg);
  return e != cudaSuccess ? e : launch_join(a, grid, stream);
}

}  // namespace

cudaError_t launch_mx4(const DecodePagedArgs& a, cudaStream_t stream) {
  if (a.c.d == 128) return a.G <= 8 ? launch<128, 1>(a, stream) : launch<128, 2>(a, stream);
  return a.G <= 8 ? launch<64, 1>(a, stream) : launch<64, 2>(a, stream);
}

}  // namespace paged
}  // namespace moda
