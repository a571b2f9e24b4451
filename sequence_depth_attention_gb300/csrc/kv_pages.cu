// Rows into and out of the paged KV cache (layouts in include/moda.h).
//
// append  q and k are turned in pairs, (a, b) -> (a c - b s, b c + a s), with
//         the cosines and sines of the token's position; k and v go into the
//         page row of (sequence, position), as bf16 or as microscaled 4-bit.
// gather  the rows back as dense bf16.
//
// Both are HBM-bound, with little arithmetic between a load and its store:
// what counts is how many warps have their loads on the way. An append's warp
// takes one token and a handful of its heads, 2 KB of rows, and asks for them
// before it knows where they go.
//   Turning: a lane owns two 16-byte vectors of a head, the two halves of 8
//   pairs (or two vectors of 4 interleaved pairs each), so that 16 values of
//   the table turn 16 elements and no lane needs another's; d/16 lanes a head.
//   4-bit rows: a lane owns one 16-byte vector, four lanes a block of 32; the
//   halves of k's pairs come by shuffle. k is turned in fp32, and again with a
//   sticky bit only where that could change a code or a scale.
// Measured: a prompt of 16384 tokens (Hq 16, Hk 4, d 128, 227 MB) 35.4 us, 96 %
// of the copy bandwidth; two vectors a lane on the way instead of four 41 us. Into
// 4-bit pages (193 MB) 41.4 us, where issue slots are 66 % and the ALU 59 % busy.
// 16001 4-bit rows of 4 heads gathered, 42 MB, 11 us (an elementwise kernel over
// as many bytes takes 10.4); as many bf16 rows, 66 MB, 13.1 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "decode_paged.cuh"

namespace moda {
namespace {

constexpr int kThreads = 128;
constexpr int kWarpsPerCta = kThreads / 32;
// CTAs of an SM, at least. Both kernels take 56 registers; the 4-bit one, held to
// them, spills 60 bytes, which costs less than a CTA fewer an SM (16384 tokens of 8 KV
// heads, at 8 CTAs, 9, 10: 42.5, 41.8, 43.2 us).
constexpr int kAppendCtasMx4 = 9;
constexpr int kAppendCtasBf16 = 8;

// -------------------------------------------------------------- page rows
// The row of (s, p) inside its page pool, for KV head 0: page * Hk * page_size
// + offset (below 2^31); -1 when there is none, which is latched unless s is
// padding.
__device__ __forceinline__ int page_row(const PagedKv& c, int s, int p, int pos_limit) {
  if (s == -1) return -1;
  if (s >= 0 && s < c.B && p >= 0 && p < pos_limit) {
    // page sizes are powers of two
    const int shift = 31 - __clz(c.page_size);
    const int page = c.table[(int64_t)s * c.max_pages + (p >> shift)];
    if (page >= 0 && page < c.num_pages)
      return ((page * c.Hk) << shift) + (p & (c.page_size - 1));
  }
  atomicCAS(c.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
  return -1;
}

// ------------------------------------------------------- microscaled 4 bits
// Scale byte of a block whose largest magnitude has the bits `amax`: the
// smallest power of two 2^E with amax <= 7 * 2^E, as E + 127. The mantissa of
// 7 = 1.75 * 2^2 is 0x600000: adding 0x1fffff carries into the exponent
// exactly when the mantissa is above it. 255 for infinities and NaN.
__device__ __forceinline__ int mx4_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255;
  const int e = (int)((amax + 0x1fffffu) >> 23) - 2;
  return min(max(e, 1), 252);
}

// 8 values times inv as e2m1 codes, value 0 in the low half of the low byte:
// round to nearest even, magnitudes over 6 to 6.
__device__ __forceinline__ uint32_t mx4_codes(const float* x, float inv) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(x[0] * inv), "f"(x[1] * inv), "f"(x[2] * inv), "f"(x[3] * inv), "f"(x[4] * inv),
        "f"(x[5] * inv), "f"(x[6] * inv), "f"(x[7] * inv));
  return w;
}

// The sum of x*c and y*s for one rounding later on: fp32 with the sticky bit
// of what lies below it ("round to odd"), so that a rounding to fewer bits
// comes out as from the exact value. x and y have 8 bits, c and s 24: both
// products are exact as head and tail, the heads' sum as well (two-sum).
__device__ __forceinline__ float turn_sticky(float x, float c, float y, float s) {
  const float t = x * c, te = fmaf(x, c, -t);
  const float p = y * s, pe = fmaf(y, s, -p);
  const float h = t + p, b = h - t;
  const float lo = ((t - (h - b)) + (p - b)) + (te + pe);
  const float hi = h + lo, rest = lo - (hi - h);
  uint32_t u = __float_as_uint(hi);
  if (rest != 0.f) {
    // toward zero where the rest points there, then the sticky bit
    if ((rest < 0.f) != (hi < 0.f)) u -= 1;
    u |= 1u;
  }
  return __uint_as_float(u);
}

// The largest magnitude's bits of a block, from each of its four lanes' own.
__device__ __forceinline__ uint32_t mx4_amax(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// 2^(127 - e) for scale byte e
__device__ __forceinline__ float mx4_inv(int e) {
  return __uint_as_float((uint32_t)(254 - min(e, 253)) << 23);
}

// A lane's 8 elements of one MX4 row as codes, and the scale byte of its block.
// All lanes of the warp call it.
__device__ __forceinline__ uint32_t mx4_row(const float* x, int& e) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, magnitude(x[i]));
  e = mx4_scale_byte(mx4_amax(m));
  return e == 255 ? 0u : mx4_codes(x, mx4_inv(e));  // a block of NaN has codes 0
}
// They go into the page (j: which eighth-of-row vector): codes by every lane,
// the block's scale by one lane of its four.
__device__ __forceinline__ void mx4_store(uint32_t w, int e, void* codes, void* scales, int64_t row, int j,
                                          int vpr) {
  reinterpret_cast<uint32_t*>(codes)[row * vpr + j] = w;
  if ((j & 3) == 0) reinterpret_cast<uint8_t*>(scales)[row * (vpr / 4) + (j >> 2)] = (uint8_t)e;
}

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ----------------------------------------------------------------- append
struct AppendGrid {
  int q_parts, parts;  // of a token: q's heads, then k's and v's
  uint32_t items;      // warps: no more than rows, which are below 2^31
  int kv_turns;        // 4-bit pages: heads of k and v that a lane takes, 1 or 2
};

__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}

// A lane's 8 cosines and 8 sines, and the turning of a and b, the halves of 8
// pairs (or 4 interleaved pairs each).
struct Turn {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* table, int rot) {
    load4(table, c);
    load4(table + 4, c + 4);
    load4(table + rot / 2, s);
    load4(table + rot / 2 + 4, s + 4);
  }
  __device__ __forceinline__ void apply(uint4& a, uint4& b, bool interleaved) const {
    float x[8], y[8];
    unpack8(a, x);
    unpack8(b, y);
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
        x[2 * i] = fmaf(x0, c[i], -(x1 * s[i]));
        x[2 * i + 1] = fmaf(x1, c[i], x0 * s[i]);
        y[2 * i] = fmaf(y0, c[i + 4], -(y1 * s[i + 4]));
        y[2 * i + 1] = fmaf(y1, c[i + 4], y0 * s[i + 4]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x0 = x[i], y0 = y[i];
        x[i] = fmaf(x0, c[i], -(y0 * s[i]));
        y[i] = fmaf(y0, c[i], x0 * s[i]);
      }
    }
    a = pack8(x);
    b = pack8(y);
  }
};

// One head of k and of v as 4-bit rows, and of k_out. The warp's rows are
// d/8 lanes each; `on`: the lane's head exists.
template <int D>
__device__ __forceinline__ void put_mx4(const KvAppendArgs& a, uint4 kr, const uint4& vr,
                                        const float* table, int64_t n, int64_t row, int h, bool on,
                                        int lane) {
  constexpr int VPR = D / 8;
  const int j = lane % VPR, half = a.rot / 16;
  const bool turned = j < 2 * half, low = j < half;
  // the pairs' other halves: the lane's own when they are interleaved
  uint4 other = kr;
  if (!a.interleaved) {
    const int partner = turned ? lane + (low ? half : -half) : lane;
    other.x = __shfl_sync(0xffffffffu, kr.x, partner);
    other.y = __shfl_sync(0xffffffffu, kr.y, partner);
    other.z = __shfl_sync(0xffffffffu, kr.z, partner);
    other.w = __shfl_sync(0xffffffffu, kr.w, partner);
  }
  float x[8], y[8], z[8], cs[8], sn[8];  // z = x cs + y sn
  auto inputs = [&] {
    unpack8(kr, x);
    unpack8(other, y);
    if (!turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f, y[i] = -0.f;  // z = x, its zero's sign too
    } else if (a.interleaved) {
      float c[4], s[4];
      load4(table + j * 4, c);
      load4(table + a.rot / 2 + j * 4, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = x[i ^ 1];
        cs[i] = c[i / 2];
        sn[i] = (i & 1) ? s[i / 2] : -s[i / 2];
      }
    } else {
      const float* t = table + (low ? j : j - half) * 8;
      load4(t, cs);
      load4(t + 4, cs + 4);
      load4(t + a.rot / 2, sn);
      load4(t + a.rot / 2 + 4, sn + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = low ? -sn[i] : sn[i];
    }
  };
  inputs();
  // z = x c + y s in fp32 is off by at most 2^-24 (|y s| + |z|). Codes and scale
  // are the exact value's wherever both ends of an interval of three times that
  // have the same; at a border, which one warp in hundreds meets, the rotation
  // is done again with a sticky bit. (16384 tokens of 8 KV heads, d = 128: always
  // with the sticky bit 51.6 us, so 46.0.)
  float off = 0.f;
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = y[i] * sn[i];
    z[i] = fmaf(x[i], cs[i], p);
    off = fmaxf(off, fabsf(p) + fabsf(z[i]));
    big = max(big, magnitude(z[i]));
  }
  if (a.k_out && on)
    *(reinterpret_cast<uint4*>(a.k_out) + (n * a.c.Hk + h) * VPR + j) = turned ? pack8(z) : kr;
  const float d = turned ? off * 0x1.8p-23f : 0.f;
  big = mx4_amax(__float_as_uint(__uint_as_float(big) + d));
  int e = mx4_scale_byte(big);
  uint32_t w = 0;
  if (e != 255) {
    float lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = z[i] - d;
    w = mx4_codes(lo, mx4_inv(e));
  }
  bool border = e == 255;
  if (!border) {
    float hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = z[i] + d;
    // the scale: the exact maximum is within 384 units in the last place below
    // `big`, as long as no element lost more than 6 bits to cancellation
    border = w != mx4_codes(hi, mx4_inv(e)) || !(off <= 64.f * __uint_as_float(big)) ||
             (big & 0x7fffffu) - 0x600001u < 512u;
  }
  if (__any_sync(0xffffffffu, turned && border)) {
    // (from what the registers still hold, and the table)
    asm volatile("" : "+r"(kr.x), "+r"(kr.y), "+r"(kr.z), "+r"(kr.w) : : "memory");
    asm volatile("" : "+r"(other.x), "+r"(other.y), "+r"(other.z), "+r"(other.w));
    inputs();
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i];
    if (turned)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = turn_sticky(x[i], cs[i], y[i], sn[i]);
    w = mx4_row(z, e);
  }
  if (on) mx4_store(w, e, a.c.k, a.c.k_scale, row, j, VPR);
  unpack8(vr, z);
  w = mx4_row(z, e);
  if (on) mx4_store(w, e, a.c.v, a.c.v_scale, row, j, VPR);
}

template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads, MX4 ? kAppendCtasMx4 : kAppendCtasBf16)
kv_append_kernel(const __grid_constant__ KvAppendArgs a, const __grid_constant__ AppendGrid g) {
  constexpr int VPR = D / 8;
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  paged::wait_for_stream();
  if (item >= g.items) return;
  const int64_t n = item / (uint32_t)g.parts;  // item = token * parts + part
  const int part = (int)(item - (uint32_t)n * g.parts);
  const int s = a.seq[n], p = a.pos[n];
  int limit = a.c.max_pages * a.c.page_size;
  if (a.rot > 0) limit = min(limit, a.rope_rows);

  if (MX4 && part >= g.q_parts) {
    // one head a lane, or two after one another with all four loads on the way first
    constexpr int HPI = 32 / VPR;
    int h = (part - g.q_parts) * (g.kv_turns * HPI) + lane / VPR;
    const uint16_t* ks = reinterpret_cast<const uint16_t*>(a.k) + n * a.k_stride + h * D + lane % VPR * 8;
    const uint16_t* vs = reinterpret_cast<const uint16_t*>(a.v) + n * a.v_stride + h * D + lane % VPR * 8;
    uint4 kr[2], vr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      kr[i] = vr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (i < g.kv_turns && h + i * HPI < a.c.Hk) {
        kr[i] = *reinterpret_cast<const uint4*>(ks + i * HPI * D);
        vr[i] = *reinterpret_cast<const uint4*>(vs + i * HPI * D);
      }
    }
    const int row = page_row(a.c, s, p, limit);
    if (row < 0) return;
#pragma unroll 1
    for (int i = 0; i < g.kv_turns; ++i) {
      put_mx4<D>(a, kr[0], vr[0], a.rope + (int64_t)p * a.rot, n, (int64_t)row + (int64_t)h * a.c.page_size, h,
                 h < a.c.Hk, lane);
      h += HPI;
      kr[0] = kr[1];
      vr[0] = vr[1];
    }
    return;
  }
  // this lane's two vectors of a head; of two heads of q, or of one of k and v
  constexpr int HPI = 64 / VPR;
  const int slot = lane % (VPR / 2), half = a.rot / 16;
  const bool turned = slot < half;
  const int v0 = turned && !a.interleaved ? slot : 2 * slot;
  const int v1 = turned && !a.interleaved ? slot + half : 2 * slot + 1;
  const bool is_q = part < g.q_parts;
  const int H = is_q ? a.Hq : a.c.Hk;
  const int h = (is_q ? part * (2 * HPI) : (part - g.q_parts) * HPI) + lane / (VPR / 2);
  const bool on = h < H, on2 = is_q ? h + HPI < H : on;
  uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x, x2 = x, y2 = x;
  {
    const uint16_t* src = is_q ? reinterpret_cast<const uint16_t*>(a.q) + n * a.q_stride
                               : reinterpret_cast<const uint16_t*>(a.k) + n * a.k_stride;
    const uint16_t* src2 = is_q ? src + HPI * D : reinterpret_cast<const uint16_t*>(a.v) + n * a.v_stride;
    const uint4* u = reinterpret_cast<const uint4*>(src + h * D);
    const uint4* u2 = reinterpret_cast<const uint4*>(src2 + h * D);
    if (on) {
      x = __ldcs(u + v0);
      y = __ldcs(u + v1);
    }
    if (on2) {
      x2 = __ldcs(u2 + v0);
      y2 = __ldcs(u2 + v1);
    }
  }
  const int row = page_row(a.c, s, p, limit);
  if (row < 0 || !on) return;
  if (turned) {
    Turn turn;
    turn.load(a.rope + (int64_t)p * a.rot + slot * 8, a.rot);
    turn.apply(x, y, a.interleaved);
    if (is_q) turn.apply(x2, y2, a.interleaved);
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(is_q ? a.q_out : a.k_out);
  if (out) {
    uint4* u = reinterpret_cast<uint4*>(out + (n * H + h) * D);
    __stcs(u + v0, x);
    __stcs(u + v1, y);
    if (is_q && on2) {
      __stcs(u + HPI * VPR + v0, x2);
      __stcs(u + HPI * VPR + v1, y2);
    }
  }
  if (!MX4 && !is_q) {
    const int64_t r = ((int64_t)row + (int64_t)h * a.c.page_size) * VPR;
    uint4* u = reinterpret_cast<uint4*>(a.c.k) + r;
    __stcs(u + v0, x);
    __stcs(u + v1, y);
    u = reinterpret_cast<uint4*>(a.c.v) + r;
    __stcs(u + v0, x2);
    __stcs(u + v1, y2);
  }
}

// ----------------------------------------------------------------- gather
// A warp: `tokens` tokens, all heads; a lane one 16-byte vector of the output.
template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads)
kv_gather_kernel(const __grid_constant__ PagedKv c, const int* seq, const int* pos, int N, int tokens,
                 uint4* k, uint4* v) {
  constexpr int VPR = D / 8;
  constexpr int HPI = 32 / VPR;  // heads at once
  const int lane = threadIdx.x & 31, j = lane % VPR, sub = lane / VPR;
  const int64_t n0 = ((int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5)) * tokens;
  paged::wait_for_stream();
  int my_row = -1;
  if (lane < tokens && n0 + lane < N)
    my_row = page_row(c, seq[n0 + lane], pos[n0 + lane], c.max_pages * c.page_size);
  // (token, heads) pairs in one line, U of them in flight
  constexpr int U = 4;
  const int per = (c.Hk + HPI - 1) / HPI;
  for (int i0 = 0; i0 < tokens * per; i0 += U) {
    uint4 x[U][2];
    float sc[U][2];
    int64_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = (i0 + u) / per, h = (i0 + u - t * per) * HPI + sub;
      const int row0 = __shfl_sync(0xffffffffu, my_row, t & 31);
      to[u] = -1;
      if (i0 + u < tokens * per && row0 >= 0 && h < c.Hk) {
        to[u] = ((n0 + t) * c.Hk + h) * VPR + j;
        const int64_t row = (int64_t)row0 + (int64_t)h * c.page_size;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const void* pages = e ? c.v : c.k;
          if constexpr (MX4) {
            x[u][e].x = reinterpret_cast<const uint32_t*>(pages)[row * VPR + j];
            const uint32_t b =
                reinterpret_cast<const uint8_t*>(e ? c.v_scale : c.k_scale)[row * (VPR / 4) + (j >> 2)];
            // 2^(b - 127); 255 is NaN, 0 is 2^-127
            sc[u][e] = __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
          } else {
            x[u][e] = reinterpret_cast<const uint4*>(pages)[row * VPR + j];
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (to[u] < 0) continue;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint4 out = x[u][e];
        if constexpr (MX4) {
          uint32_t f16[4];  // code pairs, exact
          asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
              " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
              " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
              : "=r"(f16[0]), "=r"(f16[1]), "=r"(f16[2]), "=r"(f16[3])
              : "r"(x[u][e].x));
          float f[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f16[q]));
            f[2 * q] = y.x * sc[u][e];
            f[2 * q + 1] = y.y * sc[u][e];
          }
          out = pack8(f);
        }
        (e ? v : k)[to[u]] = out;
      }
    }
  }
}

template <int D>
cudaError_t append_d(const KvAppendArgs& a, cudaStream_t stream) {
  const bool mx4 = a.c.format == MODA_KV_MX4;
  constexpr int VPR = D / 8;
  AppendGrid g;
  g.q_parts = (a.Hq + 128 / VPR - 1) / (128 / VPR);
  // 4-bit pages: two heads a lane where the warps would not be on the SMs at
  // once (16384 tokens of 8 KV heads: 46.0 us with one, 41.8), one where each
  // warp's own time counts (253 tokens: 2.4 us, with two 3.1)
  const int group = 32 / VPR, one = g.q_parts + (a.c.Hk + group - 1) / group;
  g.kv_turns = (int64_t)a.N * one <= (int64_t)a.num_sms * kAppendCtasMx4 * kWarpsPerCta ? 1 : 2;
  const int kv_heads = mx4 ? g.kv_turns * group : 64 / VPR;
  g.parts = g.q_parts + (a.c.Hk + kv_heads - 1) / kv_heads;
  g.items = (uint32_t)a.N * g.parts;
  const unsigned blocks = (g.items + kWarpsPerCta - 1) / kWarpsPerCta;
  return paged::launch_dependent(mx4 ? kv_append_kernel<D, true> : kv_append_kernel<D, false>,
                                 dim3(blocks), kThreads, 0, stream, a, g);
}

template <int D>
cudaError_t gather_d(const PagedKv& c, const int* seq, const int* pos, int N, void* k, void* v,
                     int num_sms, cudaStream_t stream) {
  // as many tokens a warp as make about one wave of warps: their look-ups are
  // made once and at once
  int tokens = 1;
  while (tokens < 32 && N > num_sms * 32 * (int64_t)tokens) tokens *= 2;
  const int64_t warps = ((int64_t)N + tokens - 1) / tokens;
  return paged::launch_dependent(
      c.format == MODA_KV_MX4 ? kv_gather_kernel<D, true> : kv_gather_kernel<D, false>,
      dim3((unsigned)((warps + kWarpsPerCta - 1) / kWarpsPerCta)), kThreads, 0, stream, c, seq, pos, N,
      tokens, (uint4*)k, (uint4*)v);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? append_d<128>(a, stream) : append_d<64>(a, stream);
}

cudaError_t launch_kv_gather(const PagedKv& c, const int* seq, const int* pos, int N, void* k,
                             void* v, int num_sms, cudaStream_t stream) {
  return c.d == 128 ? gather_d<128>(c, seq, pos, N, k, v, num_sms, stream)
                    : gather_d<64>(c, seq, pos, N, k, v, num_sms, stream);
}

}  // namespace moda
