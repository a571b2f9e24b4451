// Rows into and out of the paged KV cache (layouts in include/moda.h).
//
// append  q and k are turned in pairs, (a, b) -> (a c - b s, b c + a s), with
//         the cosines and sines of the token's position; k and v go into the
//         page row of (sequence, position), as bf16 or as microscaled 4-bit.
// gather  the rows back as dense bf16.
//
// Both are HBM-bound. A lane owns 8 consecutive elements (16 bytes), d/8 lanes
// a row of one head, so a warp works on 2 (d = 128) or 4 (d = 64) tokens at a
// time, for one kind (q, k or v) and a chunk of its heads: a lane reads its
// cosines and sines once and turns every head of the chunk with them, and the
// pair's other half comes from a lane of the same row by shuffle.
#include <cuda_bf16.h>
#include <stdint.h>

#include "decode_paged.cuh"

namespace moda {
namespace {

constexpr int kThreads = 128;
constexpr int kInFlight = 4;  // rows a lane loads before it stores the first

// -------------------------------------------------------------- page rows
// The row of (s, p) inside its page pool, for KV head 0: page * Hk * page_size
// + offset; -1 when there is none, which is latched unless s is padding.
__device__ __forceinline__ int64_t page_row(const PagedKv& c, int s, int p, int pos_limit) {
  if (s == -1) return -1;
  int page = -1;
  if (s >= 0 && s < c.B && p >= 0 && p < pos_limit) {
    page = *(c.table + (int64_t)s * c.max_pages + p / c.page_size);
    if (page >= 0 && page < c.num_pages)
      return (int64_t)page * c.Hk * c.page_size + p % c.page_size;
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

// A lane's 8 elements of one MX4 row (j: which eighth-of-row vector) into the
// page: codes by every lane, the block's scale by one lane of its four. All
// lanes of the warp call it; `on` says whose row exists.
__device__ __forceinline__ void mx4_store(const float* x, uint8_t* codes, uint8_t* scales,
                                          int64_t row, int j, int vpr, bool on) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int e = mx4_scale_byte(m);
  // 2^(127 - e); a block of NaN has codes 0
  const float inv = __uint_as_float((uint32_t)(254 - min(e, 253)) << 23);
  const uint32_t w = e == 255 ? 0u : mx4_codes(x, inv);
  if (on) {
    reinterpret_cast<uint32_t*>(codes)[row * vpr + j] = w;
    if ((j & 3) == 0) scales[row * (vpr / 4) + (j >> 2)] = (uint8_t)e;
  }
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
  int chunk;                 // heads of one work item
  int q_chunks, kv_chunks;   // items of a token group: q_chunks, then k's and v's kv_chunks
  int64_t items;
};

template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(const KvAppendArgs a, const AppendGrid g) {
  constexpr int VPR = D / 8;      // lanes of a row
  constexpr int TPW = 32 / VPR;   // tokens of a warp
  const int lane = threadIdx.x & 31;
  const int j = lane % VPR, sub = lane / VPR;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  paged::wait_for_stream();
  if (item >= g.items) return;
  const int per_group = g.q_chunks + 2 * g.kv_chunks;
  const int64_t group = item / per_group;
  int c = (int)(item - group * per_group);
  // kind 0: q, 1: k, 2: v
  const int kind = c < g.q_chunks ? 0 : c < g.q_chunks + g.kv_chunks ? 1 : 2;
  c -= kind == 0 ? 0 : kind == 1 ? g.q_chunks : g.q_chunks + g.kv_chunks;
  const int H = kind == 0 ? a.Hq : a.c.Hk;
  const int h0 = c * g.chunk, h1 = min(H, h0 + g.chunk);

  const int64_t n = group * TPW + sub;
  const bool in = n < a.N;
  const int s = in ? a.seq[n] : -1, p = in ? a.pos[n] : 0;
  int limit = a.c.max_pages * a.c.page_size;
  if (a.rot > 0) limit = min(limit, a.rope_rows);
  const int64_t row0 = page_row(a.c, s, p, limit);
  const bool on = row0 >= 0;

  // this lane's cosines and signed sines, and the lane that holds its pairs'
  // other halves (itself when the pairs are interleaved)
  const int half = a.rot / 16;  // vectors of half the turned part
  const bool turned = kind != 2 && j < 2 * half;
  const bool inter = a.interleaved;
  float cs[8], sn[8];
  int partner = lane;
  if (turned && on) {
    const float* t = a.rope + (int64_t)p * a.rot;
    if (inter) {
      const float4 c0 = *(reinterpret_cast<const float4*>(t + j * 4));
      const float4 s0 = *(reinterpret_cast<const float4*>(t + a.rot / 2 + j * 4));
      const float cc[4] = {c0.x, c0.y, c0.z, c0.w}, ss[4] = {s0.x, s0.y, s0.z, s0.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = cc[i / 2];
        sn[i] = (i & 1) ? ss[i / 2] : -ss[i / 2];
      }
    } else {
      const bool low = j < half;
      const float* tc = t + (low ? j : j - half) * 8;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c0 = *(reinterpret_cast<const float4*>(tc) + i);
        const float4 s0 = *(reinterpret_cast<const float4*>(tc + a.rot / 2) + i);
        cs[4 * i] = c0.x; cs[4 * i + 1] = c0.y; cs[4 * i + 2] = c0.z; cs[4 * i + 3] = c0.w;
        sn[4 * i] = low ? -s0.x : s0.x; sn[4 * i + 1] = low ? -s0.y : s0.y;
        sn[4 * i + 2] = low ? -s0.z : s0.z; sn[4 * i + 3] = low ? -s0.w : s0.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
  }
  if (turned && !inter) partner = lane + (j < half ? half : -half);

  const uint16_t* src = reinterpret_cast<const uint16_t*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                        (in ? n : 0) * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
  const uint4* src4 = reinterpret_cast<const uint4*>(src) + j;
  uint4* dense = reinterpret_cast<uint4*>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : nullptr);
  if (dense) dense += n * H * VPR + j;
  void* pages = kind == 1 ? a.c.k : a.c.v;
  void* scales = kind == 1 ? a.c.k_scale : a.c.v_scale;

  for (int h = h0; h < h1; h += kInFlight) {
    uint4 raw[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      raw[u] = make_uint4(0u, 0u, 0u, 0u);
      if (on && h + u < h1) raw[u] = *(src4 + (int64_t)(h + u) * VPR);
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      if (h + u >= h1) break;  // the same for the whole warp
      uint4 out = raw[u];
      float x[8], y[8], z[8];
      if (kind != 2) {
        unpack8(raw[u], x);
        if (inter) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
        } else {
          uint4 o;
          o.x = __shfl_sync(0xffffffffu, raw[u].x, partner);
          o.y = __shfl_sync(0xffffffffu, raw[u].y, partner);
          o.z = __shfl_sync(0xffffffffu, raw[u].z, partner);
          o.w = __shfl_sync(0xffffffffu, raw[u].w, partner);
          unpack8(o, y);
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = fmaf(x[i], cs[i], y[i] * sn[i]);
          out = pack8(z);
        }
        if (dense && on) dense[(int64_t)(h + u) * VPR] = out;
        if (kind == 0) continue;
      }
      const int64_t row = row0 + (int64_t)(h + u) * a.c.page_size;
      if constexpr (MX4) {
        if (kind == 2) {
          unpack8(raw[u], z);
        } else if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = turn_sticky(x[i], cs[i], y[i], sn[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = x[i];
        }
        mx4_store(z, reinterpret_cast<uint8_t*>(pages), reinterpret_cast<uint8_t*>(scales), row, j,
                  VPR, on);
      } else {
        if (on) reinterpret_cast<uint4*>(pages)[row * VPR + j] = out;
      }
    }
  }
}

// ----------------------------------------------------------------- gather
// One lane: 8 elements of one row of one head, of k and of v.
template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads)
kv_gather_kernel(const PagedKv c, const int* seq, const int* pos,
                 int64_t vecs, uint4* k, uint4* v) {
  constexpr int VPR = D / 8;
  const int limit = c.max_pages * c.page_size;
  paged::wait_for_stream();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < vecs;
       i += (int64_t)gridDim.x * kThreads) {
    const int j = (int)(i % VPR);
    const int64_t nh = i / VPR;
    const int64_t n = nh / c.Hk;
    const int h = (int)(nh - n * c.Hk);
    const int64_t row0 = page_row(c, seq[n], pos[n], limit);
    if (row0 < 0) continue;
    const int64_t row = row0 + (int64_t)h * c.page_size;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const void* pages = kv ? c.v : c.k;
      uint4 out;
      if constexpr (MX4) {
        const uint32_t w = *(reinterpret_cast<const uint32_t*>(pages) + row * VPR + j);
        const uint32_t b = *(reinterpret_cast<const uint8_t*>(kv ? c.v_scale : c.k_scale) +
                                 row * (VPR / 4) + (j >> 2));
        // 2^(b - 127); 255 is NaN, 0 is 2^-127
        const float sc = __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t q = w >> (4 * e);
          // e2m1 as the top of an fp32 pattern: 2^-126 times too small, exactly
          // (codes 0 and 0.5 are zero and a subnormal there)
          const float m = __uint_as_float((q & 7u) << 22) * __uint_as_float(253u << 23);
          x[e] = ((q & 8u) ? -m : m) * sc;
        }
        out = pack8(x);
      } else {
        out = *(reinterpret_cast<const uint4*>(pages) + row * VPR + j);
      }
      (kv ? v : k)[i] = out;
    }
  }
}

template <int D>
cudaError_t append_d(const KvAppendArgs& a, cudaStream_t stream) {
  constexpr int TPW = 32 / (D / 8);
  const int64_t groups = ((int64_t)a.N + TPW - 1) / TPW;
  // heads per item: up to 8, so that a lane's cosines and sines serve 8 heads,
  // fewer while that leaves SMs without two warps each
  AppendGrid g;
  g.chunk = 8;
  while (g.chunk > 1 &&
         groups * ((a.Hq + 2 * a.c.Hk + g.chunk - 1) / g.chunk) < (int64_t)a.num_sms * 8)
    g.chunk >>= 1;
  g.q_chunks = (a.Hq + g.chunk - 1) / g.chunk;
  g.kv_chunks = (a.c.Hk + g.chunk - 1) / g.chunk;
  g.items = groups * (g.q_chunks + 2 * g.kv_chunks);
  const int64_t blocks = (g.items + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return paged::launch_dependent(
      a.c.format == MODA_KV_MX4 ? kv_append_kernel<D, true> : kv_append_kernel<D, false>,
      dim3((unsigned)blocks), kThreads, 0, stream, a, g);
}

template <int D>
cudaError_t gather_d(const PagedKv& c, const int* seq, const int* pos, int N, void* k, void* v,
                     int num_sms, cudaStream_t stream) {
  const int64_t vecs = (int64_t)N * c.Hk * (D / 8);
  int64_t blocks = (vecs + kThreads - 1) / kThreads;
  const int64_t cap = (int64_t)num_sms * 16;
  if (blocks > cap) blocks = cap;
  return paged::launch_dependent(
      c.format == MODA_KV_MX4 ? kv_gather_kernel<D, true> : kv_gather_kernel<D, false>,
      dim3((unsigned)blocks), kThreads, 0, stream, c, seq, pos, vecs, (uint4*)k, (uint4*)v);
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
