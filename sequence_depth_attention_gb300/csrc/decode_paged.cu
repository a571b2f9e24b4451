// MoDA decode for a batch over the paged KV cache: the new token of every
// sequence attends, under one softmax, to the rows of its pages and to its L
// depth slots.
//
// One CTA per (sequence, query head), one key per warp at a time, online
// softmax per warp, the warps' states merged through shared memory.
#include <cuda_bf16.h>

#include "moda_internal.h"

namespace moda {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// E elements of a row, from element e0
template <int E>
__device__ __forceinline__ void load_bf16(const void* base, int64_t off, int e0, float* x) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + off + e0;
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = bf(p[i]);
}
template <int E>
__device__ __forceinline__ void load_mx4(const void* codes, const void* scales, int64_t row, int D,
                                         int e0, float* x) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(codes) + row * (D / 2) + e0 / 2;
  const uint32_t b = reinterpret_cast<const uint8_t*>(scales)[row * (D / 32) + e0 / 32];
  const float sc = __uint_as_float(b == 255 ? 0x7fc00000u : b << 23);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const uint32_t q = p[i / 2] >> (4 * (i & 1));
    const float m = __uint_as_float((q & 7u) << 22) * __uint_as_float(253u << 23);
    x[i] = ((q & 8u) ? -m : m) * sc;
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_paged_kernel(const DecodePagedArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm_o[kWarps][D];
  __shared__ float sm_ml[kWarps][2];
  const int h = blockIdx.x % a.Hq, b = blockIdx.x / a.Hq;
  const int hk = h / a.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedKv& c = a.c;
  int n = a.seq_lens[b];
  const int most = c.max_pages * c.page_size;
  if (n < 0 || n > most) {
    if (threadIdx.x == 0) atomicCAS(c.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
    n = n < 0 ? 0 : most;
  }
  float q[E], o[E];
  load_bf16<E>(a.q, ((int64_t)b * a.Hq + h) * D, lane * E, q);
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float sl = a.scale * kLog2e;
  for (int key = warp; key < n + a.L; key += kWarps) {
    float k[E], v[E];
    if (key < n) {
      const int page = c.table[(int64_t)b * c.max_pages + key / c.page_size];
      if (page < 0 || page >= c.num_pages) {
        if (lane == 0) atomicCAS(c.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
        continue;
      }
      const int64_t row = ((int64_t)page * c.Hk + hk) * c.page_size + key % c.page_size;
      if (c.format == MODA_KV_MX4) {
        load_mx4<E>(c.k, c.k_scale, row, D, lane * E, k);
        load_mx4<E>(c.v, c.v_scale, row, D, lane * E, v);
      } else {
        load_bf16<E>(c.k, row * D, lane * E, k);
        load_bf16<E>(c.v, row * D, lane * E, v);
      }
    } else {
      const int64_t off = (int64_t)b * a.depth_b_stride + (int64_t)hk * a.depth_hk_stride +
                          (int64_t)(key - n) * a.depth_slot_stride;
      load_bf16<E>(a.kd, off, lane * E, k);
      load_bf16<E>(a.vd, off, lane * E, v);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= sl;
    const float nm = fmaxf(m, s), ref = nm == -INFINITY ? 0.f : nm;
    const float al = exp2f(m - ref), p = exp2f(s - ref);
    m = nm;
    l = fmaf(l, al, p);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(p, v[i], o[i] * al);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) sm_o[warp][lane * E + i] = o[i];
  if (lane == 0) {
    sm_ml[warp][0] = m;
    sm_ml[warp][1] = l;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float M = -INFINITY, L = 0.f, oo = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_ml[w][0]);
    for (int w = 0; w < kWarps; ++w) {
      const float al = sm_ml[w][0] == -INFINITY ? 0.f : exp2f(sm_ml[w][0] - M);
      L = fmaf(sm_ml[w][1], al, L);
      oo = fmaf(sm_o[w][threadIdx.x], al, oo);
    }
    const bool none = n == 0 && a.L == 0;
    const int64_t r = (int64_t)b * a.Hq + h;
    reinterpret_cast<__nv_bfloat16*>(a.o)[r * D + threadIdx.x] =
        __float2bfloat16_rn(none ? 0.f : oo / L);
    if (threadIdx.x == 0 && a.lse) a.lse[r] = none ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

}  // namespace

size_t decode_paged_workspace_bytes(int Hq, int Hk, int d) { return 16; }

cudaError_t launch_decode_paged(const DecodePagedArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)(a.c.B * a.Hq);
  if (a.c.d == 128)
    decode_paged_kernel<128><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    decode_paged_kernel<64><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace moda
