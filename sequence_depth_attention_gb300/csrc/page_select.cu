// Which pages of the paged KV cache a token attends to, where it does not attend to
// all: the summaries of the pages, and the choice by them.
//
// page_means  the mean key of every page that a step has filled. A warp takes one (page,
//             KV head), the page's rows go by in 16-byte loads, sums in fp32 of values
//             times 1 / page_size (a power of two). A prompt of 16384 rows, 4 KV heads, d =
//             128: 4.4 us, where reading them takes 2.6; a decode step's 253 tokens 3.8:
//             the launch and two dependent look-ups.
// select      for each token and KV head the pages with the highest scores
//             max_g q_g . mean. A cluster of CTAs scores a (token, KV head)'s pages, 16
//             to a warp MMA with the G queries in its 8 columns, into the shared memory
//             of its first CTA, which chooses. 64 contexts of up to 32768 rows (pages of
//             16, 4 KV heads, G = 8, d = 128): 34 us, where reading the means takes 10.3.
//             What bounds it is the choice: its steps wait for one another (a histogram,
//             its sum, the next), beside which other items' scores run.
//
// The choice is that of the exact scores, so that it depends on no order of sums. A
// score s in fp32 is at most eps = 2^-14 sum_i |q_i| |mean_i| from the exact one: the
// d products are exact in fp32, and a chain of d/16 MMAs of 16 terms each, even were
// every term and every partial sum cut to 23 bits, loses less than 2^-17 of the sum of
// magnitudes. With tau the k-th largest s, a page above tau + 2 eps is among the k
// best, one below tau - 2 eps is not, and what lies between (a page or two, mostly
// the k-th alone) is scored again in fp64 where it decides.
#include <float.h>

#include "decode_paged.cuh"
#include "mx4.cuh"

namespace moda {
namespace {

using paged::wait_for_stream;

// The page of token n's row and its place in the batch; -1: none. Latches what is out
// of range.
__device__ __forceinline__ bool token_of(const PagedKv& c, int s, int p) {
  if (s == -1) return false;
  if (s >= 0 && s < c.B && p >= 0 && p < c.max_pages * c.page_size) return true;
  atomicCAS(c.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
  return false;
}

// ------------------------------------------------------------------ summaries
constexpr int kMeanWarps = 8, kMeanTokens = 32;

template <int D, bool MX4>
__global__ void __launch_bounds__(kMeanWarps * 32)
page_means_kernel(const __grid_constant__ PagedKv c, const int* seq, const int* pos, int N,
                  __nv_bfloat16* means) {
  // a lane's 16 bytes of a row: E elements, LPR lanes a row, RPL rows a load of the warp
  constexpr int E = MX4 ? 32 : 8, LPR = D / E, RPL = 32 / LPR;
  constexpr int U = 16 / RPL > 8 ? 8 : 16 / RPL > 0 ? 16 / RPL : 1;  // loads on the way: no page has fewer than 16 rows
  __shared__ int sm_page[kMeanTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_stream();
  if (warp == 0) {
    const int n = blockIdx.x * kMeanTokens + lane;
    int page = -1;
    if (n < N) {
      const int p = pos[n], s = seq[n];
      // (page sizes are powers of two)
      if (token_of(c, s, p) && (p & (c.page_size - 1)) == c.page_size - 1) {
        page = c.table[(int64_t)s * c.max_pages + (p >> (31 - __clz(c.page_size)))];
        if (page < 0 || page >= c.num_pages) {
          atomicCAS(c.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
          page = -1;
        }
      }
    }
    // filled pages first
    const uint32_t full = __ballot_sync(0xffffffffu, page >= 0);
    sm_page[lane] = -1;
    __syncwarp();
    if (page >= 0) sm_page[__popc(full & ((1u << lane) - 1u))] = page;
  }
  __syncthreads();
  const float inv = 1.f / (float)c.page_size;
  const int j = lane % LPR, r0 = lane / LPR;
  for (int item = warp;; item += kMeanWarps) {
    const int f = item / c.Hk, hk = item - f * c.Hk;
    if (f >= kMeanTokens || sm_page[f] < 0) break;
    const int64_t head = (int64_t)sm_page[f] * c.Hk + hk;
    const int64_t row0 = head * c.page_size + r0;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int r = 0; r < c.page_size; r += RPL * U) {
      uint4 x[U];
      uint32_t b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + r + u * RPL;
        x[u] = reinterpret_cast<const uint4*>(c.k)[row * LPR + j];
        if (MX4) b[u] = reinterpret_cast<const uint8_t*>(c.k_scale)[row * LPR + j];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        auto add = [&](int at, uint32_t pair) {
          acc[at] = fmaf(__uint_as_float(pair << 16), inv, acc[at]);
          acc[at + 1] = fmaf(__uint_as_float(pair & 0xffff0000u), inv, acc[at + 1]);
        };
        if constexpr (MX4) {
          uint32_t y[4];
          const uint32_t scale = mx4::scale_of(b[u]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mx4::unpack8(w[q], scale, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) add(q * 8 + 2 * i, y[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) add(2 * i, w[i]);
        }
      }
    }
#pragma unroll
    for (int sh = LPR; sh < 32; sh <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], sh);
    if (r0 == 0) {
      uint4* to = reinterpret_cast<uint4*>(means + head * D + j * E);
#pragma unroll
      for (int i = 0; i < E / 8; ++i)
        to[i] = make_uint4(sm103::pack_bf16x2(acc[8 * i], acc[8 * i + 1]),
                           sm103::pack_bf16x2(acc[8 * i + 2], acc[8 * i + 3]),
                           sm103::pack_bf16x2(acc[8 * i + 4], acc[8 * i + 5]),
                           sm103::pack_bf16x2(acc[8 * i + 6], acc[8 * i + 7]));
    }
  }
}

// --------------------------------------------------------------------- choice
constexpr int kSelWarps = 8, kSelThreads = kSelWarps * 32;
constexpr int kMaxCluster = 8;
constexpr float kEps = 0x1p-14f;
constexpr int kFew = 32;  // undecided pages that are ranked at once

struct SelectParams {
  PagedKv c;
  const __nv_bfloat16 *q, *means;
  const int *seq, *pos;
  int G, S, sink, recent, group;  // group: CTAs of a (token, KV head)
  int *pages, *rows;
};

struct SelectSmem {
  uint32_t hist[256];
  // of each warp of the group: the largest sum of magnitudes, as bits, and the largest and
  // the smallest key
  uint32_t reach[kMaxCluster][kSelWarps], top[kMaxCluster][kSelWarps], bottom[kMaxCluster][kSelWarps];
  double key[kFew];
  int index[kFew];
  int count[kSelWarps][2];
  uint32_t prefix32;
  unsigned long long prefix;
  int want, listed;
};

// Unsigned keys in the order of the floats; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double x) {
  const long long b = __double_as_longlong(x + 0.0);
  return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float((int)key < 0 ? key & 0x7fffffffu : ~key);
}

// One step of a radix choice, by warp 0: the bin in which the want-th largest lies
// (hist counts keys by the byte in question) and its place among that bin's.
__device__ __forceinline__ void choose_bin(SelectSmem& sm, int lane, uint32_t* bin) {
  // lane l: bins 255 - 8 l down to 248 - 8 l
  int mine = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) mine += sm.hist[255 - 8 * lane - i];
  int upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += x;
  }
  const int want = sm.want;
  __syncwarp();
  if (upto >= want && upto - mine < want) {
    int at = upto - mine, b = 255 - 8 * lane;
    while (at + (int)sm.hist[b] < want) at += sm.hist[b--];
    *bin = b;
    sm.want = want - at;
  }
  __syncwarp();
}

// a + b and what its rounding leaves, exactly (Knuth).
__device__ __forceinline__ float two_sum(float a, float b, float& rest) {
  const float s = __fadd_rn(a, b), x = __fsub_rn(s, a);
  rest = __fadd_rn(__fsub_rn(a, __fsub_rn(s, x)), __fsub_rn(b, x));
  return s;
}

// The exact score of a page: max over the group's queries of q . mean, to fp64's precision.
// All lanes have a head (the lanes of a head a part of it); all call it and get it. NaN
// counts as -infinity. SINGLE: products are exact in fp32 (none overflows, and those that
// underflow do not count) and are summed there in three parts, which fp64 adds up: of fp64
// operations an SM does two a cycle, conversions among them (a page took 6000 cycles).
template <int D, bool SINGLE>
__device__ __forceinline__ double exact_score(const __nv_bfloat16* q, const __nv_bfloat16* mean, int G, int lane) {
  int lgL = D == 128 ? 5 : 4;  // log2 of the lanes of a head, each two pairs of elements at least
  while (32 >> lgL < G) --lgL;
  const int head = lane >> lgL, part = lane & ((1 << lgL) - 1);
  // pairs of elements, those of a head's lanes side by side
  const uint32_t* qr = reinterpret_cast<const uint32_t*>(q + min(head, G - 1) * D) + part;
  const uint32_t* mr = reinterpret_cast<const uint32_t*>(mean) + part;
  const int steps = D / 2 >> lgL;  // 2 to D / 4
  double x = 0.0;
  float s[2] = {0.f, 0.f}, r[2] = {0.f, 0.f}, rr[2] = {0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < steps; ++i) {
    const uint32_t a = qr[i << lgL], b = mr[i << lgL];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float u = __uint_as_float(e ? a & 0xffff0000u : a << 16), v = __uint_as_float(e ? b & 0xffff0000u : b << 16);
      if constexpr (SINGLE) {
        float t, t2;
        s[e] = two_sum(s[e], __fmul_rn(u, v), t);
        r[e] = two_sum(r[e], t, t2);
        rr[e] = __fadd_rn(rr[e], t2);
      } else {
        x = fma((double)u, (double)v, x);
      }
    }
  }
  if constexpr (SINGLE) {
    float t, t2, t3;
    const float s0 = two_sum(s[0], s[1], t), r0 = two_sum(r[0], r[1], t2), r1 = two_sum(r0, t, t3);
    x = (double)s0 + ((double)r1 + (double)(t2 + t3 + rr[0] + rr[1]));
  }
  for (int sh = 1; sh < 1 << lgL; sh <<= 1) x += __shfl_xor_sync(0xffffffffu, x, sh);
  if (!(x == x)) x = -INFINITY;
  for (int sh = 1 << lgL; sh < 32; sh <<= 1) {
    const double y = __shfl_xor_sync(0xffffffffu, x, sh);
    if (y > x) x = y;
  }
  return x;
}

template <int D, int NT>
__global__ void __launch_bounds__(kSelThreads, NT == 1 ? 3 : 2)
select_pages_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ float scores[];  // of the first CTA of a group: of all candidates, as keys
  __shared__ SelectSmem sm;
  const PagedKv& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % p.group;
  const int item = blockIdx.x / p.group;
  const int n = item / c.Hk, hk = item - n * c.Hk;
  const bool clustered = p.group > 1;
  if (clustered) {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA runs
  }
  wait_for_stream();
  const int s = p.seq[n], pos = p.pos[n];
  const bool real = token_of(c, s, pos);
  const int shift = 31 - __clz(c.page_size);
  const int held = real ? (pos >> shift) + 1 : 0;
  const int* table = c.table + (int64_t)(real ? s : 0) * c.max_pages;
  int* out = p.pages + (int64_t)item * p.S;
  // Row block of page i of the sequence, -1 for one that is not in the pool (latched).
  auto block_of = [&](int i) -> int {
    const int page = table[i];
    if (page < 0 || page >= c.num_pages) {
      atomicCAS(c.err, 0u, (unsigned int)MODA_ERR_INVALID_ARG);
      return -1;
    }
    return page * c.Hk + hk;
  };
  const int kept = min(held, p.S);
  const int want = p.S - p.sink - p.recent, nc = held - p.sink - p.recent;  // of nc candidates
  if (held <= p.S || want == 0) {
    if (rank == 0) {
      for (int i = tid; i < p.S; i += kSelThreads)
        out[i] = i >= kept ? -1 : block_of(held <= p.S || i < p.sink ? i : held - p.S + i);
      if (tid == 0) p.rows[item] = kept > 0 ? ((kept - 1) << shift) + (pos & (c.page_size - 1)) + 1 : 0;
    }
    if (clustered) {
      __syncwarp();
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    return;
  }

  // ------------------------------------------------------------------- scores
  const __nv_bfloat16* q = p.q + (int64_t)item * p.G * D;
  {
    // The order of the head dimension is free: chunk i of a lane is 16 bytes, those of
    // a quad 64 that lie together; its four pairs are k = 2c, 2c + 1, 2c + 8, 2c + 9 of
    // two MMAs.
    constexpr int CH = D / 32;
    const int r0 = lane >> 2, cl = lane & 3;
    uint32_t qb[NT][CH][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (t * 8 + r0 < p.G) x = *reinterpret_cast<const uint4*>(q + (t * 8 + r0) * D + (i * 4 + cl) * 8);
        qb[t][i][0] = x.x; qb[t][i][1] = x.y; qb[t][i][2] = x.z; qb[t][i][3] = x.w;
      }
    // this CTA's candidates
    const int per = ((nc + p.group - 1) / p.group + 15) / 16 * 16;
    const int i0 = min(nc, rank * per), i1 = min(nc, i0 + per);
    if (clustered) {
      __syncwarp();
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all of the group run
    }
    uint32_t to = sm103::smem_u32(scores);
    if (clustered) to = paged::cluster_addr(to, 0);
    uint32_t reach = 0;  // bits of the largest sum of magnitudes, NaN above all
    uint32_t some_q = 0, some_mean = 0;  // is there anything but zeros?
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) some_q |= qb[t][i][e];
    auto id_of = [&](int i) -> int { return i < i1 ? block_of(p.sink + i) : -1; };
    uint32_t top = 0, bottom = 0xffffffffu;
    int a_next = id_of(i0 + warp * 16 + r0), b_next = id_of(i0 + warp * 16 + r0 + 8);
    for (int i = i0 + warp * 16; i < i1; i += kSelWarps * 16) {
      const int ia = a_next, ib = b_next;
      uint4 xa[CH], xb[CH];
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
        if (ia >= 0) xa[u] = reinterpret_cast<const uint4*>(p.means)[(int64_t)ia * (D / 8) + u * 4 + cl];
        if (ib >= 0) xb[u] = reinterpret_cast<const uint4*>(p.means)[(int64_t)ib * (D / 8) + u * 4 + cl];
      }
#pragma unroll
      for (int u = 0; u < CH; ++u)
        some_mean |= xa[u].x | xa[u].y | xa[u].z | xa[u].w | xb[u].x | xb[u].y | xb[u].z | xb[u].w;
      a_next = id_of(i + kSelWarps * 16 + r0);
      b_next = id_of(i + kSelWarps * 16 + r0 + 8);
      float z[NT][4], m[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = m[t][e] = 0.f;
#pragma unroll
        for (int u = 0; u < CH; ++u) {
          constexpr uint32_t kMag = 0x7fff7fffu;
          const uint32_t a0[4] = {xa[u].x, xb[u].x, xa[u].y, xb[u].y};
          const uint32_t a1[4] = {xa[u].z, xb[u].z, xa[u].w, xb[u].w};
          const uint32_t b0[4] = {xa[u].x & kMag, xb[u].x & kMag, xa[u].y & kMag, xb[u].y & kMag};
          const uint32_t b1[4] = {xa[u].z & kMag, xb[u].z & kMag, xa[u].w & kMag, xb[u].w & kMag};
          wmma16::mma_bf16(z[t], a0, qb[t][u][0], qb[t][u][1]);
          wmma16::mma_bf16(z[t], a1, qb[t][u][2], qb[t][u][3]);
          wmma16::mma_bf16(m[t], b0, qb[t][u][0] & kMag, qb[t][u][1] & kMag);
          wmma16::mma_bf16(m[t], b1, qb[t][u][2] & kMag, qb[t][u][3] & kMag);
        }
      }
      float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          reach = max(reach, __float_as_uint(m[t][e]) & 0x7fffffffu);
          if (t * 8 + 2 * cl + (e & 1) < p.G) best[e >> 1] = fmaxf(best[e >> 1], z[t][e]);  // drops NaN
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], 1));
        best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], 2));
      }
      // (a page that is not in the pool is never chosen before one that is)
      if (cl < 2) {
        const int at = i + r0 + 8 * cl;
        if (at < i1) {
          const uint32_t key = key_of((cl ? ib : ia) < 0 ? -INFINITY : best[cl]);
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + at * 4), "r"(key) : "memory");
          top = max(top, key);
          bottom = min(bottom, key);
        }
      }
    }
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      reach = max(reach, __shfl_xor_sync(0xffffffffu, reach, sh));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, sh));
      bottom = min(bottom, __shfl_xor_sync(0xffffffffu, bottom, sh));
    }
    // products next to or below the smallest floats: fp32 decides nothing
    const bool any_q = __any_sync(0xffffffffu, (some_q & 0x7fff7fffu) != 0);
    const bool any_mean = __any_sync(0xffffffffu, (some_mean & 0x7fff7fffu) != 0);
    if (any_q && any_mean && reach < __float_as_uint(0x1p-100f)) reach = 0x7f800000u;
    if (lane == 0) {
      uint32_t at[3] = {sm103::smem_u32(&sm.reach[rank][warp]), sm103::smem_u32(&sm.top[rank][warp]),
                        sm103::smem_u32(&sm.bottom[rank][warp])};
      const uint32_t x[3] = {reach, top, bottom};
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (clustered) at[i] = paged::cluster_addr(at[i], 0);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at[i]), "r"(x[i]) : "memory");
      }
    }
  }
  if (clustered) {
    paged::cluster_meet();
    if (rank > 0) return;
  } else {
    __syncthreads();
  }

  // ------------------------------------------------------------------- choice
  uint32_t* keys = reinterpret_cast<uint32_t*>(scores);
  uint32_t reach = 0, top = 0, bottom = 0xffffffffu;
  for (int i = lane; i < p.group * kSelWarps; i += 32) {
    reach = max(reach, (&sm.reach[0][0])[i]);
    top = max(top, (&sm.top[0][0])[i]);
    bottom = min(bottom, (&sm.bottom[0][0])[i]);
  }
  reach = __reduce_max_sync(0xffffffffu, reach);
  top = __reduce_max_sync(0xffffffffu, top);
  bottom = __reduce_min_sync(0xffffffffu, bottom);
  const float eps = __uint_as_float(reach) * kEps;  // infinite or NaN: nothing is decided by fp32
  // The want-th largest key is in [low, high]: a radix choice of 8 bits at a time from the
  // first that differs at all, until what is between them is no more than eps.
  if (tid == 0) {
    sm.want = want;
    sm.listed = 0;
  }
  int bits = 32 - __clz(top ^ bottom);  // of the keys that are not known yet
  uint32_t low = bits < 32 ? top >> bits << bits : 0u, high = low | (bits < 32 ? (1u << bits) - 1u : 0xffffffffu);
  while (bits > 0 && !(eps > FLT_MAX) && eps == eps && !(score_of(high) - score_of(low) <= eps)) {
    const int step = min(bits, 8);
    const uint32_t mask = bits < 32 ? 0xffffffffu << bits : 0u;
    bits -= step;
    sm.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < nc; i += kSelThreads)
      if ((keys[i] & mask) == low) atomicAdd(&sm.hist[keys[i] >> bits & ((1u << step) - 1u)], 1u);
    __syncthreads();
    if (warp == 0) {
      uint32_t bin = 256;
      choose_bin(sm, lane, &bin);
      if (bin < 256) sm.prefix32 = low | bin << bits;
    }
    __syncthreads();
    low = sm.prefix32;
    high = low | ((1u << bits) - 1u);
  }
  // The keys that are undecided: [least, most]; above, a page is chosen.
  uint32_t least = low, most = high;
  if (!(eps == 0.f) || bits > 0) {
    // (rounding outwards; an infinity stays alone)
    const bool any = eps <= FLT_MAX;
    least = any ? key_of(__fadd_rd(score_of(low), -2.f * eps)) : 0u;
    most = any ? key_of(__fadd_ru(score_of(high), 2.f * eps)) : 0xffffffffu;
  }
  __syncthreads();  // sm.listed is 0
  // a warp's part of the candidates, in order
  const int part = ((nc + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(nc, warp * part), w1 = min(nc, w0 + part);
  int above = 0, open = 0;
  for (int i = w0 + lane; i < w0 + part; i += 32) {
    const uint32_t k = i < w1 ? keys[i] : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i < w1 && k > most));
    open += __popc(__ballot_sync(0xffffffffu, i < w1 && k >= least && k <= most));
  }
  if (lane == 0) {
    sm.count[warp][0] = above;
    sm.count[warp][1] = open;
  }
  __syncthreads();
  int all_above = 0, all_open = 0;
  for (int w = 0; w < kSelWarps; ++w) {
    all_above += sm.count[w][0];
    all_open += sm.count[w][1];
  }
  const int need = want - all_above;  // of the open ones, 1 to all_open
  // Chosen are the keys of `from` and above, and of those that equal `tie` the first
  // `ties`.
  uint32_t from = least, tie = 0;
  int ties = 0;
  __syncthreads();  // sm.count is used again
  if (need < all_open && least == most) {  // equal scores, exact ones: by the page's number
    from = least + 1;
    tie = least;
    ties = need;
  } else if (need < all_open) {
    // Exact scores of the open ones; what is chosen gets the largest key, what is not
    // the least. (A key of 0 or of all ones would be a NaN's, which no score is.)
    from = 0xffffffffu;
    const float most_sum = __uint_as_float(reach);
    const bool single = most_sum >= 0x1p-60f && most_sum <= 0x1p120f;
    auto exact = [&](int at) -> double {  // of a candidate, by all lanes
      const int page = block_of(p.sink + at);
      const __nv_bfloat16* mean = p.means + (int64_t)max(page, 0) * D;
      const double x = single ? exact_score<D, true>(q, mean, p.G, lane) : exact_score<D, false>(q, mean, p.G, lane);
      return page < 0 ? (double)-INFINITY : x;
    };
    auto each_open = [&](auto&& f) {  // this warp's, one after another in order
      for (int i = w0; i < w1; i += 32) {
        const uint32_t k = i + lane < w1 ? keys[i + lane] : 0u;
        uint32_t set = __ballot_sync(0xffffffffu, i + lane < w1 && k >= least && k <= most);
        while (set) {
          f(i + __ffs(set) - 1);
          set &= set - 1;
        }
      }
    };
    if (all_open <= kFew) {
      each_open([&](int at) {
        if (lane == 0) sm.index[atomicAdd(&sm.listed, 1)] = at;
      });
      __syncthreads();
      for (int l = warp; l < all_open; l += kSelWarps) {
        const double x = exact(sm.index[l]);
        if (lane == 0) sm.key[l] = x + 0.0;
      }
      __syncthreads();
      if (warp == 0 && lane < all_open) {
        const double x = sm.key[lane];
        const int at = sm.index[lane];
        int before = 0;
        for (int l = 0; l < all_open; ++l)
          before += sm.key[l] > x || (sm.key[l] == x && sm.index[l] < at);
        keys[at] = before < need ? 0xffffffffu : 0u;
      }
      __syncthreads();
      // (those above `most` are chosen too)
      for (int i = tid; i < nc; i += kSelThreads)
        if (keys[i] > most && keys[i] != 0xffffffffu) keys[i] = 0xffffffffu;
    } else {
      // many that lie together: the same radix choice over 64 bits, the scores made
      // anew for each byte
      if (tid == 0) {
        sm.want = need;
        sm.prefix = 0;
      }
      for (int byte = 7; byte >= 0; --byte) {
        sm.hist[tid] = 0;
        __syncthreads();
        const unsigned long long prefix = sm.prefix;
        const unsigned long long mask = byte == 7 ? 0ull : ~0ull << (8 * byte + 8);
        each_open([&](int at) {
          const unsigned long long k = key_of(exact(at));
          if (lane == 0 && (k & mask) == prefix) atomicAdd(&sm.hist[k >> (8 * byte) & 255u], 1u);
        });
        __syncthreads();
        if (warp == 0) {
          uint32_t bin = 256;
          choose_bin(sm, lane, &bin);
          if (bin < 256) sm.prefix = prefix | (unsigned long long)bin << (8 * byte);
        }
        __syncthreads();
      }
      const unsigned long long t64 = sm.prefix;
      // sm.want of the pages that equal t64, the first ones: this warp's after the
      // earlier warps'
      int equal = 0;
      each_open([&](int at) { equal += key_of(exact(at)) == t64; });
      if (lane == 0) sm.count[warp][0] = equal;
      __syncthreads();
      int seen = 0;
      for (int w = 0; w < warp; ++w) seen += sm.count[w][0];
      const int first = sm.want;
      // (a warp changes keys of its own part alone, of one that it is past)
      each_open([&](int at) {
        const unsigned long long k = key_of(exact(at));
        const bool yes = k > t64 || (k == t64 && seen < first);
        seen += k == t64;
        __syncwarp();
        if (lane == 0) keys[at] = yes ? 0xffffffffu : 0u;
      });
      __syncthreads();
      for (int i = tid; i < nc; i += kSelThreads)
        if (keys[i] > most && keys[i] != 0xffffffffu) keys[i] = 0xffffffffu;
    }
    __syncthreads();
  }
  // In order of their numbers. (What is chosen without more ado has been counted above.)
  int mine = above + open, tied = 0;
  if (need < all_open) {
    mine = 0;
    for (int i = w0 + lane; i < w0 + part; i += 32) {
      const uint32_t k = i < w1 ? keys[i] : 0u;
      mine += __popc(__ballot_sync(0xffffffffu, i < w1 && k >= from));
      tied += __popc(__ballot_sync(0xffffffffu, i < w1 && ties > 0 && k == tie));
    }
    if (lane == 0) {
      sm.count[warp][0] = mine;
      sm.count[warp][1] = tied;
    }
    __syncthreads();
  }
  int at = 0, tied_before = 0;
  for (int w = 0; w < warp; ++w) {
    at += sm.count[w][0] + (need < all_open ? 0 : sm.count[w][1]);
    if (need < all_open) tied_before += sm.count[w][1];
  }
  at += min(tied_before, ties);
  for (int i = w0; i < w1; i += 32) {
    const uint32_t k = i + lane < w1 ? keys[i + lane] : 0u;
    const bool is_tie = i + lane < w1 && ties > 0 && k == tie;
    const uint32_t tie_set = __ballot_sync(0xffffffffu, is_tie);
    const uint32_t below = (1u << lane) - 1u;
    const bool yes = (i + lane < w1 && k >= from) || (is_tie && tied_before + __popc(tie_set & below) < ties);
    const uint32_t set = __ballot_sync(0xffffffffu, yes);
    if (yes) out[p.sink + at + __popc(set & below)] = i + lane;
    at += __popc(set);
    tied_before += __popc(tie_set);
  }
  __syncthreads();
  // their row blocks, looked up at once
  for (int i = tid; i < p.S; i += kSelThreads)
    out[i] = block_of(i < p.sink                 ? i
                      : i < p.S - p.recent ? p.sink + out[i]
                                           : held - p.S + i);
  if (tid == 0) p.rows[item] = ((p.S - 1) << shift) + (pos & (c.page_size - 1)) + 1;
}

template <int D>
cudaError_t select_d(const SelectPagesArgs& a, cudaStream_t stream) {
  const PagedKv& c = a.c;
  SelectParams p;
  p.c = c;
  p.q = (const __nv_bfloat16*)a.q;
  p.means = (const __nv_bfloat16*)a.means;
  p.seq = a.seq; p.pos = a.pos;
  p.G = a.G; p.S = a.S; p.sink = a.sink; p.recent = a.recent;
  p.pages = a.pages; p.rows = a.rows;
  // CTAs of a (token, KV head): a warp takes 16 pages at a time and waits for them, so a
  // CTA gets 256 pages of the longest context, as long as the CTAs are no more than four an
  // SM. Measured (us with nothing in L2, d = 128) against other limits:
  //   contexts x KV heads, rows    an SM:  1      2      4      8 CTAs
  //    8 x 4   32768 (page 16)           25.2   23.2   23.2   23.2
  //   16 x 8   to 32768 (16)             43.6   33.4   31.4   33.4
  //   32 x 4   to 65536 (32)             41.6   33.4   29.3   33.5
  //   64 x 4   to 32768 (16)             49.8   49.8   43.6   45.7
  //  256 x 2   to 16384 (16)             39.6   39.6   39.6   45.7
  // 128 pages a CTA, or 512: the same but for the third, 31.4 and 31.3.
  const int64_t items = (int64_t)a.N * c.Hk;
  int group = 1;
  while (group < kMaxCluster && items * group * 2 <= a.num_sms * 4 && c.max_pages >= 256 * group) group *= 2;
  p.group = group;
  const size_t smem = ((size_t)c.max_pages * 4 + 15) / 16 * 16;
  const auto kernel = a.G <= 8 ? select_pages_kernel<D, 1> : select_pages_kernel<D, 2>;
  if (smem > 32768) {
    // (the limit is the function's, not the call's: one value for all, so that calls from several
    // host threads do not lower it for each other)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxSelectPages * 4);
    if (e != cudaSuccess) return e;
  }
  return paged::launch_dependent_clusters(kernel, dim3((unsigned)(items * group)), group, kSelThreads, smem, stream, p);
}

}  // namespace

cudaError_t launch_page_means(const PagedKv& c, const int* seq, const int* pos, int N, void* means,
                              cudaStream_t stream) {
  const bool mx4 = c.format == MODA_KV_MX4;
  const auto kernel = c.d == 128 ? (mx4 ? page_means_kernel<128, true> : page_means_kernel<128, false>)
                                 : (mx4 ? page_means_kernel<64, true> : page_means_kernel<64, false>);
  return paged::launch_dependent(kernel, dim3((unsigned)((N + kMeanTokens - 1) / kMeanTokens)), kMeanWarps * 32, 0,
                                 stream, c, seq, pos, N, (__nv_bfloat16*)means);
}

cudaError_t launch_select_pages(const SelectPagesArgs& a, cudaStream_t stream) {
  return a.c.d == 128 ? select_d<128>(a, stream) : select_d<64>(a, stream);
}

}  // namespace moda
