// C-ABI entry points of the paged KV cache (declared in include/moda.h):
// argument validation and dispatch to kv_pages.cu and decode_paged.cu.
#include <stdint.h>

#include "moda.h"
#include "moda_internal.h"

namespace {

using moda::report;

moda_status ok() { return report(MODA_OK, "%s", ""); }

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

struct Range {
  const void* p;
  size_t n;
};

bool overlaps(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// The caches' byte ranges: pages of k and v, their scales.
struct CacheRanges {
  Range r[4];
};

moda_status check_cache(const moda_paged_kv* c, moda::PagedKv* out, CacheRanges* ranges) {
  if (!c) return report(MODA_ERR_INVALID_ARG, "NULL cache");
  if (c->format != MODA_KV_BF16 && c->format != MODA_KV_MX4)
    return report(MODA_ERR_INVALID_ARG, "format = %d", c->format);
  if (c->B < 0) return report(MODA_ERR_INVALID_ARG, "B = %d < 0", c->B);
  if (c->num_pages < 1 || c->max_pages < 1 || c->Hk < 1)
    return report(MODA_ERR_INVALID_ARG, "num_pages = %d, max_pages = %d, Hk = %d", c->num_pages,
                  c->max_pages, c->Hk);
  const int P = c->page_size;
  if (P != 16 && P != 32 && P != 64 && P != 128)
    return report(MODA_ERR_UNSUPPORTED, "page_size = %d (supported: 16, 32, 64, 128)", P);
  if (c->d != 64 && c->d != 128)
    return report(MODA_ERR_UNSUPPORTED, "d = %d (supported: 64, 128)", c->d);
  if (c->Hk > 4096) return report(MODA_ERR_UNSUPPORTED, "Hk = %d > 4096", c->Hk);
  if ((int64_t)c->num_pages * c->Hk > 0x7fffffffLL / P)
    return report(MODA_ERR_UNSUPPORTED, "num_pages * Hk * page_size exceeds 2^31 - 1 rows");
  if ((int64_t)c->max_pages * P > (1 << 30))
    return report(MODA_ERR_UNSUPPORTED, "max_pages * page_size = %lld > 2^30",
                  (long long)c->max_pages * P);
  // a CTA's share of a decode's units is counted in 32 bits
  if ((int64_t)c->max_pages * P > (1LL << 40) / c->Hk / (c->B > 0 ? c->B : 1))
    return report(MODA_ERR_UNSUPPORTED, "B * Hk * max_pages * page_size exceeds 2^40 rows");
  const bool mx4 = c->format == MODA_KV_MX4;
  if (!c->k || !c->v || (c->B > 0 && !c->block_table) || (mx4 && (!c->k_scale || !c->v_scale)))
    return report(MODA_ERR_INVALID_ARG, "NULL pages, scales or block table");
  if (!mx4 && (c->k_scale || c->v_scale))
    return report(MODA_ERR_INVALID_ARG, "bf16 pages have no scales");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16) || !aligned(c->block_table, 4))
    return report(MODA_ERR_MISALIGNED, "a cache pointer is not 16-byte (block_table: 4-byte) aligned");
  const size_t rows = (size_t)c->num_pages * c->Hk * P;
  const size_t pb = rows * (mx4 ? c->d / 2 : c->d * 2), sb = mx4 ? rows * (c->d / 32) : 0;
  *ranges = {{{c->k, pb}, {c->v, pb}, {c->k_scale, sb}, {c->v_scale, sb}}};
  *out = {c->format, c->num_pages, P,          c->Hk,      c->d,           c->B,
          c->max_pages, c->k,      c->v,       c->k_scale, c->v_scale,     c->block_table,
          nullptr};
  return MODA_OK;
}

// Every range of `outs` apart from all of `ins` and from one another.
moda_status check_apart(const Range* outs, int no, const Range* ins, int ni) {
  for (int a = 0; a < no; ++a) {
    for (int b = 0; b < ni; ++b)
      if (overlaps(outs[a], ins[b]))
        return report(MODA_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    for (int b = a + 1; b < no; ++b)
      if (overlaps(outs[a], outs[b])) return report(MODA_ERR_INVALID_ARG, "outputs overlap");
  }
  return MODA_OK;
}

constexpr int kMaxTokens = 1 << 24;

}  // namespace

extern "C" {

moda_status moda_kv_append(const void* q, const void* k, const void* v, long long q_stride,
                           long long k_stride, long long v_stride, const float* rope,
                           int rope_rows, int rot, int interleaved, const int* seq, const int* pos,
                           int N, int Hq, const moda_paged_kv* cache, void* q_out, void* k_out,
                           moda_stream_t stream) {
  moda::KvAppendArgs a{};
  CacheRanges cr;
  moda_status st = check_cache(cache, &a.c, &cr);
  if (st != MODA_OK) return st;
  const int d = a.c.d, Hk = a.c.Hk;
  if (N < 0) return report(MODA_ERR_INVALID_ARG, "N = %d < 0", N);
  if (Hq < 0) return report(MODA_ERR_INVALID_ARG, "Hq = %d < 0", Hq);
  if (N > kMaxTokens) return report(MODA_ERR_UNSUPPORTED, "N = %d > 2^24", N);
  if (Hq > 4096) return report(MODA_ERR_UNSUPPORTED, "Hq = %d > 4096", Hq);
  if ((int64_t)N * ((int64_t)Hq + 2 * Hk) > 0x7fffffffLL)
    return report(MODA_ERR_UNSUPPORTED, "N * (Hq + 2 Hk) = %lld rows exceed 2^31 - 1",
                  (long long)N * ((long long)Hq + 2 * Hk));
  if (rot < 0) return report(MODA_ERR_INVALID_ARG, "rot = %d < 0", rot);
  if (rot > d || rot % 16 != 0)
    return report(MODA_ERR_UNSUPPORTED, "rot = %d (a multiple of 16 up to d = %d)", rot, d);
  if (rot > 0 && (!rope || rope_rows < 1))
    return report(MODA_ERR_INVALID_ARG, "NULL or empty rope with rot = %d", rot);
  if (N == 0) return ok();
  if (!k || !v || !seq || !pos || (Hq > 0 && (!q || !q_out)))
    return report(MODA_ERR_INVALID_ARG, "NULL input or output");
  if (N == 1) {
    q_stride = (long long)Hq * d;
    k_stride = v_stride = (long long)Hk * d;
  }
  if (k_stride < (long long)Hk * d || v_stride < (long long)Hk * d || k_stride % 8 || v_stride % 8 ||
      (Hq > 0 && (q_stride < (long long)Hq * d || q_stride % 8)))
    return report(MODA_ERR_INVALID_ARG,
                  "strides %lld, %lld, %lld must be multiples of 8 and at least a token's row",
                  q_stride, k_stride, v_stride);
  const long long most = 1LL << 36;  // elements between tokens; keeps byte counts in 64 bits
  if (k_stride > most || v_stride > most || (Hq > 0 && q_stride > most))
    return report(MODA_ERR_UNSUPPORTED, "a token stride exceeds 2^36 elements");
  if (Hq == 0) q = q_out = nullptr;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(k_out, 16) || (rot > 0 && !aligned(rope, 16)) || !aligned(seq, 4) || !aligned(pos, 4))
    return report(MODA_ERR_MISALIGNED, "a tensor pointer is not 16-byte (seq, pos: 4-byte) aligned");
  auto span = [&](long long stride, int H) {
    return ((size_t)(N - 1) * stride + (size_t)H * d) * 2;
  };
  const Range ins[] = {{q, Hq > 0 ? span(q_stride, Hq) : 0},
                       {k, span(k_stride, Hk)},
                       {v, span(v_stride, Hk)},
                       {rope, rot > 0 ? (size_t)rope_rows * rot * 4 : 0},
                       {seq, (size_t)N * 4},
                       {pos, (size_t)N * 4},
                       {a.c.table, (size_t)a.c.B * a.c.max_pages * 4}};
  const Range outs[] = {{q_out, (size_t)N * Hq * d * 2},
                        {k_out, (size_t)N * Hk * d * 2},
                        cr.r[0], cr.r[1], cr.r[2], cr.r[3]};
  st = check_apart(outs, 6, ins, 7);
  if (st != MODA_OK) return st;
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.rope = rope; a.rope_rows = rope_rows; a.rot = rot; a.interleaved = interleaved != 0;
  a.seq = seq; a.pos = pos; a.N = N; a.Hq = Hq;
  a.q_out = q_out; a.k_out = k_out;
  int dev;
  st = moda::device_info(&dev, &a.c.err, &a.num_sms);
  if (st != MODA_OK) return st;
  const cudaError_t e = moda::launch_kv_append(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return report(MODA_ERR_CUDA, "kv_append launch: %s", cudaGetErrorString(e));
  return ok();
}

moda_status moda_kv_gather(const moda_paged_kv* cache, const int* seq, const int* pos, int N,
                           void* k, void* v, moda_stream_t stream) {
  moda::PagedKv c;
  CacheRanges cr;
  moda_status st = check_cache(cache, &c, &cr);
  if (st != MODA_OK) return st;
  if (N < 0) return report(MODA_ERR_INVALID_ARG, "N = %d < 0", N);
  if (N > kMaxTokens) return report(MODA_ERR_UNSUPPORTED, "N = %d > 2^24", N);
  if (N == 0) return ok();
  if (!seq || !pos || !k || !v) return report(MODA_ERR_INVALID_ARG, "NULL input or output");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(seq, 4) || !aligned(pos, 4))
    return report(MODA_ERR_MISALIGNED, "a tensor pointer is not 16-byte (seq, pos: 4-byte) aligned");
  const size_t ob = (size_t)N * c.Hk * c.d * 2;
  const Range ins[] = {cr.r[0], cr.r[1], cr.r[2], cr.r[3],
                       {seq, (size_t)N * 4},
                       {pos, (size_t)N * 4},
                       {c.table, (size_t)c.B * c.max_pages * 4}};
  const Range outs[] = {{k, ob}, {v, ob}};
  st = check_apart(outs, 2, ins, 7);
  if (st != MODA_OK) return st;
  int dev, sms;
  st = moda::device_info(&dev, &c.err, &sms);
  if (st != MODA_OK) return st;
  const cudaError_t e = moda::launch_kv_gather(c, seq, pos, N, k, v, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return report(MODA_ERR_CUDA, "kv_gather launch: %s", cudaGetErrorString(e));
  return ok();
}

size_t moda_decode_paged_workspace_bytes(int Hq, int Hk, int d) {
  if (Hk < 1 || Hq < Hk || Hq % Hk != 0 || Hq / Hk > 16 || (d != 64 && d != 128)) return 0;
  return moda::decode_paged_workspace_bytes(Hq, Hk, d);
}

moda_status moda_decode_paged(const void* q, const moda_paged_kv* cache, const int* seq_lens,
                              const void* kd, const void* vd, long long depth_b_stride,
                              long long depth_hk_stride, long long depth_slot_stride, int Hq,
                              int L, float scale, void* o, float* lse, float* workspace,
                              size_t workspace_bytes, moda_stream_t stream) {
  moda::DecodePagedArgs a{};
  CacheRanges cr;
  moda_status st = check_cache(cache, &a.c, &cr);
  if (st != MODA_OK) return st;
  const int d = a.c.d, Hk = a.c.Hk, B = a.c.B;
  if (Hq < 1) return report(MODA_ERR_INVALID_ARG, "Hq = %d < 1", Hq);
  if (Hq % Hk != 0) return report(MODA_ERR_INVALID_ARG, "Hq = %d not a multiple of Hk = %d", Hq, Hk);
  if (L < 0) return report(MODA_ERR_INVALID_ARG, "L = %d < 0", L);
  // the kernels work with scale * log2(e)
  if (!(scale > 0.f) || scale > 2e38f)
    return report(MODA_ERR_INVALID_ARG, "scale must be positive and at most 2e38");
  const int G = Hq / Hk;
  if (G > 16) return report(MODA_ERR_UNSUPPORTED, "G = Hq/Hk = %d (supported: 1 to 16)", G);
  if (L > 1024) return report(MODA_ERR_UNSUPPORTED, "L = %d > 1024", L);
  if ((int64_t)B * Hq > (1 << 24))
    return report(MODA_ERR_UNSUPPORTED, "B * Hq = %lld > 2^24", (long long)B * Hq);
  if (B == 0) return ok();
  if (!q || !seq_lens || !o || !workspace)
    return report(MODA_ERR_INVALID_ARG, "NULL q, seq_lens, o or workspace");
  if (L > 0 && (!kd || !vd)) return report(MODA_ERR_INVALID_ARG, "NULL kd or vd with L = %d", L);
  size_t db = 0;
  if (L > 0) {
    // a stride along an axis of length 1 is never stepped
    if (L == 1) depth_slot_stride = d;
    if (Hk == 1) depth_hk_stride = (long long)L * d;
    if (B == 1) depth_b_stride = (long long)Hk * L * d;
    const long long s[3] = {depth_b_stride, depth_hk_stride, depth_slot_stride};
    for (long long x : s)
      if (x < d || x % 8 != 0 || x >= (1LL << 38))
        return report(MODA_ERR_INVALID_ARG,
                      "depth strides (sequence %lld, KV head %lld, slot %lld) must be multiples of "
                      "8, at least d and below 2^38",
                      s[0], s[1], s[2]);
    db = ((size_t)(B - 1) * depth_b_stride + (size_t)(Hk - 1) * depth_hk_stride +
          (size_t)(L - 1) * depth_slot_stride + d) * 2;
  } else {
    kd = vd = nullptr;
  }
  const size_t need = moda::decode_paged_workspace_bytes(Hq, Hk, d);
  if (workspace_bytes < need)
    return report(MODA_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  if (!aligned(q, 16) || !aligned(kd, 16) || !aligned(vd, 16) || !aligned(o, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(seq_lens, 4))
    return report(MODA_ERR_MISALIGNED,
                  "a tensor pointer is not 16-byte (seq_lens, lse: 4-byte) aligned");
  const size_t qb = (size_t)B * Hq * d * 2;
  const Range ins[] = {{q, qb}, cr.r[0], cr.r[1], cr.r[2], cr.r[3], {kd, db}, {vd, db},
                       {seq_lens, (size_t)B * 4},
                       {a.c.table, (size_t)B * a.c.max_pages * 4}};
  const Range outs[] = {{o, qb}, {lse, lse ? (size_t)B * Hq * 4 : 0}, {workspace, need}};
  st = check_apart(outs, 3, ins, 9);
  if (st != MODA_OK) return st;
  a.q = q; a.kd = kd; a.vd = vd;
  a.seq_lens = seq_lens;
  a.depth_b_stride = depth_b_stride; a.depth_hk_stride = depth_hk_stride;
  a.depth_slot_stride = depth_slot_stride;
  a.Hq = Hq; a.G = G; a.L = L; a.scale = scale;
  a.o = o; a.lse = lse; a.work = workspace;
  int dev;
  st = moda::device_info(&dev, &a.c.err, &a.num_sms);
  if (st != MODA_OK) return st;
  const cudaError_t e = moda::launch_decode_paged(a, (cudaStream_t)stream);
  if (e != cudaSuccess)
    return report(MODA_ERR_CUDA, "decode_paged launch: %s", cudaGetErrorString(e));
  return ok();
}

}  // extern "C"
