"""Chunks of new tokens and selected pages over the paged KV cache, as cases to time and
compare.

A server of a MoDA model does more over its paged cache than one token at a time over
all rows. Four operators do that:

  prefill   several new tokens of each sequence (the next piece of a prompt, a draft to
            verify) attend, under one softmax, to the rows of their sequence's pages up to
            their own and to their own L depth slots; bf16 or 4-bit pages
  means     the mean key of each page that a step has filled, the page's summary
  select    for each token and KV head the pages that are worth attending to: the first,
            the last, and those whose summaries score highest against the group's queries
  selected  one new token per sequence attends to the rows of its selected pages and to
            its L depth slots

``run`` computes them in elementary torch operations, or, where ``own`` is true, by the
library's calls. Sequence lengths of a batch follow from the case alone.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request's draft of five tokens, verified: the latency of a single small call
        dict(name="prefill 5 tokens at 701", op="prefill", fmt="bf16", B=1, new_lo=5, new_hi=5, past_lo=696,
             past_hi=696, pad=0, Hq=16, Hk=4, d=128, L=46, page=64),
        # drafts of a whole batch at once, contexts of very different lengths, the batch
        # padded to its captured size
        dict(name="prefill 32 drafts", op="prefill", fmt="bf16", B=32, new_lo=1, new_hi=8, past_lo=0,
             past_hi=16000, pad=3, Hq=16, Hk=4, d=128, L=24, page=32),
        # one piece of a very long prompt
        dict(name="prefill 2048 tokens at 65536", op="prefill", fmt="bf16", B=1, new_lo=2048, new_hi=2048,
             past_lo=63488, past_hi=63488, pad=0, Hq=16, Hk=4, d=128, L=48, page=64),
        # several prompts' next pieces at once, small heads
        dict(name="prefill 7 ragged prompts d64", op="prefill", fmt="bf16", B=7, new_lo=5, new_hi=2901,
             past_lo=0, past_hi=9001, pad=0, Hq=64, Hk=8, d=64, L=64, page=16),
        # a piece of a prompt whose cache is kept in 4 bits
        dict(name="prefill mx4 1024 tokens at 32768", op="prefill", fmt="mx4", B=1, new_lo=1024, new_hi=1024,
             past_lo=31744, past_hi=31744, pad=0, Hq=16, Hk=4, d=128, L=48, page=64),
        # short drafts over 4-bit rows
        dict(name="prefill mx4 16 drafts", op="prefill", fmt="mx4", B=16, new_lo=1, new_hi=17, past_lo=0,
             past_hi=4001, pad=1, Hq=32, Hk=4, d=128, L=24, page=16),
        # a decode step of a full batch: the sequences that have just filled a page
        dict(name="means of 253 tokens mx4", op="means", fmt="mx4", B=253, new_lo=1, new_hi=1, past_lo=1,
             past_hi=8191, pad=3, Hk=4, d=128, page=16),
        # the pages of a long prompt
        dict(name="means of a prompt of 16384", op="means", fmt="bf16", B=1, new_lo=16384, new_hi=16384,
             past_lo=0, past_hi=0, pad=0, Hk=4, d=128, page=64),
        # one request with a long context
        dict(name="select 1x65536", op="select", B=1, lo=65536, hi=65536, pad=0, Hq=16, Hk=4, d=128, page=64,
             S=32, sink=1, recent=2),
        # a large ragged batch over small pages, padded
        dict(name="select 64 ragged", op="select", B=64, lo=1, hi=32768, pad=2, Hq=32, Hk=4, d=128, page=16,
             S=64, sink=1, recent=4),
        # the long context again, an eighth of its pages or fewer
        dict(name="selected 1x65536", op="selected", fmt="bf16", B=1, lo=65536, hi=65536, pad=0, Hq=16, Hk=4,
             d=128, L=48, page=64, S=32),
        # the large ragged batch with 4-bit rows
        dict(name="selected mx4 64 ragged", op="selected", fmt="mx4", B=64, lo=1, hi=32768, pad=2, Hq=32, Hk=4,
             d=128, L=24, page=16, S=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "prefill", "means", "select", "selected"))
    fmt = rng.choice(("bf16", "mx4"))
    d = rng.choice((64, 128, 128))
    Hk = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 8, 16)) if Hk < 8 else rng.choice((1, 2, 4, 8))
    if rng.random() < 0.2:  # groups of other sizes
        G = rng.choice((3, 5, 6, 7))
    page = rng.choice((16, 32, 64, 128))
    pad = rng.choice((0, 0, 1, 5))
    if op == "prefill":
        if rng.random() < 0.4:  # a batch of drafts
            B, new_hi = _log(rng, 1, 64), rng.randint(1, 32)
        else:  # pieces of prompts
            B = rng.randint(1, 8)
            new_hi = _log(rng, 8, 8192 // B)
        past_hi = _log(rng, 1, min(65536, 400000 // B))
        c = dict(op=op, fmt=fmt, B=B, new_lo=rng.randint(1, new_hi), new_hi=new_hi,
                 past_lo=rng.randint(0, past_hi), past_hi=past_hi, pad=pad, Hq=Hk * G, Hk=Hk, d=d,
                 L=rng.choice((0, 4, 24, 46, 96)), page=page)
        while work(c)["bytes"] > 5e8 or work(c)["flops"] > 1e12:  # no more than the largest listed case
            c.update(past_lo=c["past_lo"] // 2, past_hi=c["past_hi"] // 2, new_lo=(c["new_lo"] + 1) // 2,
                     new_hi=(c["new_hi"] + 1) // 2)
        return c
    if op == "means":
        if rng.random() < 0.5:
            B, new_lo, new_hi = _log(rng, 30, 300), 1, 1
        else:
            B = rng.randint(1, 8)
            new_hi = _log(rng, 2, 16384 // B)
            new_lo = rng.randint(1, new_hi)
        past_hi = _log(rng, 100, 30000 if B < 16 else 8000)
        return dict(op=op, fmt=fmt, B=B, new_lo=new_lo, new_hi=new_hi, past_lo=rng.randint(0, past_hi),
                    past_hi=past_hi, pad=pad, Hk=Hk, d=d, page=page)
    B = _log(rng, 1, 96)
    hi = _log(rng, 100, min(65536, 1000000 // B))
    lo = hi if B == 1 else rng.randint(1, hi)
    S = rng.choice((4, 16, 17, 32, 64))
    if op == "select":
        sink = rng.randint(0, 2)
        return dict(op=op, B=B, lo=lo, hi=hi, pad=pad, Hq=Hk * G, Hk=Hk, d=d, page=page, S=S, sink=sink,
                    recent=rng.randint(1, 4 - sink))
    c = dict(op=op, fmt=fmt, B=B, lo=lo, hi=hi, pad=pad, Hq=Hk * G, Hk=Hk, d=d, L=rng.choice((0, 4, 24, 46, 96)),
             page=page, S=S)
    while work(c)["bytes"] > 5e8:
        c.update(lo=(c["lo"] + 1) // 2, hi=(c["hi"] + 1) // 2)
    return c


def _spread(n, lo, hi, turn):
    """n whole numbers in [lo, hi], both ends among them when n > 1, in no order."""
    if n == 1:
        return [hi]
    got = [lo + int(((i + 1) * turn % 1.0) * (hi - lo + 1)) for i in range(n)]
    got[n // 2], got[n // 3] = lo, hi
    return got


def _lens(case):
    """Rows of each sequence that its pages hold when the pass is over, and how many of
    them are the pass's own."""
    if "new_hi" in case:
        past = _spread(case["B"], case["past_lo"], case["past_hi"], 0.6180339887)
        new = _spread(case["B"], case["new_lo"], case["new_hi"], 0.7548776662)
        return [p + n for p, n in zip(past, new)], new
    return _spread(case["B"], case["lo"], case["hi"], 0.6180339887), [1] * case["B"]


def _row_bytes(case):
    """Bytes of one key or value row of one head in the pages."""
    return case["d"] * 2 if case["fmt"] == "bf16" else case["d"] // 2 + case["d"] // 32


def work(case):
    lens, new = _lens(case)
    Hk, d, page, B = case["Hk"], case["d"], case["page"], case["B"]
    held = [-(-e // page) for e in lens]
    if case["op"] == "prefill":
        Hq, L, n = case["Hq"], case["L"], sum(new)
        b = 2 * sum(lens) * Hk * _row_bytes(case) + 2 * n * Hk * L * d * 2 + n * Hq * (4 * d + 4)
        b += 4 * (2 * B + 1) + 4 * sum(held)
        pairs = sum(m * (e - m) + m * (m + 1) // 2 + m * L for e, m in zip(lens, new))
        return {"bytes": b, "flops": 4 * d * Hq * pairs}
    if case["op"] == "means":
        full = sum(e // page - (e - m) // page for e, m in zip(lens, new))
        return {"bytes": full * Hk * (page * _row_bytes(case) + 2 * d) + 8 * (sum(new) + case["pad"]) + 4 * full,
                "flops": full * Hk * page * d}
    Hq, S = case["Hq"], case["S"]
    if case["op"] == "select":
        scored = sum(m for m in held if m > S)  # a sequence of few pages keeps them all
        return {"bytes": scored * Hk * d * 2 + 2 * B * Hq * d + 8 * B + 4 * sum(held)
                + 4 * (B + case["pad"]) * Hk * (S + 1),
                "flops": 2 * d * Hq * scored}
    L = case["L"]
    rows = sum(_rows_of(e, page, S) for e in lens)
    return {"bytes": 2 * rows * Hk * _row_bytes(case) + 2 * B * Hk * L * d * 2 + B * Hq * (4 * d + 4)
            + 4 * B * Hk * (S + 1),
            "flops": 4 * d * Hq * (rows + B * L)}


def _rows_of(length, page, S):
    """Rows in the S pages that a token at the end of `length` rows selects."""
    held = -(-length // page)
    return (min(held, S) - 1) * page + (length - 1) % page + 1


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """Codes [..., d/2] and scales [..., d/32] (bytes) of x [..., d]: blocks of 32, the
    smallest power of two whose sevenfold is not below the block's largest magnitude,
    values to the nearest e2m1."""
    blk = x.reshape(*x.shape[:-1], -1, 32).float()
    m, e = torch.frexp(blk.abs().amax(-1))
    e = torch.where(m > 0.875, e - 2, e - 3).clamp(min=-126)
    a = torch.ldexp(blk, -e.unsqueeze(-1)).abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() +
            (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code + torch.signbit(blk).byte() * 8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _pool(case, pages, g):
    """Key and value pages [pages, Hk, page, d] with rows of N(0, 1) in them."""
    shape = (pages, case["Hk"], case["page"], case["d"])
    got = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        got.append((x, None) if case["fmt"] == "bf16" else _quantise(x))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = dict(generator=g, device=DEV, dtype=torch.bfloat16)
    lens, new = _lens(case)
    B, Hk, d, page, pad = case["B"], case["Hk"], case["d"], case["page"], case["pad"]
    N = sum(new) + pad
    # the pages of the batch lie anywhere in the pool; entries past a sequence's end are 0
    held = torch.tensor([-(-e // page) for e in lens], device=DEV)
    width = max(1, int(held.max()))
    total = int(held.sum()) + 2
    used = torch.arange(width, device=DEV) < held[:, None]
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    table[used] = torch.randperm(total, generator=g, device=DEV)[: total - 2].to(torch.int32)
    s = {"case": dict(case), "table": table}
    if case["op"] == "select":
        # the choice reads no rows: the pages' shape says all that it needs of them
        s["k_pages"] = s["v_pages"] = torch.zeros((total, Hk, page, d), dtype=torch.bfloat16, device=DEV)
        # the means of `page` keys each, about as long as keys that have something in common
        s["means"] = torch.randn((total, Hk, d), **normal) * 0.5
    else:
        s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"] = _pool(case, total, g)

    if case["op"] == "prefill":
        starts = [0]
        for m in new:
            starts.append(starts[-1] + m)
        s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        L = case["L"]
        # the depth keys and values as the layers below have written them for these tokens
        s["kd"] = torch.randn((L, N, Hk, d), **normal) if L else None
        s["vd"] = torch.randn((L, N, Hk, d), **normal) if L else None
    else:
        seq = [torch.full((m,), b, dtype=torch.int32) for b, m in enumerate(new)]
        pos = [torch.arange(e - m, e, dtype=torch.int32) for e, m in zip(lens, new)]
        s["seq"] = torch.cat(seq + [torch.full((pad,), -1, dtype=torch.int32)]).to(DEV)
        s["pos"] = torch.cat(pos + [torch.zeros(pad, dtype=torch.int32)]).to(DEV)
    if case["op"] == "means":
        s["means"] = torch.zeros((total, Hk, d), dtype=torch.bfloat16, device=DEV)
        return s
    s["q"] = torch.randn((N, case["Hq"], d), **normal)
    if case["op"] == "select":
        s["pages"] = torch.zeros((N, Hk, case["S"]), dtype=torch.int32, device=DEV)
        s["rows"] = torch.zeros((N, Hk), dtype=torch.int32, device=DEV)
        return s
    s["scale"] = d ** -0.5
    s["o"] = torch.zeros((N, case["Hq"], d), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((N, case["Hq"]), dtype=torch.float32, device=DEV)
    if case["op"] == "selected":
        # a choice as `select` makes it: for each KV head some of the pages, in order,
        # the last one among them
        S = case["S"]
        kept = torch.clamp(held, max=S)
        draw_ = torch.rand((B, Hk, width), generator=g, device=DEV)
        page_no = torch.arange(width, device=DEV)
        draw_ = torch.where(page_no < held[:, None, None], draw_, torch.full_like(draw_, -1.0))
        draw_ = torch.where(page_no == held[:, None, None] - 1, torch.full_like(draw_, 2.0), draw_)
        top = draw_.topk(min(S, width), -1).indices
        first = torch.arange(top.shape[-1], device=DEV) < kept[:, None, None]
        top = torch.where(first, top, torch.full_like(top, width)).sort(-1).values
        ids = torch.gather(table[:, None].expand(-1, Hk, -1).long(), 2, top.clamp(max=width - 1))
        ids = ids * Hk + torch.arange(Hk, device=DEV)[:, None]
        s["pages"] = torch.full((N, Hk, S), -1, dtype=torch.int32, device=DEV)
        s["pages"][:B, :, : top.shape[-1]] = torch.where(first, ids, torch.full_like(ids, -1)).int()
        s["rows"] = torch.zeros((N, Hk), dtype=torch.int32, device=DEV)
        s["rows"][:B] = torch.tensor([_rows_of(e, page, S) for e in lens], dtype=torch.int32, device=DEV)[:, None]
        L = case["L"]
        s["kd"] = torch.randn((N, Hk, L, d), **normal) if L else None
        s["vd"] = torch.randn((N, Hk, L, d), **normal) if L else None
    return s


# -------------------------------------------------------------- the plain forms
def _values(codes, scales):
    """fp32 values of 4-bit rows (of bf16 rows where there are no scales)."""
    if scales is None:
        return codes.float()
    lut = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    e = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return (v.reshape(*scales.shape, 32) * e.unsqueeze(-1)).reshape(v.shape)


def _softmax_parts(z):
    """exp(z - max), its sum and the max, for rows in which anything may be masked."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    return p, p.sum(-1, keepdim=True), m


def _plain_prefill(s):
    c = s["case"]
    Hk, Hq, d, L, page = c["Hk"], c["Hq"], c["d"], c["L"], c["page"]
    lens, new = _lens(c)
    at = 0
    for b, (e, m) in enumerate(zip(lens, new)):
        here = slice(at, at + m)
        at += m
        ids = s["table"][b, : -(-e // page)].long()
        row = torch.arange(e - m, e, device=DEV)[:, None]
        hidden = torch.arange(e, device=DEV) > row  # [m, e]
        for h in range(Hk):
            heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k = _values(s["k_pages"][ids, h], None if s["k_scales"] is None else s["k_scales"][ids, h])
            v = _values(s["v_pages"][ids, h], None if s["v_scales"] is None else s["v_scales"][ids, h])
            k, v = k.reshape(-1, d)[:e], v.reshape(-1, d)[:e]
            q = s["q"][here, heads].float()  # [m, G, d]
            z = (q.reshape(-1, d) @ k.T).view(m, -1, e) * s["scale"]
            z.masked_fill_(hidden[:, None], -math.inf)
            if L:
                kd, vd = s["kd"][:, here, h].float(), s["vd"][:, here, h].float()  # [L, m, d]
                z = torch.cat((z, torch.einsum("mgd,lmd->mgl", q, kd) * s["scale"]), -1)
            p, total, top = _softmax_parts(z)
            o = (p[..., :e].reshape(-1, e) @ v).view(m, -1, d)
            if L:
                o = o + torch.einsum("mgl,lmd->mgd", p[..., e:], vd)
            s["o"][here, heads] = (o / total).bfloat16()
            s["lse"][here, heads] = (top + torch.log(total))[..., 0]
    return {"o": s["o"], "lse": s["lse"]}


def _plain_means(s):
    c = s["case"]
    fills = (s["seq"] >= 0) & (s["pos"] % c["page"] == c["page"] - 1)
    seq, pos = s["seq"][fills].long(), s["pos"][fills].long()
    ids = s["table"][seq, pos // c["page"]].long()
    rows = _values(s["k_pages"][ids], None if s["k_scales"] is None else s["k_scales"][ids])
    s["means"][ids] = (rows.sum(2) / c["page"]).bfloat16()
    return {"means": s["means"]}


def _plain_select(s):
    c = s["case"]
    Hk, d, S, page = c["Hk"], c["d"], c["S"], c["page"]
    real = s["seq"] >= 0
    seq, pos = s["seq"][real].long(), s["pos"][real].long()
    table = s["table"][seq].long()  # [n, width]
    n, width = table.shape
    q = s["q"][real].double().view(n, Hk, -1, d)
    means = s["means"].transpose(0, 1)
    score = torch.stack([(q[:, h] @ means[h][table].double().transpose(1, 2)).amax(1) for h in range(Hk)], 1)
    last = (pos // page)[:, None, None]
    at = torch.arange(width, device=DEV)
    always = (at < c["sink"]) | (at > last - c["recent"])
    score = torch.where(always, torch.full_like(score, math.inf), score)
    score = torch.where(at > last, torch.full_like(score, -math.inf), score)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :S]
    taken = torch.where(order > last, torch.full_like(order, width), order).sort(-1).values
    ids = torch.gather(table[:, None].expand(-1, Hk, -1), 2, taken.clamp(max=width - 1)) * Hk
    ids = ids + torch.arange(Hk, device=DEV)[:, None]
    s["pages"].fill_(-1)
    s["rows"].zero_()
    full = torch.full((n, Hk, S), -1, dtype=torch.int32, device=DEV)
    full[..., : taken.shape[-1]] = torch.where(taken < width, ids, torch.full_like(ids, -1)).int()
    s["pages"][real] = full
    held = torch.clamp(pos // page + 1, max=S)
    s["rows"][real] = ((held - 1) * page + pos % page + 1).int()[:, None].expand(-1, Hk).contiguous()
    return {"pages": s["pages"], "rows": s["rows"]}


def _plain_selected(s):
    c = s["case"]
    Hk, d, L = c["Hk"], c["d"], c["L"]
    N = s["q"].shape[0]
    ids = s["pages"].clamp(min=0).long()

    def dense(name):  # [N, Hk, S * page, d]
        x, sc = s[name + "_pages"], s[name + "_scales"]
        x = x.flatten(0, 1)[ids]
        return _values(x, None if sc is None else sc.flatten(0, 1)[ids]).flatten(2, 3)

    q = s["q"].float().view(N, Hk, -1, d)
    z = q @ dense("k").transpose(-1, -2) * s["scale"]
    n = z.shape[-1]
    there = torch.arange(n, device=DEV) < s["rows"][..., None]
    z = z.masked_fill(~there[:, :, None], -math.inf)
    if L:
        z = torch.cat((z, q @ s["kd"].float().transpose(-1, -2) * s["scale"]), -1)
    p, total, m = _softmax_parts(z)
    o = p[..., :n] @ dense("v")
    if L:
        o = o + p[..., n:] @ s["vd"].float()
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"o": o.view(N, -1, d).bfloat16(), "lse": (m + torch.log(total)).view(N, -1)}


# ------------------------------------------------------------- the library's calls
def _own_run(s):
    import sequence_depth_attention_gb300 as moda

    c = s["case"]
    pool = (s["k_pages"], s["v_pages"])
    scales = dict(k_scales=s.get("k_scales"), v_scales=s.get("v_scales"))
    if c["op"] == "means":
        return {"means": moda.moda_page_means(*pool, s["table"], s["seq"], s["pos"], s["means"], **scales)}
    if c["op"] == "select":
        pages, rows = moda.moda_select_pages(s["q"], s["means"], *pool, s["table"], s["seq"], s["pos"], c["S"],
                                             sink=c["sink"], recent=c["recent"], pages=s["pages"], rows=s["rows"])
        return {"pages": pages, "rows": rows}
    if "workspace" not in s:
        need = (moda.moda_prefill_paged_workspace_bytes if c["op"] == "prefill"
                else moda.moda_decode_paged_workspace_bytes)(c["Hq"], c["Hk"], c["d"])
        s["workspace"] = torch.empty(need // 4, dtype=torch.float32, device=DEV)
    rest = dict(kd=s["kd"], vd=s["vd"], o=s["o"], lse=s["lse"], workspace=s["workspace"], **scales)
    if c["op"] == "prefill":
        o, lse = moda.moda_prefill_paged(s["q"], *pool, s["table"], s["q_starts"], s["lens"], s["scale"], **rest)
    else:
        o, lse = moda.moda_decode_selected(s["q"], *pool, s["pages"], s["rows"], s["scale"], **rest)
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own_run(state)
    return {"prefill": _plain_prefill, "means": _plain_means, "select": _plain_select,
            "selected": _plain_selected}[state["case"]["op"]](state)


# ---------------------------------------------------------------------- in 64 bits
def _by_byte(codes, scales):
    """Rows in fp64; 4-bit ones through a table of all bytes, low half first."""
    if scales is None:
        return codes.double()
    both = torch.tensor([(E2M1[b % 16], E2M1[b // 16]) for b in range(256)], dtype=torch.float64,
                        device=codes.device)
    x = both[codes.int()].reshape(*scales.shape, 32)
    return (x * torch.exp2(scales.double() - 127).unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _attend(q, k, v, seen, scale):
    """o and lse of queries [h, d] over keys and values [n, d]; `seen` [h, n] or None."""
    z = q @ k.T * scale
    if seen is not None:
        z = torch.where(seen, z, torch.full_like(z, -math.inf))
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lens(case)
    Hk, d, page = case["Hk"], case["d"], case["page"]

    def rows(name, ids, h):  # head h's rows of some pages
        sc = s[name + "_scales"]
        return _by_byte(s[name + "_pages"][ids, h], None if sc is None else sc[ids, h]).reshape(-1, d)

    if case["op"] == "means":
        means = s["means"].double()
        for b, (e, m) in enumerate(zip(lens, new)):
            ids = s["table"][b, (e - m) // page : e // page].long()
            for h in range(Hk if len(ids) else 0):
                means[ids, h] = rows("k", ids, h).reshape(-1, page, d).mean(1)
        return {"means": means}

    if case["op"] == "select":
        S = case["S"]
        N = s["q"].shape[0]
        pages = torch.full((N, Hk, S), -1, dtype=torch.int32)
        got = torch.zeros((N, Hk), dtype=torch.int32)
        for b, e in enumerate(lens):
            m = (e - 1) // page + 1
            ids = s["table"][b, :m].long()
            got[b] = _rows_of(e, page, S)
            for h in range(Hk):
                q = s["q"][b].view(Hk, -1, d)[h].double()
                score = (s["means"][ids, h].double() @ q.T).amax(1).tolist()
                keep = {i for i in range(m) if i < case["sink"] or i >= m - case["recent"]}
                others = sorted((i for i in range(m) if i not in keep), key=lambda i: (-score[i], i))
                keep = sorted(keep | set(others[: max(0, S - len(keep))]))
                pages[b, h, : len(keep)] = ids.cpu()[keep].int() * Hk + h
        return {"pages": pages.to(DEV), "rows": got.to(DEV)}

    o, lse = s["o"].double(), s["lse"].double()
    L, G = case["L"], case["Hq"] // Hk
    if case["op"] == "prefill":
        # the scores of one KV head at a time, as many of its tokens at once as fit 8 GB
        at = 0
        for b, (e, m) in enumerate(zip(lens, new)):
            ids = s["table"][b, : -(-e // page)].long()
            step = max(1, int(1e9 // (G * (e + L))))
            for h in range(Hk):
                k, v = rows("k", ids, h)[:e], rows("v", ids, h)[:e]
                for t0 in range(0, m, step):
                    n = min(step, m - t0)
                    here, heads = slice(at + t0, at + t0 + n), slice(h * G, (h + 1) * G)
                    q = s["q"][here, heads].double()
                    row = torch.arange(e - m + t0, e - m + t0 + n, device=DEV)
                    seen = (torch.arange(e, device=DEV) <= row[:, None]).repeat_interleave(G, 0)
                    x, y = _attend(q.reshape(-1, d), k, v, seen, s["scale"])
                    x, y = x.view(n, G, d), y.view(n, G)
                    if L:  # the depth slots' own softmax, joined by the two sums
                        kd = s["kd"][:, here, h].double().permute(1, 2, 0)
                        vd = s["vd"][:, here, h].double().transpose(0, 1)
                        z = torch.bmm(q, kd) * s["scale"]
                        w = torch.logsumexp(z, -1)
                        both = torch.logaddexp(y, w)
                        x = x * torch.exp(y - both)[..., None] + torch.bmm(torch.exp(z - both[..., None]), vd)
                        y = both
                    o[here, heads], lse[here, heads] = x, y
            at += m
        return {"o": o, "lse": lse}

    o.zero_()
    lse.fill_(-math.inf)
    k_pages, v_pages = (s[n].flatten(0, 1) for n in ("k_pages", "v_pages"))
    k_scales, v_scales = (None if s[n] is None else s[n].flatten(0, 1) for n in ("k_scales", "v_scales"))
    for n in range(o.shape[0]):
        for h in range(Hk):
            r = int(s["rows"][n, h])
            ids = s["pages"][n, h, : -(-r // page)].long()
            k = v = torch.empty((0, d), dtype=torch.float64, device=DEV)
            if r:
                k = _by_byte(k_pages[ids], None if k_scales is None else k_scales[ids]).reshape(-1, d)[:r]
                v = _by_byte(v_pages[ids], None if v_scales is None else v_scales[ids]).reshape(-1, d)[:r]
            if L:
                k = torch.cat((k, s["kd"][n, h].double()))
                v = torch.cat((v, s["vd"][n, h].double()))
            if r + L:
                heads = slice(h * G, (h + 1) * G)
                o[n, heads], lse[n, heads] = _attend(s["q"][n, heads].double(), k, v, None, s["scale"])
    return {"o": o, "lse": lse}
