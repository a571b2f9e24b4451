"""The paged KV cache's operators, as cases to time and compare.

Serving a MoDA model keeps the sequence keys and values of many requests in one
pool of pages. Four operators work on it:

  append   rotate a step's queries and keys by their positions and write keys and
           values into the pages (bf16 rows, or 4-bit rows: e2m1 values in blocks of
           32 along d that share a power-of-two scale)
  gather   read rows back out of the pages as bf16, for a pass that wants them dense
  decode   one new token per sequence attends, under one softmax, to its pages (bf16 or
           4-bit) and to its L depth slots

``run`` computes them in elementary torch operations, or, where ``own`` is true,
by the library's calls. Sequence lengths of a batch follow from the case alone.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request, one step: the latency of a single small call
        dict(name="append 1 token", op="append", fmt="bf16", B=1, new_lo=1, new_hi=1, past_lo=700,
             past_hi=700, pad=0, Hq=16, Hk=4, d=128, rot=128, interleaved=False, page=64),
        # a full decode batch, each sequence one token further, 4-bit pages; the batch is
        # padded to its captured size
        dict(name="append 253 tokens mx4", op="append", fmt="mx4", B=253, new_lo=1, new_hi=1,
             past_lo=1, past_hi=8191, pad=3, Hq=16, Hk=4, d=128, rot=128, interleaved=False, page=16),
        # a long prompt of one request
        dict(name="append prompt 16384", op="append", fmt="bf16", B=1, new_lo=16384, new_hi=16384,
             past_lo=0, past_hi=0, pad=0, Hq=16, Hk=4, d=128, rot=128, interleaved=False, page=64),
        # several prompts' next pieces at once, part of the head rotated in interleaved pairs
        dict(name="append ragged prompts mx4 d64", op="append", fmt="mx4", B=7, new_lo=5, new_hi=2901,
             past_lo=0, past_hi=30011, pad=0, Hq=64, Hk=8, d=64, rot=32, interleaved=True, page=32),
        # a cached prefix read back for the next piece of its prompt
        dict(name="gather mx4 16001 rows", op="gather", fmt="mx4", B=1, lo=16001, hi=16001, Hk=4,
             d=128, page=64),
        # short prefixes of a few requests
        dict(name="gather bf16 d64", op="gather", fmt="bf16", B=5, lo=3, hi=701, Hk=8, d=64, page=16),
        # one request, short context
        dict(name="decode 1x701", op="decode", fmt="bf16", B=1, lo=701, hi=701, Hq=16, Hk=4, d=128,
             L=46, page=64),
        # one request, long context
        dict(name="decode 1x65536", op="decode", fmt="bf16", B=1, lo=65536, hi=65536, Hq=16, Hk=4,
             d=128, L=48, page=64),
        # a batch of requests of very different lengths, one of them just admitted
        dict(name="decode 48 ragged", op="decode", fmt="bf16", B=48, lo=0, hi=16384, Hq=16, Hk=4,
             d=128, L=24, page=32),
        # the long context again with 4-bit pages
        dict(name="decode mx4 1x65536", op="decode", fmt="mx4", B=1, lo=65536, hi=65536, Hq=16, Hk=4,
             d=128, L=48, page=64),
        # a large ragged batch, the memory that 4 bits make room for
        dict(name="decode mx4 64 ragged", op="decode", fmt="mx4", B=64, lo=1, hi=32768, Hq=32, Hk=4,
             d=128, L=24, page=16),
        # small heads, short odd contexts
        dict(name="decode mx4 16 short d64", op="decode", fmt="mx4", B=16, lo=1, hi=999, Hq=64, Hk=8,
             d=64, L=64, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "append", "gather", "decode", "decode", "decode"))
    fmt = rng.choice(("bf16", "mx4"))
    d = rng.choice((64, 128, 128))
    Hk = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 4, 8, 16)) if Hk < 8 else rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        if rng.random() < 0.5:  # a decode batch
            B, new_lo, new_hi = _log(rng, 1, 300), 1, 1
        else:  # pieces of prompts
            B = rng.randint(1, 8)
            new_hi = _log(rng, 2, 16384 // B)
            new_lo = rng.randint(1, new_hi)
        past_hi = _log(rng, 1, 30000 if B < 16 else 8000)
        return dict(op=op, fmt=fmt, B=B, new_lo=new_lo, new_hi=new_hi,
                    past_lo=rng.randint(0, past_hi), past_hi=past_hi, pad=rng.choice((0, 0, 1, 5)),
                    Hq=Hk * G, Hk=Hk, d=d, rot=rng.choice((32, 64, d)),
                    interleaved=rng.random() < 0.5, page=page)
    if op == "gather":
        B = rng.randint(1, 8)
        hi = _log(rng, 1, 24000 // B)
        return dict(op=op, fmt=fmt, B=B, lo=rng.randint(0, hi - 1) if hi > 1 else 1, hi=hi, Hk=Hk, d=d,
                    page=page)
    B = _log(rng, 1, 96)
    hi = _log(rng, 8, min(65536, 400000 // B))
    c = dict(op=op, fmt=fmt, B=B, lo=hi if B == 1 else rng.randint(0, hi), hi=hi, Hq=Hk * G, Hk=Hk,
             d=d, L=rng.choice((0, 4, 24, 46, 96)), page=page)
    while work(c)["bytes"] > 7e8:  # no more than the largest listed case
        c.update(lo=c["lo"] // 2, hi=c["hi"] // 2)
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
    them the pass brings."""
    if case["op"] == "append":
        past = _spread(case["B"], case["past_lo"], case["past_hi"], 0.6180339887)
        new = _spread(case["B"], case["new_lo"], case["new_hi"], 0.7548776662)
        return [p + n for p, n in zip(past, new)], new
    return _spread(case["B"], case["lo"], case["hi"], 0.6180339887), None


def _row_bytes(case):
    """Bytes of one key or value row of one head in the pages."""
    return case["d"] * 2 if case["fmt"] == "bf16" else case["d"] // 2 + case["d"] // 32


def work(case):
    lens, new = _lens(case)
    Hk, d, page = case["Hk"], case["d"], case["page"]
    row = _row_bytes(case)
    if case["op"] == "append":
        n, Hq, rot = sum(new), case["Hq"], case["rot"]
        positions = len({p for e, m in zip(lens, new) for p in range(e - m, e)})
        b = n * (Hq + 2 * Hk) * d * 2 + positions * rot * 4 + 8 * (n + case["pad"])
        b += 4 * sum((e - 1) // page - (e - m) // page + 1 for e, m in zip(lens, new))
        b += n * (Hq + Hk) * d * 2 + 2 * n * Hk * row
        if case["fmt"] == "mx4":  # the rows as the pages give them back
            b += 2 * n * Hk * d * 2
        return {"bytes": b, "flops": 3 * n * (Hq + Hk) * rot}
    if case["op"] == "gather":
        n = sum(lens)
        return {"bytes": 2 * n * Hk * (row + d * 2) + 8 * n + 4 * sum(-(-e // page) for e in lens),
                "flops": 0}
    n, Hq, L, B = sum(lens), case["Hq"], case["L"], case["B"]
    b = 2 * n * Hk * row + 2 * B * Hk * L * d * 2 + B * Hq * (4 * d + 4)
    b += 4 * B + 4 * sum(-(-e // page) for e in lens)
    return {"bytes": b, "flops": 4 * d * Hq * (n + B * L)}


# ------------------------------------------------------------------ the inputs
def _quantise(x):
    """Codes [..., d/2] and scales [..., d/32] (bytes) of x [..., d], any float type:
    blocks of 32, the smallest power of two whose sevenfold is not below the block's
    largest magnitude (1.75 and 2^2 make 7; 2^-126 at least), values to the nearest e2m1,
    ties to the even code, 7 to 6."""
    blk = x.reshape(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(blk.abs().amax(-1).double())  # amax = m 2^e with m in [0.5, 1)
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
    lens, new = _lens(case)
    B, Hk, d, page = case["B"], case["Hk"], case["d"], case["page"]
    # the pages of the batch lie anywhere in the pool; entries past a sequence's end are 0
    held = torch.tensor([-(-e // page) for e in lens], device=DEV)
    width = max(1, int(held.max()))
    total = int(held.sum()) + 2
    used = torch.arange(width, device=DEV) < held[:, None]
    table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
    table[used] = torch.randperm(total, generator=g, device=DEV)[: total - 2].to(torch.int32)
    s = {"case": dict(case), "table": table}
    s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"] = _pool(case, total, g)

    if case["op"] == "decode":
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        draw_ = dict(generator=g, device=DEV, dtype=torch.bfloat16)
        s["q"] = torch.randn((B, case["Hq"], d), **draw_)
        s["kd"] = torch.randn((B, Hk, case["L"], d), **draw_) if case["L"] else None
        s["vd"] = torch.randn((B, Hk, case["L"], d), **draw_) if case["L"] else None
        s["scale"] = d ** -0.5
        s["o"] = torch.empty((B, case["Hq"], d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((B, case["Hq"]), dtype=torch.float32, device=DEV)
        return s

    first = [e - m for e, m in zip(lens, new)] if new else [0] * B
    seq = [torch.full((e - f,), b, dtype=torch.int32) for b, (e, f) in enumerate(zip(lens, first))]
    pos = [torch.arange(f, e, dtype=torch.int32) for e, f in zip(lens, first)]
    pad = case.get("pad", 0)
    s["seq"] = torch.cat(seq + [torch.full((pad,), -1, dtype=torch.int32)]).to(DEV)
    s["pos"] = torch.cat(pos + [torch.zeros(pad, dtype=torch.int32)]).to(DEV)
    N = s["seq"].numel()
    if case["op"] == "gather":
        s["k"] = torch.zeros((N, Hk, d), dtype=torch.bfloat16, device=DEV)
        s["v"] = torch.zeros((N, Hk, d), dtype=torch.bfloat16, device=DEV)
        return s

    # queries, keys and values side by side, as one projection writes them
    Hq, rot = case["Hq"], case["rot"]
    qkv = torch.randn((N, (Hq + 2 * Hk) * d), generator=g, device=DEV, dtype=torch.bfloat16)
    s["q"] = qkv[:, : Hq * d].view(N, Hq, d)
    s["k"] = qkv[:, Hq * d : (Hq + Hk) * d].view(N, Hk, d)
    s["v"] = qkv[:, (Hq + Hk) * d :].view(N, Hk, d)
    # the model's rotation table: a row of cosines and sines for each position
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(max(lens), dtype=torch.float64, device=DEV)[:, None] * freq
    s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    s["q_out"] = torch.zeros((N, Hq, d), dtype=torch.bfloat16, device=DEV)
    s["k_out"] = torch.zeros((N, Hk, d), dtype=torch.bfloat16, device=DEV)
    if case["fmt"] == "mx4":
        s["k_back"] = torch.zeros((N, Hk, d), dtype=torch.bfloat16, device=DEV)
        s["v_back"] = torch.zeros((N, Hk, d), dtype=torch.bfloat16, device=DEV)
    return s


# -------------------------------------------------------------- the plain forms
def _values(codes, scales):
    """fp32 values of 4-bit rows."""
    lut = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    e = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return (v.reshape(*scales.shape, 32) * e.unsqueeze(-1)).reshape(v.shape)


def _rotated(x, cos, sin, rot, interleaved):
    """x [N, H, d] in fp64 with its first `rot` elements turned by cos, sin [N, rot/2]."""
    x = x.double()
    c, n = cos[:, None].double(), sin[:, None].double()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    real = s["seq"] >= 0
    seq, pos = s["seq"][real].long(), s["pos"][real].long()
    at, off = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    cos, sin = s["rope"][pos].split(c["rot"] // 2, -1)
    s["q_out"][real] = _rotated(s["q"][real], cos, sin, c["rot"], c["interleaved"]).bfloat16()
    k = _rotated(s["k"][real], cos, sin, c["rot"], c["interleaved"])
    s["k_out"][real] = k.bfloat16()
    v = s["v"][real]
    if c["fmt"] == "bf16":
        s["k_pages"][at, :, off] = s["k_out"][real]
        s["v_pages"][at, :, off] = v
        return {n: s[n] for n in ("q_out", "k_out", "k_pages", "v_pages")}
    s["k_pages"][at, :, off], s["k_scales"][at, :, off] = _quantise(k)
    s["v_pages"][at, :, off], s["v_scales"][at, :, off] = _quantise(v)
    s["k_back"][real] = _values(s["k_pages"][at, :, off], s["k_scales"][at, :, off]).bfloat16()
    s["v_back"][real] = _values(s["v_pages"][at, :, off], s["v_scales"][at, :, off]).bfloat16()
    return {n: s[n] for n in ("q_out", "k_out", "k_back", "v_back")}


def _plain_gather(s):
    c = s["case"]
    seq, pos = s["seq"].long(), s["pos"].long()
    at, off = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["fmt"] == "bf16":
        return {"k": s["k_pages"][at, :, off], "v": s["v_pages"][at, :, off]}
    return {n: _values(s[n + "_pages"][at, :, off], s[n + "_scales"][at, :, off]).bfloat16()
            for n in ("k", "v")}


def _plain_decode(s):
    c, table = s["case"], s["table"].long()
    B, Hk, d = c["B"], c["Hk"], c["d"]

    def dense(pages, scales):  # [B, Hk, width * page, d]
        x = pages[table].float() if scales is None else _values(pages[table], scales[table])
        return x.transpose(1, 2).reshape(B, Hk, -1, d)

    q = s["q"].float().view(B, Hk, -1, d)
    z = q @ dense(s["k_pages"], s["k_scales"]).transpose(-1, -2) * s["scale"]
    n = z.shape[-1]
    there = torch.arange(n, device=DEV) < s["lens"][:, None]
    z = z.masked_fill(~there[:, None, None], -math.inf)
    if c["L"]:
        z = torch.cat((z, q @ s["kd"].float().transpose(-1, -2) * s["scale"]), -1)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    o = p[..., :n] @ dense(s["v_pages"], s["v_scales"])
    if c["L"]:
        o = o + p[..., n:] @ s["vd"].float()
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return {"o": o.view(B, -1, d).bfloat16(), "lse": (m + torch.log(total)).view(B, -1)}


# ------------------------------------------------------------- the library's calls
def _own_run(s):
    import sequence_depth_attention_gb300 as moda

    c = s["case"]
    cache = (s["k_pages"], s["v_pages"], s["table"])
    scales = dict(k_scales=s["k_scales"], v_scales=s["v_scales"])
    if c["op"] == "decode":
        if "workspace" not in s:
            n = moda.moda_decode_paged_workspace_bytes(c["Hq"], c["Hk"], c["d"])
            s["workspace"] = torch.empty(n // 4, dtype=torch.float32, device=DEV)
        o, lse = moda.moda_decode_paged(s["q"], *cache, s["lens"], s["scale"], kd=s["kd"], vd=s["vd"],
                                        o=s["o"], lse=s["lse"], workspace=s["workspace"], **scales)
        return {"o": o, "lse": lse}
    if c["op"] == "gather":
        k, v = moda.moda_kv_gather(*cache, s["seq"], s["pos"], k=s["k"], v=s["v"], **scales)
        return {"k": k, "v": v}
    moda.moda_kv_append(s["q"], s["k"], s["v"], *cache, s["seq"], s["pos"], rope=s["rope"],
                        interleaved=c["interleaved"], q_out=s["q_out"], k_out=s["k_out"], **scales)
    if c["fmt"] == "bf16":
        return {n: s[n] for n in ("q_out", "k_out", "k_pages", "v_pages")}
    moda.moda_kv_gather(*cache, s["seq"], s["pos"], k=s["k_back"], v=s["v_back"], **scales)
    return {n: s[n] for n in ("q_out", "k_out", "k_back", "v_back")}


def run(state):
    if own:
        return _own_run(state)
    return {"append": _plain_append, "gather": _plain_gather,
            "decode": _plain_decode}[state["case"]["op"]](state)


# ---------------------------------------------------------------------- in 64 bits
def _by_byte(codes, scales):
    """4-bit rows in fp64 through a table of all bytes: low half first."""
    half = [E2M1[i] for i in range(16)]
    both = torch.tensor([(half[b % 16], half[b // 16]) for b in range(256)], dtype=torch.float64,
                        device=codes.device)
    x = both[codes.int()].reshape(*scales.shape, 32)
    return (x * torch.exp2(scales.double() - 127).unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _nearest(x):
    """fp64 rows as 4-bit rows hold them: by the distance to every e2m1 magnitude."""
    blk = x.reshape(-1, 32)
    big = blk.abs().amax(1)
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.ones_like(big)) / 7))
    e = torch.where(torch.exp2(e - 1) * 7 >= big, e - 1, e)  # log2 may be off next to a border
    e = torch.where(torch.exp2(e) * 7 < big, e + 1, e)
    e = torch.where(big > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    t = blk.abs() / torch.exp2(e)[:, None]
    near, far = torch.zeros_like(t), torch.full_like(t, math.inf)
    for code in (0, 2, 4, 6, 1, 3, 5, 7):  # even codes first: they win the ties
        gap = (t - E2M1[code]).abs()
        near = torch.where(gap < far, torch.full_like(t, E2M1[code]), near)
        far = torch.minimum(gap, far)
    return (torch.copysign(near, blk) * torch.exp2(e)[:, None]).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _lens(case)
    Hk, d, page = case["Hk"], case["d"], case["page"]

    def rows(name, b, n):  # the first n rows of sequence b, [Hk, n, d]
        ids = s["table"][b, : -(-n // page)].long()
        x = s[name + "_pages"][ids]
        x = x.double() if case["fmt"] == "bf16" else _by_byte(x, s[name + "_scales"][ids])
        return x.transpose(0, 1).reshape(Hk, -1, d)[:, :n]

    if case["op"] == "decode":
        os, lses = [], []
        for b, n in enumerate(lens):
            q = s["q"][b].double().view(Hk, -1, d)
            k, v = rows("k", b, n), rows("v", b, n)
            if case["L"]:
                k = torch.cat((k, s["kd"][b].double()), 1)
                v = torch.cat((v, s["vd"][b].double()), 1)
            z = q @ k.transpose(1, 2) * s["scale"]
            if z.shape[-1]:
                lse = torch.logsumexp(z, -1)
                o = torch.exp(z - lse[..., None]) @ v
            else:
                lse = torch.full(z.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
                o = torch.zeros_like(q)
            os.append(o.reshape(-1, d))
            lses.append(lse.reshape(-1))
        return {"o": torch.stack(os), "lse": torch.stack(lses)}

    if case["op"] == "gather":
        return {n: torch.cat([rows(n, b, m).transpose(0, 1) for b, m in enumerate(lens)])
                for n in ("k", "v")}

    out = {"q_out": s["q_out"].double(), "k_out": s["k_out"].double()}
    bf16 = case["fmt"] == "bf16"
    for n in ("k", "v"):
        out[n + ("_pages" if bf16 else "_back")] = s[n + "_pages"].double() if bf16 else s[n + "_back"].double()
    half, at = case["rot"] // 2, 0
    for b, (end, m) in enumerate(zip(lens, new)):
        here = slice(at, at + m)
        at += m
        turn = torch.complex(s["rope"][end - m : end, :half].double(), s["rope"][end - m : end, half:].double())

        def turned(x):  # pairs of elements as complex numbers
            x = x.double().clone()
            lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"]
                      else (slice(0, half), slice(half, 2 * half)))
            y = torch.complex(x[..., lo], x[..., hi]) * turn[:, None]
            x[..., lo], x[..., hi] = y.real, y.imag
            return x

        k, v = turned(s["k"][here]), s["v"][here].double()
        out["q_out"][here], out["k_out"][here] = turned(s["q"][here]), k
        if bf16:
            p = torch.arange(end - m, end, device=DEV)
            ids = s["table"][b][p // page].long()
            out["k_pages"][ids, :, p % page] = k
            out["v_pages"][ids, :, p % page] = v
        else:
            out["k_back"][here], out["v_back"][here] = _nearest(k), _nearest(v)
    return out
