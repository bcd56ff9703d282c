"""Cases for measuring the operators of a paged KV cache held in 4 bits, with their
plain forms.

A cached row (one token's K or V of one head, D values) is held in groups of 32
consecutive values.  For the values x of a group

    m = the largest fp16 <= min(x)
    s = the smallest fp16 >= (max(x) - m) / 15
    n = floor((x - m) / s + 1/2)         whole numbers 0..15; all 0 where s = 0

and the cached value is m + s n.  A group for which m or s is not finite (an infinity
or NaN among its values, or values past fp16's range) has s = NaN and m = 0: all of it
reads as NaN.

Operators (``case["op"]``):

* ``write``  - new K/V rows are quantised into their pages as they are written, and read
  back as the values that they now stand for (which is what comes out).
* ``read``   - rows of a cache are gathered through the block table and given back.
* ``attend`` - dense decode attention over the cached tokens, some query tokens at the
  end of each request (causal among themselves where asked for).
* ``sparse`` - attention over a list of selected tokens for each request and query.

``own`` false: the plain form in torch operations.  ``own`` true: the library.
"""

import math
import zlib

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
TYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)
GROUP = 32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token for each of 16 requests: what every decode step writes
        dict(name="write_token", op="write", B=16, len_lo=1024, len_hi=8192, n_lo=1, n_hi=1,
             page=64, Hkv=8, D=128, type="bf16", fused=0),
        # one to eight drafted tokens for 64 requests, K and V being slices of the fused
        # projection's output; small pages and heads of 64
        dict(name="write_drafts", op="write", B=64, len_lo=100, len_hi=4000, n_lo=1, n_hi=8,
             page=16, Hkv=2, D=64, type="fp16", fused=8),
        # eight prompts of about 16k tokens each
        dict(name="write_prompt", op="write", B=8, len_lo=12000, len_hi=20768, n_lo=0, n_hi=0,
             page=64, Hkv=8, D=128, type="bf16", fused=0),

        # the last 128 tokens of 16 requests, e.g. for a window computed in 16 bits
        dict(name="read_window", op="read", B=16, len_lo=100, len_hi=5000, n_lo=128, n_hi=128,
             page=16, Hkv=2, D=64, type="bf16", fused=0),
        # 16 whole requests of up to 16k tokens, e.g. before a prompt is continued
        dict(name="read_prompt", op="read", B=16, len_lo=2000, len_hi=16384, n_lo=0, n_hi=0,
             page=64, Hkv=8, D=128, type="bf16", fused=0),

        # the paged-KV worked example: a handful of short requests, latency is everything
        dict(name="attend_example", op="attend", lens="403,96,241,30,176", page=16, Hq=8, Hkv=2,
             D=64, Nq=1, causal=False),
        # 64 ragged requests of 1k to 32k tokens in 16-token pages
        dict(name="attend_ragged", op="attend", B=64, len_lo=1024, len_hi=32768, page=16, Hq=32,
             Hkv=8, D=128, Nq=1, causal=False),
        # 32 requests over 7k to 11k tokens, each with four drafted tokens
        dict(name="attend_drafts", op="attend", B=32, len_lo=7001, len_hi=11000, page=64, Hq=32,
             Hkv=8, D=128, Nq=4, causal=True),
        # 16 requests of 131072 tokens: a long decode without a selection
        dict(name="attend_long", op="attend", B=16, len_lo=131072, len_hi=131072, page=64, Hq=64,
             Hkv=8, D=128, Nq=1, causal=False),

        # the worked example with at most 64 selected tokens
        dict(name="sparse_example", op="sparse", lens="403,96,241,30,176", page=16, Hq=8, Hkv=2,
             D=64, Nq=1, k=64, holes=False),
        # 256 requests of 8192 tokens, 1024 selected
        dict(name="sparse_batch", op="sparse", B=256, len_lo=8192, len_hi=8192, page=64, Hq=32,
             Hkv=8, D=128, Nq=1, k=1024, holes=False),
        # 16 requests of 131072 tokens, 2048 selected
        dict(name="sparse_long", op="sparse", B=16, len_lo=131072, len_hi=131072, page=64, Hq=64,
             Hkv=8, D=128, Nq=1, k=2048, holes=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "sparse", "sparse"])
    page = rng.choice([1, 5, 16, 16, 17, 32, 48, 64, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 8, 16])
    D = rng.choice([64, 128, 128])
    B = _log(rng, 1, 256)
    hi = _log(rng, 1, 65536)
    # no more cached tokens than the largest listed cases have
    while B * hi * Hkv * D > 16 * 131072 * 8 * 128:
        hi = max(1, hi // 2)
    c = dict(op=op, B=B, len_lo=max(1, hi // rng.choice([1, 2, 8])), len_hi=hi, page=page,
             Hkv=Hkv, D=D, empty=B > 4 and rng.random() < 0.3)
    if op in ("write", "read"):
        n_hi = rng.choice([0, _log(rng, 1, hi)])  # 0: all of each request
        if n_hi == 0:
            while B * hi * Hkv * D > 131072 * 8 * 128:
                hi = max(1, hi // 2)
            c.update(len_lo=min(c["len_lo"], hi), len_hi=hi)
        while B * n_hi * Hkv * D > 131072 * 8 * 128:
            n_hi = max(1, n_hi // 2)
        c.update(n_lo=rng.choice([0, n_hi]) if B > 4 else n_hi, n_hi=n_hi,
                 type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), fused=rng.choice([0, 0, 1, 4]))
        if op == "read":
            c["fused"] = 0
        return c
    G = rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 12, 16])
    Nq = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
    while B * Nq > 2048 or B * Nq * G * Hkv * hi > 16 * 64 * 131072:
        if Nq > 1:
            Nq -= 1
        elif B > 1:
            B = B // 2
        else:
            hi = hi // 2
    c.update(B=B, len_lo=min(c["len_lo"], hi), len_hi=hi, Hq=G * Hkv, Nq=Nq)
    if op == "attend":
        c["causal"] = rng.random() < 0.5
    else:
        k = _log(rng, 1, 2048)
        while B * Nq * k * Hkv * D > 256 * 1024 * 8 * 128:
            k = max(1, k // 2)
        c.update(k=k, holes=rng.random() < 0.4)
    return c


# ------------------------------------------------------------- block tables

def _layout(c, seed):
    """Lengths, table and rows of a case (host).  The lengths are the case's own; the
    order of the requests and of the pages is the seed's."""
    sizes = sorted((k, v) for k, v in c.items() if k != "name")
    rs = np.random.RandomState(zlib.crc32(repr(sizes).encode()))
    P = c["page"]
    if "lens" in c:
        lens = np.array([int(x) for x in c["lens"].split(",")], np.int64)
    else:
        lens = rs.randint(c["len_lo"], c["len_hi"] + 1, size=c["B"])
        if c.get("empty"):  # a padded batch: some requests hold nothing
            lens[rs.random_sample(c["B"]) < 0.1] = 0
    B = len(lens)
    new = None
    if "n_hi" in c:  # rows written or read: the last tokens of each request
        new = rs.randint(c["n_lo"], c["n_hi"] + 1, size=B) if c["n_hi"] else lens
        new = np.minimum(new, lens)
    extra = int(rs.randint(0, 3))
    rs = np.random.RandomState(seed % (2 ** 31) + 17)
    order = rs.permutation(B) if "lens" not in c else np.arange(B)
    lens = lens[order]
    pages = -(-lens // P)
    total = int(pages.sum())
    num_pages = total + 1 + extra
    deal = rs.permutation(num_pages)[:total].astype(np.int32)
    table = np.full((B, max(1, int(pages.max())) + extra), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = deal[at:at + pages[b]]
        at += pages[b]
    starts = None
    if new is not None:
        starts = np.concatenate([[0], np.cumsum(new[order])]).astype(np.int32)
    return dict(lens=lens.astype(np.int32), table=table, num_pages=num_pages, starts=starts, rs=rs)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _rows(n, c, gen, kind, bias):
    """n tokens of K or V [n, Hkv, D] in fp32: channels of different size, those of K
    with a mean of their own and a few large ones."""
    x = torch.randn((n, c["Hkv"], c["D"]), generator=gen, device="cuda", dtype=torch.float32)
    x.mul_(bias["scale_" + kind])
    return x.add_(bias["mean_" + kind])


def _bias(c, gen):
    shape = (c["Hkv"], c["D"])
    r = [torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) for _ in range(4)]
    big = 1.0 + 3.0 * (r[2].abs() > 2.2).float()
    return dict(scale_k=(0.3 * r[0]).exp() * 0.6, mean_k=r[1] * 0.3 * big,
                scale_v=(0.4 * r[3]).exp() * 0.5, mean_v=torch.zeros_like(r[0]))


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    c = dict(case)
    L = _layout(c, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 3)
    B, N, P, Hkv, D = len(L["lens"]), L["num_pages"], c["page"], c["Hkv"], c["D"]
    s = dict(case=c, B=B, P=P, lens_host=L["lens"].tolist(), lens=_dev(L["lens"]),
             table=_dev(L["table"]))
    bias = _bias(c, gen)
    # the cache, as a user's program holds it: filled by what was written before
    cache = _empty(N, P, Hkv, D)
    if c["op"] != "write":
        step = max(1, (1 << 27) // (P * Hkv * D))
        for i in range(0, N, step):
            n = min(step, N - i)
            k = _rows(n * P, c, gen, "k", bias).to(BF16)
            v = _rows(n * P, c, gen, "v", bias).to(BF16)
            _fill(cache, k, v, i, n)
    s["cache"] = cache
    if L["starts"] is not None:
        n = int(L["starts"][-1])
        t = TYPES[c["type"]]
        s["starts"] = _dev(L["starts"])
        s["starts_host"] = L["starts"].tolist()
        if c["op"] == "write":
            k, v = (_rows(n, c, gen, x, bias).to(t) for x in "kv")
            if c["fused"]:  # [tokens, query heads + K heads + V heads, D]
                qkv = torch.zeros((n, c["fused"] + 2 * Hkv, D), dtype=t, device="cuda")
                qkv[:, c["fused"]:c["fused"] + Hkv] = k
                qkv[:, c["fused"] + Hkv:] = v
                k, v = qkv[:, c["fused"]:c["fused"] + Hkv], qkv[:, c["fused"] + Hkv:]
            s["k"], s["v"] = k, v
        s["out_k"] = torch.empty((n, Hkv, D), dtype=t, device="cuda")
        s["out_v"] = torch.empty((n, Hkv, D), dtype=t, device="cuda")
        return s
    s["q"] = torch.randn((B, c["Nq"], c["Hq"], D), generator=gen, device="cuda").to(BF16)
    if c["op"] == "sparse":
        s["list"] = _dev(_lists(c, L))
    if own:
        from top_sparse_attention_pks_gb300.decoder import Q4Attention, Q4SparseAttention
        if c["op"] == "attend":
            s["att"] = Q4Attention(s["lens"], s["table"], s["q"], cache, causal=c["causal"],
                                   lse=True)
        else:
            s["att"] = Q4SparseAttention(s["lens"], s["table"], s["list"], s["q"], cache,
                                         trim=not c["holes"], lse=True)
    return s


def _lists(c, L):
    """Selected tokens [B, Nq, k]: as a top-k gives them (ascending, -1 behind), or in any
    order with holes."""
    rs, k = L["rs"], c["k"]
    out = np.full((len(L["lens"]), c["Nq"], k), -1, np.int64)
    for b, n in enumerate(L["lens"].tolist()):
        for i in range(c["Nq"]):
            if n <= k:
                pick = np.arange(n)
            else:  # one from each of k equal parts
                edge = np.arange(k + 1) * n // k
                pick = edge[:-1] + (rs.random_sample(k) * np.diff(edge)).astype(np.int64)
            if c["holes"]:
                row = np.full(k, -1)
                at = rs.permutation(k)[:len(pick)]
                row[at] = rs.permutation(pick)
                row[rs.random_sample(k) < 0.1] = -1
                out[b, i] = row
            else:
                out[b, i, :len(pick)] = pick
    return out


def _empty(N, P, Hkv, D):
    if own:
        from top_sparse_attention_pks_gb300.decoder import Q4Cache
        return Q4Cache(N, P, Hkv, D)
    rows = N * P

    def side():
        return dict(code=torch.zeros((rows, Hkv, D // 2), dtype=torch.uint8, device="cuda"),
                    s=torch.zeros((rows, Hkv, D // GROUP), dtype=torch.float16, device="cuda"),
                    m=torch.zeros((rows, Hkv, D // GROUP), dtype=torch.float16, device="cuda"))
    return dict(k=side(), v=side())


def _fill(cache, k, v, page, n):
    """Pages page .. page + n of a new cache, whole."""
    if own:
        P = k.shape[0] // n
        lens = torch.tensor([n * P], dtype=torch.int32, device="cuda")
        table = torch.arange(page, page + n, dtype=torch.int32, device="cuda")[None]
        starts = torch.tensor([0, n * P], dtype=torch.int32, device="cuda")
        cache.write(k, v, lens, table, starts)
        return
    P = k.shape[0] // n
    for name, x in (("k", k), ("v", v)):
        _put(cache[name], slice(page * P, (page + n) * P), x)


# ------------------------------------------------------------- plain form

def _beside(h, up):
    """The next fp16 above (or below) each h; the infinities lie beyond 65504."""
    bits = h.view(torch.int16)
    away = torch.where(bits >= 0, 1, -1) * (1 if up else -1)
    zero = torch.full_like(bits, 1 if up else -32767)  # the smallest of its sign
    return torch.where(h == 0, zero, (bits + away).to(torch.int16)).view(torch.float16)


def _quantise(x):
    """x [..., D] -> codes (uint8 [..., D]), s and m (fp16 [..., D / 32])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    m = lo.half()
    m = torch.where(m.float() > lo, _beside(m, False), m)
    # what lies next to a border between two numbers needs more than 32 bits
    y = hi.double() - m.double()
    y = y / torch.full_like(y, 15.0)
    s = y.half()
    s = torch.where(s.double() < y, _beside(s, True), s)
    less = _beside(s, False)
    s = torch.where((s > 0) & (less.double() >= y), less, s)
    bad = ~(m.isfinite() & s.isfinite())
    d = (g.double() - m.double()[..., None]) / s.double()[..., None]
    n = torch.where((s > 0)[..., None], (d + 0.5).floor(), torch.zeros_like(d))
    n = torch.where(bad[..., None], torch.zeros_like(n), n).to(torch.uint8).flatten(-2)
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    return n, s, torch.where(bad, torch.zeros_like(m), m)


def _put(side, rows, x):
    step = max(1, (1 << 26) // (x.shape[1] * x.shape[2]))
    for i in range(0, x.shape[0], step):
        n, s, m = _quantise(x[i:i + step])
        at = slice(rows.start + i, rows.start + i + n.shape[0]) if isinstance(rows, slice) else \
            rows[i:i + step]
        side["code"][at] = n[..., 0::2] | (n[..., 1::2] << 4)
        side["s"][at] = s
        side["m"][at] = m


def _values(side, rows):
    """fp32 [n, Hkv, D] of the given pool rows."""
    c = side["code"][rows]
    n = torch.stack([c & 15, c >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    return (n * side["s"][rows].float()[..., None] + side["m"][rows].float()[..., None]).flatten(-2)


def _positions(s):
    """Pool rows of the tokens that the rows of a write or read stand for."""
    starts = s["starts"].long()
    n = s["starts_host"][-1]
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(starts, i, right=True) - 1
    pos = s["lens"].long()[b] - starts[b + 1] + i
    return s["table"][b, pos // s["P"]].long() * s["P"] + pos % s["P"]


def run(state):
    return _own_run(state) if own else _plain_run(state)


def _own_run(s):
    op = s["case"]["op"]
    if op in ("attend", "sparse"):
        out = s["att"]()
        return dict(out=out, lse=s["att"].lse)
    if op == "write":
        s["cache"].write(s["k"], s["v"], s["lens"], s["table"], s["starts"])
    s["cache"].read(s["lens"], s["table"], s["starts"], s["out_k"], s["out_v"])
    return dict(k=s["out_k"], v=s["out_v"])


def _plain_run(s):
    op = s["case"]["op"]
    if op in ("attend", "sparse"):
        return _plain_attend(s)
    rows = _positions(s)
    if op == "write":
        _put(s["cache"]["k"], rows, s["k"])
        _put(s["cache"]["v"], rows, s["v"])
    step = max(1, (1 << 27) // (s["out_k"].shape[1] * s["out_k"].shape[2]))
    for name in "kv":
        out = s["out_" + name]
        for i in range(0, out.shape[0], step):
            out[i:i + step] = _values(s["cache"][name], rows[i:i + step]).to(out.dtype)
    return dict(k=s["out_k"], v=s["out_v"])


def _seen(s, b, i):
    """Tokens (positions) that query i of request b attends to."""
    c = s["case"]
    n = s["lens_host"][b]
    if c["op"] == "sparse":
        t = s["list"][b, i].long()
        return t[t >= 0]
    return torch.arange(max(0, n - c["Nq"] + i + 1) if c["causal"] else n, device="cuda")


def _plain_attend(s):
    c = s["case"]
    Nq, Hq, Hkv, D, P = c["Nq"], c["Hq"], c["Hkv"], c["D"], s["P"]
    G = Hq // Hkv
    out = torch.zeros((s["B"], Nq, Hq, D), dtype=BF16, device="cuda")
    lse = torch.full((s["B"], Nq, Hq), -math.inf, dtype=torch.float32, device="cuda")
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        if c["op"] == "attend":  # all queries of a request over the same rows
            t = torch.arange(n, device="cuda")
            sets = [(slice(0, Nq), t)]
        else:
            sets = [(slice(i, i + 1), _seen(s, b, i)) for i in range(Nq)]
        for qs, t in sets:
            if t.numel() == 0:
                continue
            rows = s["table"][b, t // P].long() * P + t % P
            k = _values(s["cache"]["k"], rows).permute(1, 2, 0)
            v = _values(s["cache"]["v"], rows).permute(1, 0, 2)
            q = s["q"][b, qs].float()
            nq = q.shape[0]
            q = q.view(nq, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, nq * G, D)
            x = (q @ k).view(Hkv, nq, G, -1) * (1.0 / math.sqrt(D))
            if c.get("causal"):
                lim = n - Nq + torch.arange(Nq, device="cuda") + 1
                x = x.masked_fill((t[None, :] >= lim[:, None])[None, :, None, :], -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = (x - m).exp()
            l = p.sum(-1, keepdim=True)
            o = (p.view(Hkv, nq * G, -1) @ v).view(Hkv, nq, G, D)
            o = torch.where(l > 0, o / l.clamp_min(1e-30), torch.zeros_like(o))
            out[b, qs] = o.permute(1, 0, 2, 3).reshape(nq, Hq, D).to(BF16)
            lse[b, qs] = (m + l.log())[..., 0].permute(1, 0, 2).reshape(nq, Hq)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------- work, exact

def work(case):
    c = dict(case)
    L = _layout(c, 0)
    lens = L["lens"].astype(np.int64)
    row = c["Hkv"] * (c["D"] // 2 + c["D"] // GROUP * 4)  # codes, and s and m of each group
    if L["starts"] is not None:
        n = int(L["starts"][-1])
        wide = c["Hkv"] * c["D"] * (4 if c["type"] == "fp32" else 2)
        # written: the new rows in and their codes out; read back: codes in, values out
        return dict(bytes=float(2 * n * (row + wide) * (2 if c["op"] == "write" else 1)),
                    flops=float(2 * n * c["Hkv"] * c["D"] * (6 if c["op"] == "write" else 2)))
    qo = len(lens) * c["Nq"] * c["Hq"]
    if c["op"] == "sparse":
        seen = np.minimum(lens, c["k"]).repeat(c["Nq"])
        if c["holes"]:
            seen = seen * 0.9
        read, pairs = float(seen.sum()), float(seen.sum())
        index = len(lens) * c["Nq"] * c["k"] * 4
    else:
        i = np.arange(c["Nq"])[None, :]
        lim = np.clip(lens[:, None] - c["Nq"] + i + 1, 0, None) if c["causal"] else \
            np.repeat(lens[:, None], c["Nq"], 1)
        read, pairs = float(lens.sum()), float(lim.sum())
        index = int((-(-lens // c["page"])).sum()) * 4
    return dict(bytes=float(read * 2 * row + qo * (c["D"] * 4 + 4) + index),
                flops=float(4 * c["D"] * c["Hq"] * pairs))


def _step_fp16(y):
    """Distance between neighbours of fp16 at |y| (64 bits)."""
    e = torch.frexp(y.abs())[1].long().clamp_min(-13)  # |y| in [2^(e-1), 2^e)
    return ((e - 11 + 1023) << 52).view(torch.float64)


def _exact_values(x):
    """What rows x [..., D] stand for once cached, in 64 bits."""
    g = x.double().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    u = _step_fp16(lo)
    m = torch.floor(lo / u) * u
    s = (hi - m) / torch.full_like(m, 15.0)
    u = _step_fp16(s)
    s = (torch.ceil(s / u) * u)[..., None]
    m = m[..., None]
    n = torch.floor((g - m) / torch.where(s == 0, torch.ones_like(s), s) + 0.5)
    return torch.where(s == 0, m.expand_as(g), m + n * s).flatten(-2)


def exact(case, seed):
    """From the definitions in 64 bits: the inputs are made again as in ``prepare``, page
    by page, and no cache is built."""
    c = dict(case)
    L = _layout(c, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 3)
    N, P, Hkv, D = L["num_pages"], c["page"], c["Hkv"], c["D"]
    bias = _bias(c, gen)
    pool = None
    if c["op"] != "write":
        pool = [torch.empty((N * P, Hkv, D), dtype=BF16, device="cuda") for _ in range(2)]
        step = max(1, (1 << 27) // (P * Hkv * D))
        for i in range(0, N, step):
            n = min(step, N - i)
            for x, name in zip(pool, "kv"):
                x[i * P:(i + n) * P] = _rows(n * P, c, gen, name, bias).to(BF16)
    table, lens = _dev(L["table"]).long(), L["lens"].tolist()

    def rows_of(b, t):
        return table[b, t // P] * P + t % P

    if L["starts"] is not None:
        st = L["starts"].tolist()
        t = TYPES[c["type"]]
        if c["op"] == "write":
            new = [_rows(st[-1], c, gen, x, bias).to(t) for x in "kv"]
        r = {}
        for j, name in enumerate("kv"):
            out = torch.empty((st[-1], Hkv, D), dtype=torch.float64)
            for b in range(len(lens)):
                n = st[b + 1] - st[b]
                for i in range(0, n, 8192):
                    w = min(8192, n - i)
                    if c["op"] == "write":
                        x = new[j][st[b] + i:st[b] + i + w]
                    else:
                        x = pool[j][rows_of(b, torch.arange(lens[b] - n + i, lens[b] - n + i + w,
                                                            device="cuda"))]
                    out[st[b] + i:st[b] + i + w] = _exact_values(x).cpu()
            r[name] = out
        return r
    Nq, Hq = c["Nq"], c["Hq"]
    G = Hq // Hkv
    q = torch.randn((len(lens), Nq, Hq, D), generator=gen, device="cuda").to(BF16).double()
    lists = _dev(_lists(c, L)).long() if c["op"] == "sparse" else None
    out = torch.zeros((len(lens), Nq, Hq, D), dtype=torch.float64)
    lse = torch.full((len(lens), Nq, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        if lists is None:
            every = rows_of(b, torch.arange(n, device="cuda"))
        for i in range(Nq):
            if lists is None:
                if i == 0:
                    kk, vv = (_exact_values(x[every]) for x in pool)
                lim = max(0, n - Nq + i + 1) if c["causal"] else n
            else:
                t = lists[b, i]
                t = t[t >= 0]
                lim = t.numel()
                kk, vv = (_exact_values(x[rows_of(b, t)]) for x in pool)
            if lim == 0:
                continue
            x = torch.einsum("hgd,nhd->hgn", q[b, i].view(Hkv, G, D), kk[:lim]) / math.sqrt(D)
            z = torch.logsumexp(x, -1)
            o = torch.einsum("hgn,nhd->hgd", torch.exp(x - z[..., None]), vv[:lim])
            out[b, i] = o.reshape(Hq, D).cpu()
            lse[b, i] = z.reshape(Hq).cpu()
    return dict(out=out, lse=lse)
