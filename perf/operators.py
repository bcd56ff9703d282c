"""Cases for measuring the page operators of a paged KV cache and the attention
over a batch that shares prefixes, with their plain forms.

Operators (``case["op"]``):

* ``prefix``  - dense decode attention of a batch whose requests alias the pages of
  a shared prefix; the prefix's K/V take part once for all of them.
* ``fork``    - rows of a block table become aliases of other rows.
* ``extend``  - rows grow by some tokens: pages are taken, a partial page that is
  still shared is copied first (copy-on-write).
* ``free``    - rows are truncated or given back; pages nobody holds become free.
* ``compact`` - pages in use move to the lowest ids and the tables follow.

``own`` false: the plain form in torch operations.  ``own`` true: the library.
"""

import math
import zlib

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the paged-KV worked example (three of five requests share 64 tokens): a
        # handful of short requests, where latency is everything
        dict(name="prefix_example", op="prefix", lens="403,96,241,30,176", groups="0,0,0,-1,-1",
             shared="64,64,64,0,0", page=16, Hq=8, Hkv=2, D=64, Nq=1, causal=False, slack=3),
        # 64 ragged requests (1k to 32k tokens) in groups of 8 that share a system
        # prompt of 2000 tokens: most of the bytes are the requests' own
        dict(name="prefix_ragged", op="prefix", B=64, fam=8, pre_lo=2000, pre_hi=2000, own_lo=0,
             own_hi=30768, page=16, Hq=32, Hkv=8, D=128, Nq=1, causal=False, slack=100),
        # 32 requests with four drafted tokens each (causal), in groups of 8 over
        # prompts of about 8k tokens
        dict(name="prefix_draft", op="prefix", B=32, fam=8, pre_lo=7001, pre_hi=9000, own_lo=4,
             own_hi=2048, page=64, Hq=32, Hkv=8, D=128, Nq=4, causal=True, slack=40),
        # 128 samples of one 131072-token prompt, up to 1024 tokens of their own: the
        # prefix part is a large dense contraction
        dict(name="prefix_samples", op="prefix", B=128, fam=128, pre_lo=131072, pre_hi=131072,
             own_lo=1, own_hi=1024, page=64, Hq=64, Hkv=8, D=128, Nq=1, causal=False, slack=64),

        # a beam of 8 on a short prompt
        dict(name="fork_beam", op="fork", B=16, fam=8, n=8, pre_lo=403, pre_hi=403, own_lo=0,
             own_hi=40, page=16, slack=5, partial=False),
        # 64 continuations of each of 16 prompts of up to 32k tokens, some from the
        # middle of the prompt, in 16-token pages
        dict(name="fork_samples", op="fork", B=1040, fam=1, n=1024, pre_lo=8000, pre_hi=32768,
             own_lo=0, own_hi=0, page=16, slack=8192, partial=True),

        # one decoded token for 16 rows, half of them on a page they share
        dict(name="extend_token", op="extend", B=16, fam=4, fresh=0.5, pre_lo=100, pre_hi=900,
             own_lo=0, own_hi=300, add_lo=1, add_hi=1, page=16, Hkv=2, D=64, Di=64, slack=20),
        # 256 rows just forked from 32 prompts, each growing by up to 256 tokens: every
        # row copies the partial page that it shares
        dict(name="extend_forks", op="extend", B=256, fam=8, fresh=1.0, pre_lo=1024, pre_hi=8191,
             own_lo=0, own_hi=0, add_lo=1, add_hi=256, page=64, Hkv=8, D=128, Di=128, slack=2048),

        # rejected drafts: 32 rows drop up to 8 tokens
        dict(name="free_drafts", op="free", B=32, fam=4, n=32, pre_lo=500, pre_hi=4000, own_lo=16,
             own_hi=500, cut=8, page=16, slack=10),
        # 768 finished samples of 16 prompts of up to 32k tokens give their pages back
        dict(name="free_samples", op="free", B=1024, fam=64, n=768, pre_lo=8000, pre_hi=32768,
             own_lo=1, own_hi=512, cut=0, page=16, slack=4096),

        # a small cache, a quarter of it holes
        dict(name="compact_small", op="compact", B=24, fam=4, pre_lo=100, pre_hi=900, own_lo=0,
             own_hi=300, page=16, Hkv=2, D=64, Di=64, holes=0.25),
        # 64 requests of up to 8k tokens left after as much again was freed
        dict(name="compact_large", op="compact", B=64, fam=4, pre_lo=1000, pre_hi=4096, own_lo=1,
             own_hi=4096, page=64, Hkv=8, D=128, Di=128, holes=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "fork", "extend", "free", "compact"])
    page = rng.choice([1, 5, 16, 16, 17, 32, 48, 64, 64, 128])
    if op == "prefix":
        Hkv = rng.choice([1, 2, 3, 4, 8, 8])
        G = rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 12, 16])
        Nq = rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 17])
        B = min(_log(rng, 1, 256), 4096 // Nq)
        fam = _log(rng, 1, B)
        pre = _log(rng, 1, 65536)
        own_hi = _log(rng, 1, 16384)
        # no more cached tokens and no more products than the largest listed case
        while (B // fam + 1) * pre + B * own_hi > 400_000:
            pre, own_hi = max(1, pre // 2), max(1, own_hi // 2)
        while B * Nq * G * Hkv * (pre + own_hi) > 128 * 64 * 100_000 and B > 1:
            B = max(1, B // 2)
            fam = min(fam, B)
        return dict(op=op, B=B, fam=fam, pre_lo=max(1, pre * 2 // 3), pre_hi=pre,
                    own_lo=rng.choice([0, 0, 1, Nq]), own_hi=max(Nq, own_hi), page=page,
                    Hq=G * Hkv, Hkv=Hkv, D=rng.choice([64, 128]), Nq=Nq,
                    causal=rng.random() < 0.5, slack=_log(rng, 1, 64), empty=rng.random() < 0.3,
                    fresh=rng.choice([0.0, 0.0, 0.5]))
    B = _log(rng, 2, 512)
    fam = _log(rng, 1, B)
    pre = _log(rng, 1, 16384)
    own_hi = _log(rng, 1, 2048)
    if op in ("extend", "compact"):
        while (B // fam + 1) * pre + B * own_hi > 200_000:
            pre, own_hi = max(1, pre // 2), max(1, own_hi // 2)
    c = dict(op=op, B=B, fam=fam, pre_lo=max(1, pre // 2), pre_hi=pre, own_lo=0, own_hi=own_hi,
             page=page, slack=_log(rng, 1, 300))
    if op == "fork":
        c.update(n=rng.randint(1, max(1, B // 2)), partial=rng.random() < 0.5)
    elif op == "free":
        c.update(n=rng.randint(1, B), cut=rng.choice([0, 1, 8, 100]))
    else:
        c.update(Hkv=rng.choice([1, 2, 3, 8]), D=rng.choice([64, 128]), Di=rng.choice([64, 128]))
        if op == "extend":
            a = _log(rng, 1, 300)
            c.update(fresh=rng.choice([0.0, 0.5, 1.0]), add_lo=rng.choice([0, 1]), add_hi=a)
        else:
            c.update(holes=rng.choice([0.0, 0.1, 0.4, 0.6]))
            del c["slack"]
    return c


# ------------------------------------------------------------- block tables

def _ints(text):
    return [int(x) for x in text.split(",")]


def _layout(c, seed):
    """Lengths, aliased table and the pool's size of a case (host).

    Families of ``fam`` rows share a prompt of pre_lo..pre_hi tokens.  A row either
    still stands on the prompt's own pages, the last partial one among them
    ("fresh", probability c["fresh"]), or has its own pages from the prompt's last
    whole page on and own_lo..own_hi tokens more.  The lengths are the case's
    own; the order of the rows and of the pages is the seed's.
    """
    sizes = sorted((k, v) for k, v in c.items() if k != "name")
    rs = np.random.RandomState(zlib.crc32(repr(sizes).encode()))
    P = c["page"]
    if "lens" in c:
        lens = np.array(_ints(c["lens"]), np.int64)
        group = np.array(_ints(c["groups"]), np.int64)
        shared = np.array(_ints(c["shared"]), np.int64)
        fresh = np.zeros(len(lens), bool)
        prompt = shared
    else:
        B = c["B"]
        group = np.arange(B) // c["fam"]
        prompt = rs.randint(c["pre_lo"], c["pre_hi"] + 1, size=B)[group * c["fam"]]
        fresh = rs.random_sample(B) < c.get("fresh", 0.0)
        lens = prompt + np.where(fresh, 0, rs.randint(c["own_lo"], c["own_hi"] + 1, size=B))
        if c.get("empty"):  # a padded batch: some rows hold nothing
            lens[rs.random_sample(B) < 0.1] = 0
        if c["op"] == "fork":  # the highest rows are spare
            lens[B - min(c["n"], B - 1):] = 0
    B = len(lens)
    order = np.arange(B)
    max_pages = int(max(1, (-(-(lens + c.get("add_hi", 0)) // P)).max())) + rs.randint(0, 3)
    rs = np.random.RandomState(seed % (2 ** 31) + 11)
    if "lens" not in c:
        live = B - min(c["n"], B - 1) if c["op"] == "fork" else B
        order[:live] = rs.permutation(live)
    lens, group, prompt, fresh = lens[order], group[order], prompt[order], fresh[order]
    pages = -(-lens // P)
    whole = np.where(lens == 0, 0, np.where(fresh, -(-prompt // P), np.minimum(prompt // P, pages)))
    whole = np.where(group < 0, 0, whole)
    table = np.full((B, max_pages), -1, np.int32)
    held = {}
    total = 0
    for b in range(B):  # ids 0, 1, ... in order of first use
        w, n = int(whole[b]), int(pages[b])
        if w:
            have = held.get(int(group[b]))
            if have is None:
                have = held[int(group[b])] = np.zeros(0, np.int32)
            if len(have) < w:
                have = np.concatenate([have, np.arange(total, total + w - len(have), dtype=np.int32)])
                total += w - len(held[int(group[b])])
                held[int(group[b])] = have
            table[b, :w] = have[:w]
        table[b, w:n] = np.arange(total, total + n - w, dtype=np.int32)
        total += n - w
    if "holes" in c:
        num_pages = int(total / (1.0 - c["holes"])) + 1
    else:
        num_pages = total + c["slack"]
        if "add_hi" in c:  # room for the growth: whole pages and a copy a row
            num_pages += B * (-(-c["add_hi"] // P) + 2)
    deal = rs.permutation(num_pages).astype(np.int32)
    table = np.where(table >= 0, deal[np.maximum(table, 0)], -1).astype(np.int32)
    return dict(lens=lens.astype(np.int32), group=group.astype(np.int32), table=table,
                num_pages=num_pages, used=total, rs=rs)


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(BF16)


def _pool(num_pages, c, gen):
    out = torch.empty((num_pages, c["page"], c["Hkv"], c["D"]), dtype=BF16, device="cuda")
    step = max(1, (1 << 26) // (c["page"] * c["Hkv"] * c["D"]))
    for i in range(0, num_pages, step):
        out[i:i + step] = _randn(out[i:i + step].shape, gen)
    return out


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    c = dict(case)
    L = _layout(c, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 5)
    B = len(L["lens"])
    s = dict(case=c, B=B, P=c["page"], num_pages=L["num_pages"])
    if c["op"] == "prefix":
        s["lens_host"] = L["lens"].tolist()
        s["lens"] = torch.from_numpy(L["lens"]).cuda()
        s["table"] = torch.from_numpy(L["table"]).cuda()
        s["group"] = torch.from_numpy(L["group"]).cuda()
        s["k"] = _pool(L["num_pages"], c, gen)
        s["v"] = _pool(L["num_pages"], c, gen)
        s["q"] = _randn((B, c["Nq"], c["Hq"], c["D"]), gen)
        if own:
            from top_sparse_attention_pks_gb300.decoder import PrefixAttention
            # the workspace and output buffers that a decode loop keeps
            s["att"] = PrefixAttention(s["lens"], s["table"], s["q"], s["k"], s["v"],
                                       prefix_group=s["group"], causal=c["causal"], lse=True)
        return s

    rs = L["rs"]
    lens, table = L["lens"], L["table"]
    if c["op"] == "fork":
        n = min(c["n"], B - 1)
        live = B - n
        src = np.sort(rs.randint(0, live, size=n)).astype(np.int32)
        dst = (B - n + rs.permutation(n)).astype(np.int32)
        keep = lens[src].copy()
        if c["partial"]:
            cut = rs.random_sample(n) < 0.5
            keep = np.where(cut, (keep * rs.random_sample(n)).astype(np.int32), keep)
        s.update(src=_dev(src), dst=_dev(dst), keep=_dev(keep))
    elif c["op"] == "free":
        rows = rs.permutation(B)[: c["n"]].astype(np.int32)
        if c["cut"]:
            keep = np.maximum(lens[rows] - rs.randint(0, c["cut"] + 1, size=len(rows)), 0)
        else:
            keep = np.zeros(len(rows))
        s.update(rows=_dev(rows), keep=_dev(keep))
    elif c["op"] == "extend":
        add = rs.randint(c["add_lo"], c["add_hi"] + 1, size=B).astype(np.int64)
        s["add"] = _dev(add)
    N = s["num_pages"]
    ref = np.bincount(table[table >= 0].reshape(-1), minlength=N).astype(np.int32)
    # lengths, table and reference counts (or the library's state) sit in one buffer
    # each side puts back before a pass: the operators work in place
    nl, nt = _pad(B), _pad(table.size)
    if own:
        from top_sparse_attention_pks_gb300 import pks
        tail = -(-pks.pks_pages_state_bytes(N) // 4)
    else:
        tail = N
    buf = torch.zeros(nl + nt + tail, dtype=torch.int32, device="cuda")
    s["lens"] = buf[:B]
    s["table"] = buf[nl:nl + table.size].view(B, table.shape[1])
    s["lens"].copy_(_dev(lens))
    s["table"].copy_(_dev(table))
    s["pools"] = []
    if c["op"] in ("extend", "compact"):
        s["pools"] = [_pool(N, c, gen), _pool(N, c, gen),
                      torch.randint(-127, 128, (N, c["page"], c["Di"]), generator=gen,
                                    device="cuda", dtype=torch.int8)]
    if own:
        from top_sparse_attention_pks_gb300.decoder import PageTable
        s["pages"] = PageTable(s["lens"], s["table"], N, c["page"], pools=s["pools"],
                               state=buf[nl + nt:].view(torch.uint8))
    else:
        s["ref"] = buf[nl + nt:]
        s["ref"].copy_(_dev(ref))
    s["buf"], s["saved"] = buf, buf.clone()
    return s


def _pad(n):
    return -(-n // 64) * 64  # 256 bytes


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


# --------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if op == "prefix":
        return _own_prefix(state) if own else _plain_prefix(state)
    state["buf"].copy_(state["saved"])
    if own:
        return _own_pages(state, op)
    return {"fork": _plain_fork, "extend": _plain_extend, "free": _plain_free,
            "compact": _plain_compact}[op](state)


def _own_prefix(s):
    att = s["att"]
    out = att()
    return dict(out=out, lse=att.lse)


def _own_pages(s, op):
    pg = s["pages"]
    if op == "fork":
        pg.fork(s["src"], s["dst"], s["keep"])
    elif op == "extend":
        pg.extend(s["add"])
    elif op == "free":
        pg.free(s["rows"], s["keep"])
    else:
        pg.compact()
    r = dict(lens=s["lens"], table=s["table"], ref=pg.refs, n_free=pg.n_free, pools=s["pools"])
    if op == "compact":
        r["page_map"] = pg.page_map
    return r


def _limits(c, n, device):
    """Tokens each of a request's queries attends to: all n, or up to its own."""
    Nq = c["Nq"]
    i = torch.arange(Nq, device=device)
    return (n - Nq + i + 1).clamp(0, n) if c["causal"] else torch.full_like(i, n)


def _plain_prefix(s):
    c = s["case"]
    Nq, Hq, Hkv, D = c["Nq"], c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    out = torch.zeros((s["B"], Nq, Hq, D), dtype=BF16, device="cuda")
    lse = torch.full((s["B"], Nq, Hq), -math.inf, dtype=torch.float32, device="cuda")
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        pg = s["table"][b, : -(-n // s["P"])].long()
        k = s["k"][pg].reshape(-1, Hkv, D)[:n].float().permute(1, 2, 0)
        v = s["v"][pg].reshape(-1, Hkv, D)[:n].float().permute(1, 0, 2)
        q = s["q"][b].float().view(Nq, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, Nq * G, D)
        x = (q @ k).view(Hkv, Nq, G, n) * (1.0 / math.sqrt(D))
        lim = _limits(c, n, "cuda")
        if c["causal"]:
            t = torch.arange(n, device="cuda")
            x = x.masked_fill((t[None, :] >= lim[:, None])[None, :, None, :], -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
        p = (x - m).exp()
        l = p.sum(-1, keepdim=True)
        o = (p.view(Hkv, Nq * G, n) @ v).view(Hkv, Nq, G, D)
        o = torch.where(l > 0, o / l.clamp_min(1e-30), torch.zeros_like(o))
        out[b] = o.permute(1, 0, 2, 3).reshape(Nq, Hq, D).to(BF16)
        lse[b] = (m + l.log())[..., 0].permute(1, 0, 2).reshape(Nq, Hq)
    return dict(out=out, lse=lse)


def _plain_result(s, **more):
    r = dict(lens=s["lens"], table=s["table"], ref=s["ref"],
             n_free=(s["ref"] == 0).sum().to(torch.int32), pools=s["pools"])
    r.update(more)
    return r


def _pages_of(n, P):
    return (n + (P - 1)) // P


def _columns(s):
    return torch.arange(s["table"].shape[1], device="cuda")[None, :]


def _plain_fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    took = _columns(s) < _pages_of(s["keep"], s["P"])[:, None]
    from_src = s["table"][src]
    s["table"][dst] = torch.where(took, from_src, s["table"][dst])
    s["lens"][dst] = s["keep"]
    ids = from_src[took].long()
    s["ref"].index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    return _plain_result(s)


def _plain_free(s):
    rows = s["rows"].long()
    col = _columns(s)
    old = s["table"][rows]
    gone = (col >= _pages_of(s["keep"], s["P"])[:, None]) & \
        (col < _pages_of(s["lens"][rows], s["P"])[:, None])
    ids = old[gone].long()
    s["ref"].index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    s["table"][rows] = torch.where(gone, torch.full_like(old, -1), old)
    s["lens"][rows] = s["keep"]
    return _plain_result(s)


def _plain_extend(s):
    P, ref, table = s["P"], s["ref"], s["table"]
    B = s["B"]
    lens, add = s["lens"].long(), s["add"].long()
    row = torch.arange(B, device="cuda")
    had, want = _pages_of(lens, P), _pages_of(lens + add, P)
    # a growing row whose last page is partly filled and held by others too takes a
    # copy of it, unless all its holders grow: then the last of them keeps it
    grows = (add > 0) & (lens % P > 0)
    tail = torch.where(grows, table[row, (lens // P).clamp_max(table.shape[1] - 1)].long(), 0)
    holders = torch.zeros_like(ref).index_add_(0, tail, grows.int())
    last = torch.full_like(ref, -1, dtype=torch.int64).scatter_reduce_(
        0, tail, torch.where(grows, row, -1), "amax")
    copies = grows & (ref[tail] > 1) & ~((holders[tail] == ref[tail]) & (last[tail] == row))
    need = torch.where(add > 0, want - had, 0) + copies
    start = need.cumsum(0) - need
    free = (ref == 0).nonzero()[:, 0]
    cr = copies.nonzero()[:, 0]
    src, to = tail[cr], free[start[cr]]
    for pool in s["pools"]:
        t = torch.arange(P, device="cuda")[None, :] < (lens[cr] % P)[:, None]
        t = t.reshape(t.shape + (1,) * (pool.dim() - 2))
        pool[to] = torch.where(t, pool[src], pool[to])
    ref.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    col = _columns(s)
    new = (col >= had[:, None]) & (col < want[:, None])
    at = (start + copies)[:, None] + col - had[:, None]
    table.copy_(torch.where(new, free[at.clamp(0, free.numel() - 1)].int(), table))
    table[cr, (lens // P)[cr]] = to.int()
    ref[free[: int(need.sum())]] = 1
    s["lens"].add_(s["add"])
    return _plain_result(s)


def _plain_compact(s):
    ref, N = s["ref"], s["num_pages"]
    used = ref > 0
    n_used = int(used.sum())
    src = used[n_used:].nonzero()[:, 0] + n_used
    dst = (~used[:n_used]).nonzero()[:, 0]
    page_map = torch.where(used, torch.arange(N, device="cuda"), -1).int()
    page_map[src] = dst.int()
    for pool in s["pools"]:
        pool[dst] = pool[src]
    held = (_columns(s) < _pages_of(s["lens"], s["P"])[:, None])
    new = page_map[s["table"].long().clamp_min(0)]
    s["table"].copy_(torch.where(held, new, s["table"]))
    ref[dst] = ref[src]
    ref[src] = 0
    return _plain_result(s, page_map=page_map)


# ------------------------------------------------------------- work, exact

def work(case):
    c = dict(case)
    L = _layout(c, 0)
    lens, table, P = L["lens"].astype(np.int64), L["table"], c["page"]
    B = len(lens)
    if c["op"] == "prefix":
        row = c["Hkv"] * c["D"] * 2
        # tokens held by each distinct page: the longest stay of any request on it
        held = np.zeros(L["num_pages"], np.int64)
        for b in range(B):
            n = int(-(-lens[b] // P))
            tok = np.full(n, P)
            if n:
                tok[-1] = lens[b] - (n - 1) * P
            np.maximum.at(held, table[b, :n], tok)
        i = np.arange(c["Nq"])[None, :]
        lim = np.clip(lens[:, None] - c["Nq"] + i + 1, 0, lens[:, None]) if c["causal"] else \
            np.repeat(lens[:, None], c["Nq"], 1)
        qo = B * c["Nq"] * c["Hq"]
        return dict(bytes=float(held.sum() * 2 * row + qo * (c["D"] * 4 + 4) + (-(-lens // P)).sum() * 4),
                    flops=float(4 * c["D"] * c["Hq"] * lim.sum()))
    entries = int((table >= 0).sum())
    if c["op"] == "fork":
        n = min(c["n"], B - 1)
        part = 0.75 if c["partial"] else 1.0
        return dict(bytes=float(n * (part * entries / (B - n) * 4 + 16) + entries * 12), flops=0.0)
    if c["op"] == "free":
        per = entries / B if not c["cut"] else 1 + c["cut"] / P / 2
        return dict(bytes=float(c["n"] * (per * 16 + 12)), flops=0.0)
    token = 2 * c["Hkv"] * c["D"] * 2 + c["Di"]
    if c["op"] == "extend":
        add = (c["add_lo"] + c["add_hi"]) / 2
        share = c["fresh"] * min(1.0, P - 1) * (c["fam"] - 1) / c["fam"]
        return dict(bytes=float(B * (share * P / 2 * token * 2 + (1 + add / P) * 12 + 12)), flops=0.0)
    used = L["used"]
    moved = used * (1.0 - used / L["num_pages"])
    return dict(bytes=float(moved * P * token * 2 + entries * 8 + L["num_pages"] * 8), flops=0.0)


def exact(case, seed):
    """The attention in 64 bits, a request at a time.  The page operators give whole
    numbers and copies: nothing to be exact about."""
    c = dict(case)
    if c["op"] != "prefix":
        return None
    s = prepare(case, seed)
    Hkv, D, P, Nq = c["Hkv"], c["D"], c["page"], c["Nq"]
    G = c["Hq"] // Hkv
    out = torch.zeros((s["B"], Nq, c["Hq"], D), dtype=torch.float64)
    lse = torch.full((s["B"], Nq, c["Hq"]), -math.inf, dtype=torch.float64)
    kf, vf = s["k"].view(-1, Hkv, D), s["v"].view(-1, Hkv, D)
    for b, n in enumerate(s["lens_host"]):
        t = torch.arange(n, device="cuda")
        rows = s["table"][b].long()[t // P] * P + t % P
        for h in range(Hkv):
            kk, vv = kf[rows, h].double(), vf[rows, h].double()
            for i in range(Nq):
                lim = max(0, n - Nq + i + 1) if c["causal"] else n
                if lim == 0:
                    continue
                x = s["q"][b, i, h * G:(h + 1) * G].double() @ kk[:lim].T / math.sqrt(D)
                z = torch.logsumexp(x, 1)
                w = torch.exp(x - z[:, None])
                out[b, i, h * G:(h + 1) * G] = (w @ vv[:lim]).cpu()
                lse[b, i, h * G:(h + 1) * G] = z.cpu()
    return dict(out=out, lse=lse)
