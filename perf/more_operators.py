"""Workloads of the operators of a serving step over long contexts: page tables
and slots from the requests' lengths, norms of q and k heads with the rotation
(and the cache) in one pass, attention with a sliding window and first tokens
that stay visible, attention of a batch that shares a prefix.

`own` false: `run` computes an operator in plain torch, in 32 bits (angles in
64), rounded once at the end.  `own` true: `run` makes the library's calls.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn, "fp32": torch.float32}
QMAX = {"int8": 127.0, "e4m3": 448.0}
TINY = torch.finfo(torch.float32).tiny
EPS = 1e-6


def listed():
    return [
        # one decode step of 25 serving slots: a token each, now and then a page
        dict(name="plan_decode", kind="plan", batch=25, new_max=1, kv_max=32768, page=64, trims=False, pad=7, lens=1),
        # a large server's mixed step: single tokens, chunks of prompts, rejected drafts and finished requests
        dict(name="plan_mixed", kind="plan", batch=1500, new_max=512, kv_max=8192, page=16, trims=True, pad=61, lens=2),
        # a decode step's fp32 products of 25 slots, 32 q heads on 8, into e4m3 pages
        dict(name="qkv_decode", kind="qkv", tokens=25, heads=32, kv_heads=8, dim=128, rot=128, layout="half", inp="fp32", type="e4m3", page=16, pages=512, far=32768, lens=3),
        # a long prompt's fp32 products into bf16 pages
        dict(name="qkv_prompt", kind="qkv", tokens=16381, heads=32, kv_heads=8, dim=128, rot=128, layout="half", inp="fp32", type="bf16", page=64, pages=320, far=65536, lens=4),
        # packed prompts of a 27B-shaped model (40 heads of 128 on 40) to rows for the prompts' attention, half of each head rotated
        dict(name="qk_rows", kind="qk", tokens=8191, heads=40, kv_heads=40, dim=128, rot=64, layout="interleaved", inp="bf16", far=65536, lens=5),
        # one user's decode step late in a long chat, window of 1024: latency counts
        dict(name="window_one", kind="window", batch=1, q_max=1, kv_max=32768, window=1024, sinks=4, heads=32, kv_heads=8, dim=128, type="bf16", page=64, ragged=False, lens=6),
        # 25 serving slots, ragged contexts up to 32768, window of 4096, 8-bit pages
        dict(name="window_slots", kind="window", batch=25, q_max=1, kv_max=32768, window=4096, sinks=16, heads=32, kv_heads=8, dim=128, type="int8", page=64, ragged=True, lens=7),
        # chunks of long prompts over what the cache holds
        dict(name="window_chunk", kind="window", batch=4, q_max=1024, kv_max=16384, window=2048, sinks=4, heads=32, kv_heads=8, dim=128, type="bf16", page=128, ragged=True, lens=8),
        # one long prompt of an 8B-shaped model, window of 4096: the largest product
        dict(name="window_prompt", kind="window_prompt", batch=1, q_max=16384, window=4096, sinks=64, heads=32, kv_heads=8, dim=128, ragged=False, lens=9),
        # four users behind one short instruction, bf16 pages: latency counts
        dict(name="shared_few", kind="shared", groups="4", q_max=1, prefix_max=2048, own_max=256, heads=32, kv_heads=8, dim=128, type="bf16", page=64, lens=10),
        # 64 slots behind one long system prompt
        dict(name="shared_slots", kind="shared", groups="64", q_max=1, prefix_max=16384, own_max=2048, heads=32, kv_heads=8, dim=128, type="int8", page=64, lens=11),
        # drafts of three groups of samples, heads of 64, 8-bit floating-point pages
        dict(name="shared_drafts", kind="shared", groups="16 5 9", q_max=8, prefix_max=6000, own_max=1000, heads=16, kv_heads=16, dim=64, type="e4m3", page=16, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["plan", "qkv", "qk", "window", "window", "window_prompt", "shared", "shared"])
    c = dict(kind=kind, lens=rng.randrange(1 << 20))
    if kind == "plan":
        c.update(batch=_log_int(rng, 1, 2048), new_max=_log_int(rng, 1, 512), kv_max=_log_int(rng, 64, 32768),
                 page=rng.choice([16, 32, 64, 128, 256]), trims=rng.random() < 0.6, pad=rng.randrange(100))
        return c
    c["dim"] = rng.choice([64, 128])
    kv_heads, group = rng.choice([(1, 8), (2, 7), (4, 8), (8, 4), (8, 3), (5, 4), (16, 1), (16, 2), (40, 1)])
    heads = kv_heads * group
    c.update(heads=heads, kv_heads=kv_heads)
    if kind in ("qkv", "qk"):
        t = _log_int(rng, 1, 8192)
        c.update(tokens=t, rot=rng.choice([c["dim"], c["dim"], c["dim"] // 2]), layout=rng.choice(["half", "interleaved"]),
                 inp=rng.choice(["fp32", "bf16"]), far=_log_int(rng, 64, 131072))
        if kind == "qkv":
            page = rng.choice([16, 32, 64, 128])
            c.update(type=rng.choice(["bf16", "e4m3"]), page=page, pages=-(-t // page) + rng.randrange(8, 40))
        return c
    if kind != "window_prompt":
        c.update(type=rng.choice(["bf16", "int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]))
    if kind == "shared":
        pre, mine = _log_int(rng, 16, 16384), _log_int(rng, 1, 2048)
        q = 1 if rng.random() < 0.5 else min(mine, _log_int(rng, 2, 32))
        most = max(1, min(32, (1 << 29) // (q * (pre + mine) * heads), 64_000_000 // (mine * kv_heads * c["dim"])))
        c.update(groups=" ".join(str(_log_int(rng, 1, most)) for _ in range(rng.randint(1, 3))), q_max=q, prefix_max=pre, own_max=mine)
        return c
    window, sinks = _log_int(rng, 1, 4096), rng.choice([0, 1, 4, 17, 64, 128])
    c.update(window=window, sinks=sinks, ragged=rng.random() < 0.7)
    if kind == "window":
        kv = _log_int(rng, 16, 32768)
        q = 1 if rng.random() < 0.4 else min(kv, _log_int(rng, 2, 1024))
        seen = min(kv, window + sinks + q)
        most = max(1, min(32, 190_000_000 // (kv * kv_heads * c["dim"]), (1 << 29) // (q * seen * heads)))
        c.update(batch=_log_int(rng, 1, most), q_max=q, kv_max=kv)
    else:
        q = _log_int(rng, 1, 8192)
        most = max(1, min(32, 16384 // q, (1 << 30) // (q * min(q, window + sinks) * heads)))
        c.update(batch=_log_int(rng, 1, most), q_max=q)
    return c


# --------------------------------------------------------------------------
# what a case fixes: lengths and frequencies
# --------------------------------------------------------------------------

def _requests(case):
    """(tokens held, new tokens) of a planning step's sequences, from the case alone."""
    rng = random.Random(case["lens"])
    held, new = [], []
    for _ in range(case["batch"]):
        n = rng.randint(0, case["kv_max"])
        kind = rng.random()
        if case["new_max"] == 1 or kind < 0.6:
            m = 1
        elif kind < 0.8:
            m = rng.randint(1, case["new_max"])
        else:
            m = rng.choice([0, 1])
        if case["trims"] and n > 0 and rng.random() < 0.15:
            m = -n if rng.random() < 0.3 else -rng.randint(1, min(n, 8))
        held.append(n)
        new.append(m)
    return held, new


def _lengths(case):
    """(new tokens, tokens held) of each sequence, from the case alone."""
    rng = random.Random(case["lens"])
    if case["kind"] == "shared":
        q, own_len = [], []
        for _ in range(sum(_groups(case))):
            n = max(1, min(case["own_max"], int(case["own_max"] * rng.uniform(0.05, 1.1))))
            own_len.append(n)
            q.append(1 if case["q_max"] == 1 else rng.randint(1, min(case["q_max"], n)))
        return q, own_len
    most = case["kv_max"] if case["kind"] == "window" else case["q_max"]
    n = [most] * case["batch"]
    if case["ragged"]:
        n = [max(1, min(most, int(most * rng.uniform(0.05, 1.1)))) for _ in n]
        n[rng.randrange(len(n))] = most
    if case["kind"] != "window":
        return n, n
    q = [min(case["q_max"], v) for v in n]
    if case["ragged"] and case["q_max"] > 1:
        q = [rng.randint(1, v) for v in q]
    return q, n


def _groups(case):
    """Sequences of each group."""
    return [int(v) for v in case["groups"].split()]


def _prefixes(case):
    """Shared tokens of each group."""
    rng = random.Random(case["lens"] + 1)
    n = [max(1, int(case["prefix_max"] * rng.uniform(0.3, 1.0))) for _ in _groups(case)]
    n[rng.randrange(len(n))] = case["prefix_max"]
    page = case["page"]
    return [max(page, v // page * page) for v in n]  # whole pages: what is shared


def _frequencies(rot):
    """Radians a position for each pair."""
    return 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _start(n, device):
    return torch.tensor([0] + n, device=device).cumsum(0).to(torch.int32)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind = case["kind"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    def ints(n, dtype=torch.int32):
        return torch.tensor(n, dtype=dtype, device=dev)

    s = {"case": dict(case)}
    if kind == "plan":
        page = case["page"]
        held, new = _requests(case)
        pages = [-(-v // page) for v in held]
        after = [-(-(v + m) // page) for v, m in zip(held, new)]
        taken = sum(max(0, b - a) for a, b in zip(pages, after))
        n_pages = sum(pages) + taken + 5
        deal = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        width = max(max(pages), max(after), 1)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32)
        host = deal.cpu()
        at = 0
        for b, v in enumerate(pages):
            table[b, :v] = host[at:at + v]
            at += v
        t = sum(max(0, m) for m in new) + case["pad"]
        free = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        free[:n_pages - at] = deal[at:]
        s.update(kv_len=ints(held), n_new=ints(new), table=table.to(dev), free=free, n_free=ints([n_pages - at]), taken=taken,
                 given=sum(max(0, a - b) for a, b in zip(pages, after)), n_pages=n_pages,
                 q_start=torch.empty(case["batch"] + 1, dtype=torch.int32, device=dev), positions=torch.empty(max(t, 1), dtype=torch.int32, device=dev),
                 slots=torch.empty(max(t, 1), dtype=torch.int32, device=dev), len_out=ints(held), n_free_out=ints([0]))
        return s

    dim, heads, kv_heads = case["dim"], case["heads"], case["kv_heads"]
    if kind in ("qkv", "qk"):
        t = case["tokens"]
        first = int(torch.randint(0, case["far"], (1,), generator=g, device=dev))
        s["pos"] = (torch.randint(0, case["far"], (t,), generator=g, device=dev) if t < 64
                    else first + torch.arange(t, device=dev)).to(torch.int32)
        # the three products of a layer side by side
        x = normal(t, (heads + 2 * kv_heads) * dim, dtype=TYPES[case["inp"]])
        s["q"], s["k"], s["v"] = x[:, :heads * dim], x[:, heads * dim:(heads + kv_heads) * dim], x[:, (heads + kv_heads) * dim:]
        s["wq"], s["wk"] = (1 + 0.2 * normal(dim, dtype=torch.float32)).bfloat16(), (1 + 0.2 * normal(dim, dtype=torch.float32)).bfloat16()
        s["freq"] = _frequencies(case["rot"]).to(dev)
        s["q_out"] = torch.empty(t, heads * dim, dtype=torch.bfloat16, device=dev)
        if kind == "qk":
            s["k_out"] = torch.empty(t, kv_heads * dim, dtype=torch.bfloat16, device=dev)
            return s
        s["slots"] = torch.randperm(case["pages"] * case["page"], generator=g, device=dev)[:t].to(torch.int32)
        pages = case["pages"]
    if kind == "window_prompt":
        n, _ = _lengths(case)
        t = sum(n)
        s.update(n=n, start=_start(n, dev), q=normal(t, heads * dim), k=normal(t, kv_heads * dim), v=normal(t, kv_heads * dim),
                 out=torch.empty(t, heads * dim, dtype=torch.bfloat16, device=dev))
        return s

    # a cache: pages dealt out in no order, slots that nobody wrote hold an earlier user's values
    page, typ = case["page"], case["type"]
    if kind != "qkv":
        q, n = _lengths(case)
        shared = [0] * len(n)
        if kind == "shared":
            pre = _prefixes(case)
            shared = [v // page for v, m in zip(pre, _groups(case)) for _ in range(m)]
            n = [v * page + m for v, m in zip(shared, n)]
            s.update(pre=pre, prefix_len=ints(pre), group_start=_start(_groups(case), dev))
        need = [-(-v // page) for v in n]
        pages = sum(a - b for a, b in zip(need, shared)) + 3
        if kind == "shared":
            pages += sum(v // page for v in pre)
        table = torch.zeros(len(n), max(need), dtype=torch.int32)
        deal = torch.randperm(pages, generator=g, device=dev).cpu().to(torch.int32)
        at = b = 0
        for group, many in enumerate(_groups(case) if kind == "shared" else [1] * len(n)):
            common = shared[b]
            table[b:b + many, :common] = deal[at:at + common]
            at += common
            for b in range(b, b + many):
                v = need[b] - common
                table[b, common:need[b]] = deal[at:at + v]
                at += v
            b += 1
        t = sum(q)
        s.update(q_n=q, n=n, start=_start(q, dev), kv_len=ints(n), table=table.to(dev), q=normal(t, heads * dim),
                 out=torch.empty(t, heads * dim, dtype=torch.bfloat16, device=dev))
    shape = (pages, kv_heads, page, dim)
    for name in ("ck", "cv"):
        if typ == "bf16":
            s[name], s[name + "s"] = normal(*shape), None
            continue
        x = torch.randn(shape, generator=g, device=dev)
        sc = (x.abs().amax(-1) / QMAX[typ]).clamp_min(TINY)
        x /= sc[..., None]
        s[name] = x.round_().to(torch.int8) if typ == "int8" else x.to(TYPES[typ])
        s[name + "s"] = sc
        del x
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _plan(s):
    page = s["case"]["page"]
    dev = s["table"].device
    held, new = s["kv_len"].long(), s["n_new"].long()
    after = held + new
    had, has = (held + page - 1) // page, (after + page - 1) // page
    more, less = (has - had).clamp_min(0), (had - has).clamp_min(0)
    n_free = s["n_free"].long()
    # pages that trimmed sequences give back go on top of the list, in order
    if s["given"]:
        r = torch.arange(s["given"], device=dev)
        end = less.cumsum(0)
        b = torch.searchsorted(end, r, right=True)
        s["free"][n_free + r] = s["table"][b, has[b] + r - (end[b] - less[b])]
    # pages are taken from the top, in order
    if s["taken"]:
        r = torch.arange(s["taken"], device=dev)
        end = more.cumsum(0)
        b = torch.searchsorted(end, r, right=True)
        s["table"][b, had[b] + r - (end[b] - more[b])] = s["free"][n_free + s["given"] - 1 - r]
    grown = new.clamp_min(0)
    s["q_start"][0] = 0
    s["q_start"][1:] = grown.cumsum(0)
    row = torch.arange(s["slots"].numel(), device=dev)
    b = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    there = b < grown.numel()
    b = b.clamp_max(grown.numel() - 1)
    pos = torch.where(there, held[b] + row - s["q_start"][b], 0)
    s["positions"].copy_(pos)
    at = (pos // page).clamp_max(s["table"].shape[1] - 1)
    s["slots"].copy_(torch.where(there, s["table"][b, at].long() * page + pos % page, -1))
    s["len_out"].copy_(after)
    s["n_free_out"].copy_(n_free + s["given"] - s["taken"])


def _plan_out(s):
    return [s[name] for name in ("q_start", "positions", "slots", "len_out", "n_free_out", "table", "free")]


def _norm_rotate(x, w, pos, freq, layout):
    """x [T, heads, dim] in 32 bits: each head over its root mean square, times w, rotated."""
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a = pos.double()[:, None, None] * freq
    c, s = a.cos().float(), a.sin().float()
    rot = 2 * freq.numel()
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if layout == "interleaved" else (y[..., :rot // 2], y[..., rot // 2:])
    p, q = a * c - b * s, b * c + a * s
    y = torch.stack((p, q), -1).flatten(-2) if layout == "interleaved" else torch.cat((p, q), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _quantise(x, typ):
    if typ == "bf16":
        return x.to(torch.bfloat16), None
    scale = (x.abs().amax(-1) / QMAX[typ]).clamp_min(TINY)
    return (x / scale[..., None]).to(TYPES[typ]), scale


def _qkv(s):
    c = s["case"]
    split = lambda x: x.float().unflatten(1, (-1, c["dim"]))
    q = _norm_rotate(split(s["q"]), s["wq"], s["pos"], s["freq"], c["layout"])
    k = _norm_rotate(split(s["k"]), s["wk"], s["pos"], s["freq"], c["layout"])
    s["q_out"].copy_(q.flatten(1))
    if c["kind"] == "qk":
        s["k_out"].copy_(k.flatten(1))
        return
    page, off = (s["slots"] // c["page"]).long(), (s["slots"] % c["page"]).long()
    for name, x in (("ck", k), ("cv", split(s["v"]))):
        code, scale = _quantise(x, c["type"])
        s[name][page, :, off] = code
        if scale is not None:
            s[name + "s"][page, :, off] = scale


def _qkv_out(s):
    if s["case"]["kind"] == "qk":
        return [s["q_out"], s["k_out"]]
    return {name: s[name] for name in ("q_out", "ck", "cv", "cks", "cvs") if s[name] is not None}


def _gather(s, seq_table, key):
    """Values of the keys `key` [B, L] of the sequences of a table [B, pages]: K and V as [B, kv_heads, L, dim]."""
    page = s["case"]["page"]
    at = seq_table.long().gather(1, key // page)
    out = []
    for name in ("ck", "cv"):
        x = s[name][at, :, key % page].float()
        if s[name + "s"] is not None:
            x = x * s[name + "s"][at, :, key % page][..., None]
        out.append(x.transpose(1, 2))
    return out


def _softmax_values(scores, sees, v):
    """Rows of scores [.., rows, keys] over the keys they see, times v; zeros where a row sees none."""
    p = torch.softmax(scores.masked_fill_(~sees, -math.inf), -1)
    return torch.where(sees.any(-1, keepdim=True), p, 0.0) @ v


def _places(start, t):
    """The sequence of each packed row, and its place there."""
    row = torch.arange(t, device=start.device)
    seq = torch.searchsorted(start[1:].long(), row, right=True)
    return seq, row - start[seq]


def _window(s):
    c = s["case"]
    dev, dim, kv_heads, group = s["q"].device, c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    start, n = s["start"].long(), s["kv_len"].long()
    t, b, q_max = s["q"].shape[0], n.numel(), c["q_max"]
    n_q = start[1:] - start[:-1]
    # keys that some row may see: the first ones, and those from the first row's window on
    low = torch.maximum(n - n_q + 1 - c["window"], torch.tensor(c["sinks"], device=dev))
    span = min(c["kv_max"], c["window"] + q_max)
    key = torch.cat((torch.arange(min(c["sinks"], c["kv_max"]), device=dev).expand(b, -1), low[:, None] + torch.arange(span, device=dev)), 1)
    there = key < n[:, None]
    k, v = _gather(s, s["table"], torch.where(there, key, 0))
    rows = (start[:-1, None] + torch.arange(q_max, device=dev)).clamp_max(t - 1)
    q = s["q"].float().view(t, kv_heads, group, dim)[rows].permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, kv_heads, group * q_max, dim]
    up = n[:, None] - n_q[:, None] + torch.arange(1, q_max + 1, device=dev)
    sees = there[:, None] & (key[:, None] < up[..., None]) & ((key[:, None] < c["sinks"]) | (key[:, None] >= up[..., None] - c["window"]))
    sees = sees[:, None].repeat(1, 1, group, 1)
    o = _softmax_values(q @ k.transpose(-1, -2) / math.sqrt(dim), sees, v)
    o = o.view(b, kv_heads, group, q_max, dim).permute(0, 3, 1, 2, 4).reshape(b, q_max, -1)
    seq, off = _places(start, t)
    s["out"].copy_(o[seq, off])


def _window_prompt(s):
    c = s["case"]
    dim, kv_heads, group = c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    at = 0
    for n in s["n"]:
        for i in range(0, n, 1024):  # the queries i .. e - 1 and the keys they see
            e = min(n, i + 1024)
            lo = max(0, i + 1 - c["window"])
            key = torch.arange(lo, e, device=s["q"].device)
            if min(lo, c["sinks"]):
                key = torch.cat((torch.arange(min(lo, c["sinks"]), device=key.device), key))
            k, v = (s[name][at + key].float().view(-1, kv_heads, dim).transpose(0, 1) for name in ("k", "v"))
            q = s["q"][at + i:at + e].float().view(e - i, kv_heads, group, dim).permute(1, 2, 0, 3).flatten(1, 2)
            up = torch.arange(i + 1, e + 1, device=key.device)[:, None]
            sees = (key < up) & ((key < c["sinks"]) | (key >= up - c["window"]))
            o = _softmax_values(q @ k.transpose(-1, -2) / math.sqrt(dim), sees.repeat(group, 1), v)
            s["out"][at + i:at + e] = o.view(kv_heads, group, e - i, dim).permute(2, 0, 1, 3).reshape(e - i, -1)
        at += n


def _shared(s):
    c = s["case"]
    dev, dim, kv_heads, group = s["q"].device, c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    q_max = c["q_max"]
    t = s["q"].shape[0]
    b = 0
    for many, pre in zip(_groups(c), s["pre"]):
        start, n = s["start"][b:b + many + 1].long(), s["kv_len"][b:b + many].long()
        n_q = start[1:] - start[:-1]
        own_max = c["own_max"]
        pk, pv = _gather(s, s["table"][b:b + 1], torch.arange(pre, device=dev)[None])
        key = pre + torch.arange(own_max, device=dev).expand(many, -1)
        there = key < n[:, None]
        k, v = _gather(s, s["table"][b:b + many], torch.where(there, key, 0))
        rows = (start[:-1, None] + torch.arange(q_max, device=dev)).clamp_max(t - 1)
        q = s["q"].float().view(t, kv_heads, group, dim)[rows].permute(0, 2, 3, 1, 4).flatten(2, 3)  # [many, kv_heads, rows, dim]
        up = n[:, None] - n_q[:, None] + torch.arange(1, q_max + 1, device=dev)
        sees = (there[:, None] & (key[:, None] < up[..., None])).repeat(1, group, 1)[:, None]
        r = q.shape[2]
        flat = q.transpose(0, 1).flatten(1, 2)  # [kv_heads, many * rows, dim]: the prefix once for all of them
        first = (flat @ pk[0].transpose(-1, -2)).unflatten(1, (many, r)).transpose(0, 1)
        p = torch.cat((first, (q @ k.transpose(-1, -2)).masked_fill_(~sees, -math.inf)), -1)
        p = torch.softmax(p.mul_(1 / math.sqrt(dim)), -1)
        o = (p[..., :pre].transpose(0, 1).flatten(1, 2) @ pv[0]).unflatten(1, (many, r)).transpose(0, 1) + p[..., pre:] @ v
        o = o.view(many, kv_heads, group, q_max, dim).permute(0, 3, 1, 2, 4).reshape(many, q_max, -1)
        lo, hi = sum(s["q_n"][:b]), sum(s["q_n"][:b + many])
        seq, off = _places(start - lo, hi - lo)
        s["out"][lo:hi] = o[seq, off].to(torch.bfloat16)
        b += many


def run(s):
    if own:
        return _run_own(s)
    kind = s["case"]["kind"]
    if kind == "plan":
        _plan(s)
        return _plan_out(s)
    if kind in ("qkv", "qk"):
        _qkv(s)
        return _qkv_out(s)
    {"window": _window, "window_prompt": _window_prompt, "shared": _shared}[kind](s)
    return s["out"]


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _handles(s):
    """What a program makes once: the frequency table, the norms' weights and the cache's description."""
    import ternary_sparse_binary_b200 as wal
    c = s["case"]
    if c["kind"] == "plan":  # the pages themselves are not looked at
        s["cache"] = wal.KvCache.empty(s["n_pages"], c["page"], 1, 64)
    if "rot" in c:
        s["rope"] = wal.Rope(c["dim"], c["rot"], base=1e6, layout=c["layout"])
        s["norm"] = wal.HeadNorm(s["wq"], s["wk"], eps=EPS)
    if "ck" in s:
        s["cache"] = wal.KvCache(s["ck"], s["cv"], s["cks"], s["cvs"])
    s["wal"] = wal


def _run_own(s):
    if "wal" not in s:
        _handles(s)
    c, wal = s["case"], s["wal"]
    kind = c["kind"]
    if kind == "plan":
        s["cache"].plan(s["n_new"], s["kv_len"], s["table"], s["free"], s["n_free"], s["q_start"], s["positions"], s["slots"],
                        kv_len_out=s["len_out"], n_free_out=s["n_free_out"])
        return _plan_out(s)
    if kind == "qk":
        s["rope"].apply_qk(s["q"], s["k"], s["pos"], s["q_out"], s["k_out"], norm=s["norm"])
        return _qkv_out(s)
    if kind == "qkv":
        s["cache"].append_qkv(s["q"], s["k"], s["v"], s["slots"], s["q_out"], positions=s["pos"], rope=s["rope"], norm=s["norm"])
        return _qkv_out(s)
    if kind == "window":
        s["cache"].attend(s["q"], s["start"], s["kv_len"], s["table"], s["out"], max_q=c["q_max"], max_kv=c["kv_max"], window=c["window"],
                          sinks=c["sinks"])
    elif kind == "window_prompt":
        wal.attn_prompt(s["q"], s["k"], s["v"], s["start"], s["out"], head_dim=c["dim"], max_len=c["q_max"], window=c["window"], sinks=c["sinks"])
    else:
        s["cache"].attend_shared(s["q"], s["start"], s["kv_len"], s["table"], s["group_start"], s["prefix_len"], s["out"], max_q=c["q_max"],
                                 max_kv=max(s["n"]), max_prefix=max(s["pre"]), max_own=c["own_max"])
    return s["out"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _seen(up, window, sinks):
    """Keys that a row with `up` keys up to itself sees."""
    return min(up, window + min(sinks, max(0, up - window)))


def work(case):
    size = {"bf16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
    kind = case["kind"]
    if kind == "plan":
        page = case["page"]
        held, new = _requests(case)
        pages = lambda n: -(-n // page)
        moved = sum(abs(pages(v + m) - pages(v)) for v, m in zip(held, new))
        t = sum(max(0, m) for m in new)
        return {"bytes": 16 * case["batch"] + 8 * moved + 8 * (t + case["pad"]), "flops": 4 * (t + case["batch"])}
    dim, heads, row = case["dim"], case["heads"], 2 * case["kv_heads"]
    if kind == "qk":
        n = case["tokens"] * (heads + case["kv_heads"]) * dim
        return {"bytes": n * (size[case["inp"]] + 2) + 4 * case["tokens"], "flops": 7 * n}
    if kind == "window_prompt":
        n, _ = _lengths(case)
        pairs = sum(_seen(i + 1, case["window"], case["sinks"]) for v in n for i in range(v))
        return {"bytes": 2 * sum(n) * dim * (2 * heads + row), "flops": 4 * dim * heads * pairs}
    held = row * (dim * size[case["type"]] + (0 if case["type"] == "bf16" else 4))  # one token in the cache
    if kind == "qkv":
        t = case["tokens"]
        return {"bytes": t * ((heads + row) * dim * size[case["inp"]] + 2 * heads * dim + held + 8), "flops": t * dim * (7 * heads + 8 * row)}
    q, n = _lengths(case)
    if kind == "window":
        keys = pairs = 0
        for m, v in zip(q, n):
            pairs += sum(_seen(v - m + i + 1, case["window"], case["sinks"]) for i in range(m))
            low = max(0, v - m + 1 - case["window"])
            keys += v - low + min(low, case["sinks"])
    else:
        pre = _prefixes(case)
        of = [v for v, many in zip(pre, _groups(case)) for _ in range(many)]
        keys = sum(pre) + sum(n)
        pairs = sum(m * (p + v) - m * (m - 1) // 2 for m, v, p in zip(q, n, of))
    return {"bytes": keys * held + 4 * sum(q) * heads * dim, "flops": 4 * dim * heads * pairs}


# --------------------------------------------------------------------------
# the same in 64 bits, from the definition
# --------------------------------------------------------------------------

def _exact_plan(case, s):
    """One sequence after the other, in whole numbers on the host."""
    page = case["page"]
    held, new = s["kv_len"].tolist(), s["n_new"].tolist()
    table, free, top = s["table"].tolist(), s["free"].tolist(), s["n_free"].item()
    pages_of = lambda n: math.ceil(n / page)
    for b, m in enumerate(new):
        if m < 0:
            for i in range(pages_of(held[b] + m), pages_of(held[b])):
                free[top] = table[b][i]
                top += 1
    start, positions, slots = [0], [], []
    for b, m in enumerate(new):
        for i in range(pages_of(held[b]), pages_of(held[b] + m)):
            top -= 1
            table[b][i] = free[top]
        for p in range(held[b], held[b] + m):
            positions.append(p)
            slots.append(table[b][p // page] * page + p % page)
        start.append(len(slots))
    rest = s["slots"].numel() - len(slots)
    after = [v + m for v, m in zip(held, new)]
    values = [start, positions + [0] * rest, slots + [-1] * rest, after, [top], table, free]
    return [torch.tensor(v, dtype=torch.int32, device="cuda") for v in values]


def _exact_head(x, w, pos, freq, layout):
    x = x * w.double() * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
    y = x.clone()
    half = freq.numel()
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + half)
        a = pos.double() * freq[i]
        z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * torch.complex(a.cos(), a.sin())[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_codes(x, typ):
    if typ == "bf16":
        return x, None
    scale = torch.clamp(x.abs().max(-1).values / QMAX[typ], min=TINY)
    y = x / scale.unsqueeze(-1)  # three bits behind the leading one, steps of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale


def _exact_rows(q, k, v, up, low, sinks, group):
    """Rows q [n, heads, dim] over k, v [keys, kv_heads, dim]; row i sees j < up[i] with j >= low[i] or j < sinks."""
    n, heads, dim = q.shape
    out = torch.zeros(n, heads, dim, dtype=torch.float64, device=q.device)
    step = 1 + (1 << 24) // max(1, len(k))
    for i in range(0, n, step):
        u, l = up[i:i + step], low[i:i + step]
        first, last = max(0, int(l.min())), int(u.max())
        j = torch.arange(len(k), device=q.device)
        j = j[((j >= first) | (j < sinks)) & (j < last)]
        hidden = ~((j < u[:, None]) & ((j >= l[:, None]) | (j < sinks)))
        for h in range(heads):
            e = q[i:i + step, h] @ k[j, h // group].T * dim ** -0.5
            e[hidden] = -math.inf
            e = torch.exp(e - e.amax(1, keepdim=True))
            out[i:i + step, h] = (e @ v[j, h // group]) / e.sum(1, keepdim=True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "plan":
        return _exact_plan(case, s)
    dim, heads, kv_heads = case["dim"], case["heads"], case["kv_heads"]
    split = lambda x: x.double().reshape(len(x), -1, dim)
    if kind in ("qkv", "qk"):
        q = _exact_head(split(s["q"]), s["wq"], s["pos"], s["freq"], case["layout"]).flatten(1)
        k = _exact_head(split(s["k"]), s["wk"], s["pos"], s["freq"], case["layout"])
        if kind == "qk":
            return [q, k.flatten(1)]
        out = {"q_out": q}
        slot = s["slots"].long()
        made = {"ck": _exact_codes(k, case["type"]), "cv": _exact_codes(split(s["v"]), case["type"])}
        for key, new in [(name, made[name][0]) for name in made] + [(name + "s", made[name][1]) for name in made]:
            if s[key] is not None:
                flat = s[key].double().transpose(1, 2).flatten(0, 1)  # [slots, heads, ...]
                flat[slot] = new
                out[key] = flat.unflatten(0, (-1, case["page"])).transpose(1, 2)
        return out
    start = s["start"].tolist()
    out = torch.empty(start[-1], heads, dim, dtype=torch.float64, device="cuda")
    for b, (lo, hi) in enumerate(zip(start, start[1:])):
        if kind == "window_prompt":
            k, v = split(s["k"][lo:hi]), split(s["v"][lo:hi])
        else:
            n = s["n"][b]
            pages = s["table"][b, : -(-n // case["page"])].long()
            k, v = ((s[x][pages].double() * (1.0 if s[x + "s"] is None else s[x + "s"][pages].double().unsqueeze(-1)))
                    .transpose(1, 2).reshape(-1, kv_heads, dim)[:n] for x in ("ck", "cv"))
        up = torch.arange(len(k) - (hi - lo) + 1, len(k) + 1, device="cuda")
        low = up - case["window"] if "window" in case else torch.zeros_like(up)
        out[lo:hi] = _exact_rows(split(s["q"][lo:hi]), k, v, up, low, case.get("sinks", 0), heads // kv_heads)
    return out.reshape(start[-1], -1)
