"""Workloads of the attention operators: rotary positions, the paged KV cache
(append, read back), attention over the cache and over a whole prompt.

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


def listed():
    return [
        # one decode step of 25 concurrent sequences of an 8B-shaped model: the q heads after their fp32 product
        dict(name="rope_decode", kind="rope", tokens=25, heads=32, dim=128, rot=128, layout="half", inp="fp32", scaling="none", far=32768, lens=1),
        # a long packed prompt, positions scaled by parts for a long context, part of each head rotated
        dict(name="rope_prompt", kind="rope", tokens=16384, heads=40, dim=128, rot=64, layout="interleaved", inp="bf16", scaling="parts", far=131072, lens=2),
        # the same decode step's keys and values into an 8-bit cache (25 rows, pages of 16)
        dict(name="append_decode", kind="append", tokens=25, kv_heads=8, dim=128, rot=128, layout="half", inp="fp32", type="e4m3", page=16, pages=512, scaling="none", far=32768, lens=3),
        # a prompt's keys and values into an 8-bit cache
        dict(name="append_prompt", kind="append", tokens=16381, kv_heads=8, dim=128, rot=128, layout="half", inp="bf16", type="e4m3", page=64, pages=320, scaling="linear", far=65536, lens=4),
        # written in integers and read back for a few sequences (prefix reuse, checks of a cache)
        dict(name="append_read", kind="append_read", tokens=2000, kv_heads=8, dim=128, rot=64, layout="interleaved", inp="fp32", type="int8", page=32, pages=128, scaling="none", far=4096, batch=5, lens=5),
        # a whole 8-bit cache of 25 ragged sequences read back to bf16 rows
        dict(name="read_int8", kind="read", batch=25, kv_max=8192, kv_heads=8, dim=128, type="int8", page=64, lens=6),
        # one user's decode step at a context of 2048, bf16 cache: the smallest attention call, latency counts
        dict(name="decode_one", kind="paged", batch=1, q_max=1, kv_max=2048, heads=32, kv_heads=8, dim=128, type="bf16", page=64, ragged=False, lens=7),
        # 25 serving slots, ragged contexts up to 32768, 8-bit cache: the memory-bound decode step
        dict(name="decode_slots", kind="paged", batch=25, q_max=1, kv_max=32768, heads=32, kv_heads=8, dim=128, type="int8", page=64, ragged=True, lens=8),
        # a chunk of a long prompt over what the cache holds already
        dict(name="chunk_long", kind="paged", batch=2, q_max=1024, kv_max=16384, heads=32, kv_heads=8, dim=128, type="bf16", page=128, ragged=True, lens=9),
        # several drafted tokens per slot, ungrouped heads of 64, 8-bit floating-point cache
        dict(name="chunk_draft", kind="paged", batch=16, q_max=100, kv_max=4096, heads=16, kv_heads=16, dim=64, type="e4m3", page=16, ragged=True, lens=10),
        # a batch of ragged prompts, one head of keys per query head (27B-shaped projections)
        dict(name="prompt_packed", kind="prompt", batch=9, q_max=1000, heads=40, kv_heads=40, dim=128, ragged=True, lens=11),
        # one long prompt of an 8B-shaped model: the largest product
        dict(name="prompt_long", kind="prompt", batch=1, q_max=8192, heads=32, kv_heads=8, dim=128, ragged=False, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "append_read", "read", "paged", "paged", "paged", "prompt", "prompt"])
    c = dict(kind=kind, lens=rng.randrange(1 << 20), dim=rng.choice([64, 128]))
    kv_heads, group = rng.choice([(1, 8), (2, 7), (4, 8), (8, 4), (8, 3), (5, 4), (16, 1), (16, 2), (40, 1)])
    if kind in ("rope", "append", "append_read"):
        c.update(rot=rng.choice([c["dim"], c["dim"], c["dim"] // 2]), layout=rng.choice(["half", "interleaved"]),
                 inp=rng.choice(["fp32", "bf16"]), scaling=rng.choice(["none", "linear", "parts"]),
                 far=_log_int(rng, 64, 131072), tokens=_log_int(rng, 1, 8192))
    if kind == "rope":
        c.update(heads=kv_heads * group)
    elif kind in ("append", "append_read"):
        page = rng.choice([16, 32, 64, 128])
        c.update(kv_heads=kv_heads, page=page, pages=-(-c["tokens"] // page) + rng.randrange(8, 40))
        if kind == "append":
            c.update(type=rng.choice(["bf16", "e4m3"]))
        else:
            c["batch"] = rng.randrange(1, 9)
            c["pages"] += c["batch"]
            c.update(type=rng.choice(["bf16", "int8", "e4m3"]))
    elif kind == "read":
        kv = _log_int(rng, 16, 8192)
        c.update(batch=_log_int(rng, 1, max(1, min(32, 190_000_000 // (kv * kv_heads * 4 * c["dim"])))), kv_max=kv, kv_heads=kv_heads,
                 type=rng.choice(["bf16", "int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]))
    elif kind == "paged":
        kv = _log_int(rng, 16, 32768)
        q = 1 if rng.random() < 0.4 else min(kv, _log_int(rng, 2, 1024))
        most = max(1, min(32, 190_000_000 // (kv * kv_heads * c["dim"]), (1 << 30) // (q * kv * kv_heads * group)))
        c.update(batch=_log_int(rng, 1, most), q_max=q, kv_max=kv, heads=kv_heads * group, kv_heads=kv_heads,
                 type=rng.choice(["bf16", "int8", "e4m3"]), page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
    else:
        q = _log_int(rng, 1, 6000)
        most = max(1, min(32, 16384 // q, (1 << 30) // (q * q * kv_heads * group)))
        c.update(batch=_log_int(rng, 1, most), q_max=q, heads=kv_heads * group, kv_heads=kv_heads, ragged=rng.random() < 0.7)
    return c


# --------------------------------------------------------------------------
# what a case fixes: lengths and frequencies
# --------------------------------------------------------------------------

def _lengths(case):
    """(new tokens, tokens held) of each sequence, from the case alone."""
    rng = random.Random(case["lens"])
    kind = case["kind"]
    if kind == "append_read":  # `tokens` cut into `batch` pieces
        b, t = case["batch"], case["tokens"]
        cut = sorted(rng.randrange(t + 1) for _ in range(b - 1))
        n = [hi - lo for lo, hi in zip([0] + cut, cut + [t])]
        return n, n
    most = case["kv_max"] if kind in ("read", "paged") else case["q_max"]
    n = [most] * case["batch"]
    if case.get("ragged", True):
        n = [max(1, min(most, int(most * rng.uniform(0.05, 1.1)))) for _ in n]
        n[rng.randrange(len(n))] = most
    if kind != "paged":
        return n, n
    q = [min(case["q_max"], v) for v in n]
    if case["ragged"] and case["q_max"] > 1:
        q = [rng.randint(1, v) for v in q]
    return q, n


def _frequencies(rot, scaling):
    """Radians a position for each pair (64 bits) and the factor on the result."""
    base, factor, original = 1e6, 4.0, 32768.0
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":  # fast pairs as they are, slow ones interpolated, a ramp between
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return (1 - keep) * f / factor + keep * f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _start(n, device):
    return torch.tensor([0] + n, device=device).cumsum(0).to(torch.int32)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    kind, dim = case["kind"], case["dim"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = {"case": dict(case)}
    if "rot" in case:
        s["freq"], s["mscale"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = s["freq"].to(dev)
        first = int(torch.randint(0, case["far"], (1,), generator=g, device=dev))
        t = case["tokens"]
        # a decode step: every row at a place of its own; a prompt: rows one after another
        s["pos"] = (torch.randint(0, case["far"], (t,), generator=g, device=dev) if t < 64
                    else first + torch.arange(t, device=dev)).to(torch.int32)
    if kind == "rope":
        s["x"] = normal(case["tokens"], case["heads"] * dim, dtype=TYPES[case["inp"]])
        s["out"] = torch.empty(case["tokens"], case["heads"] * dim, dtype=torch.bfloat16, device=dev)
        return s
    if kind == "prompt":
        n, _ = _lengths(case)
        t = sum(n)
        s.update(n=n, start=_start(n, dev), q=normal(t, case["heads"] * dim), k=normal(t, case["kv_heads"] * dim),
                 v=normal(t, case["kv_heads"] * dim), out=torch.empty(t, case["heads"] * dim, dtype=torch.bfloat16, device=dev))
        return s

    # a cache: pages dealt out in no order, slots that nobody wrote hold an earlier user's values
    page, heads, typ = case["page"], case["kv_heads"], case["type"]
    if kind != "append":
        q, n = _lengths(case)
        need = [-(-v // page) for v in n]
        pages = case.get("pages", sum(need) + 3)
        table = torch.zeros(case["batch"], max(max(need), 1), dtype=torch.int32)
        deal = torch.randperm(pages, generator=g, device=dev).cpu().to(torch.int32)
        at = 0
        for b, v in enumerate(need):
            table[b, :v] = deal[at:at + v]
            at += v
        s.update(n=n, table=table.to(dev), start=_start(q, dev), kv_len=torch.tensor(n, dtype=torch.int32, device=dev))
    else:
        pages = case["pages"]
    shape = (pages, heads, page, dim)
    if typ == "bf16":
        s["k"], s["v"] = normal(*shape), normal(*shape)
        s["ks"] = s["vs"] = None
    else:
        for name in ("k", "v"):
            x = torch.randn(shape, generator=g, device=dev)
            sc = (x.abs().amax(-1) / QMAX[typ]).clamp_min(TINY)
            x /= sc[..., None]
            s[name] = x.round_().to(torch.int8) if typ == "int8" else x.to(TYPES[typ])
            s[name + "s"] = sc
            del x
    if kind in ("append", "append_read"):
        t = case["tokens"]
        s["new_k"] = normal(t, heads * dim, dtype=TYPES[case["inp"]])
        s["new_v"] = normal(t, heads * dim, dtype=TYPES[case["inp"]])
        if kind == "append":
            s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:t].to(torch.int32)
        else:
            seq, off = _places(s["start"], t)
            s["slots"] = s["table"][seq, off // page] * page + (off % page).to(torch.int32)
    if kind in ("read", "append_read"):
        t = sum(s["n"])
        s["out_k"] = torch.empty(t, heads * dim, dtype=torch.bfloat16, device=dev)
        s["out_v"] = torch.empty(t, heads * dim, dtype=torch.bfloat16, device=dev)
    if kind == "paged":
        t = int(s["start"][-1])
        s["q"] = normal(t, case["heads"] * dim)
        s["out"] = torch.empty(t, case["heads"] * dim, dtype=torch.bfloat16, device=dev)
    return s


def _places(start, t):
    """The sequence of each packed row, and its place there."""
    row = torch.arange(t, device=start.device)
    seq = torch.searchsorted(start[1:].long(), row, right=True)
    return seq, row - start[seq]


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _rotate(x, pos, freq, mscale, layout):
    """x [T, heads, dim] in 32 bits, rotated in its first 2 * len(freq) columns."""
    a = pos.double()[:, None, None] * freq
    c, s = (a.cos() * mscale).float(), (a.sin() * mscale).float()
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
    y = x / scale[..., None]
    return (y.round().to(torch.int8) if typ == "int8" else y.to(TYPES[typ])), scale


def _append(s):
    c = s["case"]
    k = s["new_k"].float().view(-1, c["kv_heads"], c["dim"])
    v = s["new_v"].float().view(-1, c["kv_heads"], c["dim"])
    k = _rotate(k, s["pos"], s["freq"], s["mscale"], c["layout"])
    page, off = (s["slots"] // c["page"]).long(), (s["slots"] % c["page"]).long()
    for name, x in (("k", k), ("v", v)):
        code, scale = _quantise(x, c["type"])
        s[name][page, :, off] = code
        if scale is not None:
            s[name + "s"][page, :, off] = scale


def _read(s):
    c = s["case"]
    seq, off = _places(s["start"], s["out_k"].shape[0])
    page, at = s["table"][seq, off // c["page"]].long(), off % c["page"]
    out = []
    for name in ("k", "v"):
        x = s[name][page, :, at].float()
        if s[name + "s"] is not None:
            x = x * s[name + "s"][page, :, at][..., None]
        out.append(x.to(torch.bfloat16).flatten(1))
    return out


def _attend(q, k, v, start, kv_len, q_max):
    """Packed q [T, heads, dim] over padded k, v [B, kv_heads, L, dim], all 32 bits: [T, heads * dim] bf16."""
    t, heads, dim = q.shape
    b, kv_heads, most, _ = k.shape
    start = start.long()
    n_q = start[1:] - start[:-1]
    rows = start[:-1, None] + torch.arange(q_max, device=q.device)
    padded = q[rows.clamp_max(t - 1)].view(b, q_max, kv_heads, heads // kv_heads, dim).permute(0, 2, 3, 1, 4)
    key = torch.arange(most, device=q.device)
    v = torch.where((key < kv_len[:, None])[:, None, :, None], v, 0.0)
    limit = kv_len[:, None] - n_q[:, None] + torch.arange(q_max, device=q.device)
    sees = (key <= limit[..., None]) & (key < kv_len[:, None, None])
    p = (padded.flatten(2, 3) @ k.transpose(-1, -2)).view(b, kv_heads, -1, q_max, most) / math.sqrt(dim)
    p = torch.softmax(p.masked_fill_(~sees[:, None, None], -math.inf), -1)
    o = (p.flatten(2, 3) @ v).view(b, kv_heads, -1, q_max, dim).permute(0, 3, 1, 2, 4).reshape(b, q_max, heads * dim)
    seq, off = _places(start, t)
    return o[seq, off].to(torch.bfloat16)


def _paged(s):
    c = s["case"]
    table = s["table"].long()

    def dense(x, scale):
        y = x[table].float()  # [B, pages, heads, page, dim]
        if scale is not None:
            y = y * scale[table][..., None]
        return y.transpose(1, 2).flatten(2, 3)

    return _attend(s["q"].float().view(-1, c["heads"], c["dim"]), dense(s["k"], s["ks"]), dense(s["v"], s["vs"]),
                   s["start"], s["kv_len"], c["q_max"])


def _prompt(s):
    c = s["case"]
    start = s["start"].long()
    n = start[1:] - start[:-1]
    rows = (start[:-1, None] + torch.arange(c["q_max"], device=start.device)).clamp_max(s["q"].shape[0] - 1)

    def dense(x):
        return x.float().view(-1, c["kv_heads"], c["dim"])[rows].transpose(1, 2)

    return _attend(s["q"].float().view(-1, c["heads"], c["dim"]), dense(s["k"]), dense(s["v"]), start, n, c["q_max"])


def _cache_out(s):
    return {name: s[name] for name in ("k", "v", "ks", "vs") if s[name] is not None}


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["kind"] == "rope":
        x = s["x"].float().view(-1, c["heads"], c["dim"])
        return _rotate(x, s["pos"], s["freq"], s["mscale"], c["layout"]).to(torch.bfloat16).flatten(1)
    if c["kind"] == "append":
        _append(s)
        return _cache_out(s)
    if c["kind"] == "append_read":
        _append(s)
        return _read(s)
    if c["kind"] == "read":
        return _read(s)
    return _paged(s) if c["kind"] == "paged" else _prompt(s)


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _handles(s):
    """What a program makes once: the frequency table and the cache's description."""
    import ternary_sparse_binary_b200 as wal
    c = s["case"]
    if "rot" in c:
        kw = {"none": {}, "linear": dict(scaling="linear", factor=4.0),
              "parts": dict(scaling="parts", factor=4.0, original_len=32768, slow=1.0, fast=32.0)}[c["scaling"]]
        s["rope"] = wal.Rope(c["dim"], c["rot"], base=1e6, layout=c["layout"], **kw)
    if "page" in c:
        s["cache"] = wal.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    s["wal"] = wal


def _run_own(s):
    if "wal" not in s:
        _handles(s)
    c, wal = s["case"], s["wal"]
    kind = c["kind"]
    if kind == "rope":
        s["rope"].apply(s["x"], s["pos"], s["out"])
        return s["out"]
    if kind in ("append", "append_read"):
        s["cache"].append(s["new_k"], s["new_v"], s["slots"], positions=s["pos"], rope=s["rope"])
        if kind == "append":
            return _cache_out(s)
    if kind in ("append_read", "read"):
        s["cache"].read(s["table"], s["start"], s["out_k"], s["out_v"], max_len=max(s["n"]))
        return [s["out_k"], s["out_v"]]
    if kind == "paged":
        s["cache"].attend(s["q"], s["start"], s["kv_len"], s["table"], s["out"], max_q=c["q_max"], max_kv=c["kv_max"])
        return s["out"]
    wal.attn_prompt(s["q"], s["k"], s["v"], s["start"], s["out"], head_dim=c["dim"], max_len=c["q_max"])
    return s["out"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
    kind, dim = case["kind"], case["dim"]
    if kind == "rope":
        n = case["tokens"] * case["heads"] * dim
        return {"bytes": n * (size[case["inp"]] + 2) + 4 * case["tokens"], "flops": 3 * n}
    row = case["kv_heads"] * 2  # (head, K or V) rows of one token
    if kind == "prompt":
        n, _ = _lengths(case)
        t = sum(n)
        return {"bytes": 2 * t * dim * (2 * case["heads"] + row),
                "flops": sum(2 * dim * case["heads"] * v * (v + 1) for v in n)}
    held = row * (dim * size[case["type"]] + (0 if case["type"] == "bf16" else 4))  # one token in the cache
    if kind in ("append", "append_read"):
        t = case["tokens"]
        b = t * (row * dim * size[case["inp"]] + held + 8)
        if kind == "append_read":
            b += t * (held + row * dim * 2)
        return {"bytes": b, "flops": 8 * t * row * dim}
    q, n = _lengths(case)
    if kind == "read":
        return {"bytes": sum(n) * (held + row * dim * 2), "flops": sum(n) * row * dim}
    pairs = sum(m * v - m * (m - 1) // 2 for m, v in zip(q, n))
    return {"bytes": sum(n) * held + 4 * sum(q) * case["heads"] * dim, "flops": 4 * dim * case["heads"] * pairs}


# --------------------------------------------------------------------------
# the same in 64 bits, from the definition, one row or one sequence at a time
# --------------------------------------------------------------------------

def _exact_rotate(x, pos, freq, mscale, layout):
    half = freq.numel()
    y = x.clone()
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + half)
        turn = torch.polar(torch.full_like(pos, mscale, dtype=torch.float64), pos.double() * freq[i])[:, None]
        z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_codes(x, typ):
    if typ == "bf16":
        return x, None, x
    scale = torch.clamp(x.abs().max(-1).values / QMAX[typ], min=TINY)
    y = x / scale.unsqueeze(-1)
    if typ == "int8":
        y = torch.round(y)
    else:  # three bits behind the leading one, steps of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        y = torch.round(y / step) * step
    return y, scale, y * scale.unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    kind, dim = case["kind"], case["dim"]
    if kind == "rope":
        x = s["x"].double().reshape(-1, case["heads"], dim)
        return _exact_rotate(x, s["pos"], s["freq"], s["mscale"], case["layout"]).reshape(x.shape[0], -1)
    if kind in ("append", "append_read"):
        heads = case["kv_heads"]
        k = _exact_rotate(s["new_k"].double().reshape(-1, heads, dim), s["pos"], s["freq"], s["mscale"], case["layout"])
        v = s["new_v"].double().reshape(-1, heads, dim)
        made = {"k": _exact_codes(k, case["type"]), "v": _exact_codes(v, case["type"])}
        if kind == "append_read":
            return [made[name][2].reshape(len(k), -1) for name in ("k", "v")]
        slot = s["slots"].long()
        out = {}
        for name in ("k", "v"):
            for key, new in ((name, made[name][0]), (name + "s", made[name][1])):
                if s[key] is not None:
                    flat = s[key].double().transpose(1, 2).flatten(0, 1)  # [slots, heads, ...]
                    flat[slot] = new
                    out[key] = flat.unflatten(0, (-1, case["page"])).transpose(1, 2)
        return out

    def sequence(b):
        """K and V of sequence b, [tokens, kv_heads, dim]."""
        n = s["n"][b]
        pages = s["table"][b, : -(-n // case["page"])].long()
        both = []
        for name in ("k", "v"):
            x = s[name][pages].double()
            if s[name + "s"] is not None:
                x *= s[name + "s"][pages].double().unsqueeze(-1)
            both.append(x.transpose(1, 2).reshape(-1, case["kv_heads"], dim)[:n])
        return both

    if kind == "read":
        both = [sequence(b) for b in range(case["batch"])]
        return [torch.cat([x[i] for x in both]).reshape(-1, case["kv_heads"] * dim) for i in (0, 1)]
    start = s["start"].tolist()
    group = case["heads"] // case["kv_heads"]
    out = torch.empty(start[-1], case["heads"], dim, dtype=torch.float64, device="cuda")
    for b, (lo, hi) in enumerate(zip(start, start[1:])):
        if kind == "prompt":
            k, v = (s[name][lo:hi].double().reshape(hi - lo, -1, dim) for name in ("k", "v"))
        else:
            k, v = sequence(b)
        q = s["q"][lo:hi].double().reshape(hi - lo, -1, dim)
        hidden = torch.ones(hi - lo, len(k), dtype=torch.bool, device="cuda").triu(len(k) - (hi - lo) + 1)
        for h in range(case["heads"]):
            e = q[:, h] @ k[:, h // group].T * dim ** -0.5
            e[hidden] = -math.inf
            e = torch.exp(e - e.amax(1, keepdim=True))
            out[lo:hi, h] = (e @ v[:, h // group]) / e.sum(1, keepdim=True)
    return out.reshape(start[-1], -1)
