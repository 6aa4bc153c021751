"""Attention with a sliding window and first tokens that stay visible vs the FP64 oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from oracle import step_oracle as so

from attn_util import TYPES, assert_close, attention_tolerance, bf16, random_cache
from gpu_util import needs_gpu, wal
from test_gpu_attention import SENTINEL, dev, i32
from test_gpu_attention_nonfinite import WITHIN, normal, us

pytestmark = [pytest.mark.gpu, needs_gpu]


def check(got, q, ks, vs, start, heads, kv_heads, D, window, sinks, sc):
    for b, (k, v) in enumerate(zip(ks, vs)):
        qb = q[start[b]:start[b + 1]].reshape(-1, heads, D)
        if len(qb):
            o, a = so.attend(qb, k, v, sc, heads // kv_heads, so.window_sees(len(qb), len(k), window, sinks))
            tol = attention_tolerance(o, a, qb, k, sc)
            assert_close(got[start[b]:start[b + 1], :heads * D].reshape(o.shape), o, tol, f"sequence {b}")


def run_paged(lens, n_q, window, sinks, heads=8, kv_heads=2, D=128, page=32, typ="bf16", seed=0, spread=2.0, bounds=None, scale=None,
              gone=True):
    """One call; with `gone`, the pages that no new token sees are taken out of the table."""
    w = wal()
    rng = np.random.default_rng(seed)
    tensors, table, ks, vs = random_cache(rng, lens, page, kv_heads, D, typ, spread)
    cache = w.KvCache(*[dev(t) for t in tensors])
    lead, trail, pad = 2, 3, 8
    start = lead + np.concatenate([[0], np.cumsum(n_q)])
    T = int(start[-1]) + trail
    q = bf16(rng.normal(size=(T, heads * D)))
    Q = torch.full((T, heads * D + pad), float("nan"), dtype=torch.bfloat16)
    Q[:, :heads * D] = torch.from_numpy(q).bfloat16()
    O = torch.full((T, heads * D + pad), SENTINEL, dtype=torch.bfloat16, device="cuda")
    max_q, max_kv = bounds or (max(max(n_q), 1), max(max(lens), 1))
    nb = max(cache.attend_workspace_bytes(heads, T, len(lens), max_q, max_kv, window, sinks), 512)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    tab = np.full((len(lens), max(-(-max_kv // page), table.shape[1])), -9, np.int32)
    tab[:, :table.shape[1]] = table
    if gone:
        for b, (L, n) in enumerate(zip(lens, n_q)):
            seen = so.window_sees(n, L, window, sinks).any(0)
            for i in range(-(-L // page)):
                if not seen[i * page:(i + 1) * page].any():
                    tab[b, i] = -9
    cache.attend(Q.cuda()[:, :heads * D], i32(start), i32(lens), torch.from_numpy(tab).cuda(), O[:, :heads * D], max_q=max_q, max_kv=max_kv,
                 ws=ws, scale=scale, window=window, sinks=sinks)
    w.attention.status(ws)
    got = O.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == SENTINEL), "columns past the heads were written"
    assert np.all(got[:lead] == SENTINEL) and np.all(got[T - trail:] == SENTINEL), "rows of no sequence were written"
    check(got, q, ks, vs, start, heads, kv_heads, D, window, sinks, 1 / math.sqrt(D) if scale is None else scale)


def run_prompt(lens, window, sinks, heads=8, kv_heads=2, D=128, seed=0, spread=2.0):
    w = wal()
    rng = np.random.default_rng(seed)
    lead, trail, pad = 1, 2, 8
    start = lead + np.concatenate([[0], np.cumsum(lens)])
    T = int(start[-1]) + trail
    x, t = {}, {}
    for name, h in (("q", heads), ("k", kv_heads), ("v", kv_heads)):
        x[name] = bf16(rng.normal(size=(T, h * D)) * (spread if name == "k" else 1))
        buf = torch.full((T, h * D + pad), float("nan"), dtype=torch.bfloat16)
        buf[lead:T - trail, :h * D] = torch.from_numpy(x[name][lead:T - trail]).bfloat16()
        t[name] = buf.cuda()[:, :h * D]
    O = torch.full((T, heads * D + pad), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((512,), 0xFF, dtype=torch.uint8, device="cuda")
    w.attn_prompt(t["q"], t["k"], t["v"], i32(start), O[:, :heads * D], head_dim=D, max_len=max(max(lens), 1), ws=ws, window=window, sinks=sinks)
    w.attention.status(ws)
    got = O.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == SENTINEL)
    assert np.all(got[:lead] == SENTINEL) and np.all(got[T - trail:] == SENTINEL)
    ks, vs = ([x[name][start[b]:start[b + 1]].reshape(n, kv_heads, D) for b, n in enumerate(lens)] for name in ("k", "v"))
    check(got, x["q"], ks, vs, start, heads, kv_heads, D, window, sinks, 1 / math.sqrt(D))


WINDOWS = [(1, 0), (1, 1), (15, 4), (16, 16), (17, 0), (64, 17), (100, 130), (300, 3), (129, 64)]


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_single_tokens(window, sinks, typ):
    run_paged([1, 16, 37, 300, 0, 129, 700], [1] * 7, window, sinks, typ=typ, seed=window)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("sinks", [0, 20])
@pytest.mark.parametrize("n", [1, 90])
def test_pages(n, sinks, page, typ):
    run_paged([page - 1, page + 1, 3 * page + 5, 5 * page + 100, n], [min(n, page - 1), n, n, n, n], page + 9, sinks, D=64, page=page, typ=typ, seed=page)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("heads,kv_heads,D", [(4, 4, 64), (7, 1, 128), (16, 1, 64), (40, 1, 128), (128, 1, 64)])
@pytest.mark.parametrize("n", [1, 33])
def test_head_layouts(n, heads, kv_heads, D, typ):
    run_paged([150, 20, 260, 700], [n, 20 if n > 1 else 1, n, n], 70, 5, heads, kv_heads, D, 16, typ, seed=heads + D)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("n_q,lens", [([2, 4, 3], [2, 100, 500]), ([16, 9, 0], [300, 9, 40]), ([70, 33, 1], [70, 400, 650]),
                                      ([129, 400], [129, 1000])])
def test_chunks(n_q, lens, window, sinks, typ):
    run_paged(lens, n_q, window, sinks, typ=typ, seed=sum(n_q) + window)


@pytest.mark.parametrize("typ", list(TYPES))
def test_long(typ):
    """Windows whose keys are split over CTAs, of single tokens and of chunks; pages that no token sees are gone."""
    run_paged([9000, 3000, 4100], [1, 1, 1], 2500, 10, typ=typ, seed=5, page=64)
    run_paged([9000, 700], [90, 2], 3000, 70, 4, 1, typ=typ, seed=6, page=128)
    run_paged([5000], [300], 2000, 0, 2, 1, 64, typ=typ, seed=7, page=256)


@pytest.mark.parametrize("n_q", [1, 3, 60])
def test_rows_without_keys(n_q):
    for typ in TYPES:
        run_paged([1, 0, 2, n_q], [n_q] * 4, 1, 0, page=16, typ=typ, seed=n_q)
        run_paged([1, 0, 2, n_q], [n_q] * 4, 2, 1, page=16, typ=typ, seed=n_q, bounds=(n_q, 4000))


@pytest.mark.parametrize("scale", [0.0, 0.5, -0.2])
def test_scale_and_loose_bounds(scale):
    run_paged([90, 200], [1, 1], 33, 2, D=64, scale=scale)
    run_paged([90, 200], [70, 40], 33, 2, D=64, scale=scale, bounds=(500, 30000))


@pytest.mark.parametrize("window,sinks", WINDOWS + [(2000, 0), (5, 3000)])
def test_prompts(window, sinks):
    run_prompt([1, 100, 0, 257, 33, 600], window, sinks, seed=window)
    run_prompt([700, 129], window, sinks, 4, 4, 64, seed=sinks)


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 383, 640])
def test_prompt_lengths(n):
    run_prompt([n, 3], 100, 4, 4, 2, seed=n, spread=4.0)
    run_prompt([n], 128, 0, 3, 1, 64, seed=n, spread=4.0)


def test_prompt_long():
    run_prompt([2500], 700, 40, 4, 1, seed=1)
    run_prompt([2500], 1024, 0, 2, 2, seed=2)


def test_a_window_beyond_the_sequence_is_none():
    w = wal()
    T = 300
    q, k, v = normal(T, 1024), normal(T, 256), normal(T, 256)
    outs = [torch.empty_like(q) for _ in range(3)]
    for out, kw in zip(outs, ({}, dict(window=T), dict(window=2 ** 40, sinks=5))):
        w.attn_prompt(q, k, v, i32([0, T]), out, head_dim=128, max_len=T, **kw)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---- non-finite values -----------------------------------------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("sinks", [0, 5])
def test_hidden_nonfinite_values_stay_hidden_in_prompts(sinks, where, bad):
    """Token j of sequence 1 is bad: only the rows whose window holds it may change."""
    w = wal()
    lens, window, D, j = [70, 700, 50], 90, 64, 250
    start = np.concatenate([[0], np.cumsum(lens)])
    T = int(start[-1])
    q, k, v = normal(T, 4 * D), normal(T, 2 * D), normal(T, 2 * D)
    call = lambda out: w.attn_prompt(q, k, v, i32(start), out, head_dim=D, max_len=700, window=window, sinks=sinks)
    ref, out = torch.empty_like(q), torch.empty_like(q)
    call(ref)
    (k if where == "k" else v)[start[1] + j, :D] = bad
    call(out)
    hit = torch.zeros(T, 4 * D, dtype=torch.bool, device="cuda")
    hit[start[1] + j:start[1] + j + window, :2 * D] = True
    r, o = ref.float(), out.float()
    # a row near the bad key may be computed another way: the weights' and the output's roundings to bf16
    assert torch.isfinite(o[~hit]).all()
    assert torch.all((o - r)[~hit].abs() <= 2.0 ** -7 * r[~hit].abs() + 6 * 2.0 ** -8)
    if where == "v" or bad != bad:
        assert not torch.isfinite(o[hit]).any()


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n_q,L,split", [(4, 9000, True), (60, 700, False), (300, 9000, True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_hidden_nonfinite_values_stay_hidden_in_pages(bad, n_q, L, split, typ):
    """A bad V (or its scale) at the first key of the first row's window, which the rows behind it do not see."""
    w = wal()
    D, page, window = 64, 32, 3000 if split else 100
    n = -(-L // page)
    shape = (n, 2, page, D)
    if typ == "bf16":
        cache = w.KvCache(normal(*shape), normal(*shape))
    else:
        code = lambda: torch.randint(0, 100, shape, device="cuda", dtype=torch.uint8).view(TYPES[typ])
        cache = w.KvCache(code(), code(), *[torch.full(shape[:3], 0.01, device="cuda") for _ in range(2)])
    table = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    q = normal(n_q, 8 * D)
    call = lambda out: cache.attend(q, i32([0, n_q]), i32([L]), table, out, max_q=n_q, max_kv=L, window=window, sinks=3)
    ref, out = torch.empty_like(q), torch.empty_like(q)
    call(ref)
    for back in (0, 1):  # the first row's first key, and the second's
        j = L - n_q + 1 - window + back
        x = cache.v[j // page, :, j % page] if typ == "bf16" else cache.v_scale[j // page, :, j % page]
        old = x.clone()
        x.fill_(bad)
        call(out)
        x.copy_(old)
        o, r = out.float(), ref.float()
        assert not torch.isfinite(o[:back + 1]).any()
        rest = slice(back + 1, None)
        assert torch.isfinite(o[rest]).all()
        assert torch.all((o - r)[rest].abs() <= 2.0 ** -7 * r[rest].abs() + 6 * 2.0 ** -8)


def test_a_nan_that_all_see_takes_no_longer():
    w = wal()
    T, D = 4096, 64
    q, k, v, out = normal(T, 8 * D), normal(T, 2 * D), normal(T, 2 * D), torch.empty(T, 8 * D, dtype=torch.bfloat16, device="cuda")
    call = lambda: w.attn_prompt(q, k, v, i32([0, T]), out, head_dim=D, max_len=T, window=500, sinks=4)
    clean = us(call)
    v[:1] = float("nan")
    took = us(call)
    assert torch.isnan(out).all()
    assert took <= WITHIN * clean, f"{took:.0f} us against {clean:.0f}"


# ---- index values ------------------------------------------------------------------------

@pytest.mark.parametrize("n_q,L", [(1, 300), (1, 9000), (40, 300), (40, 9000)])
def test_reports(n_q, L):
    """Lengths and starts out of range leave a sequence out; a page that a token sees is checked, another is not."""
    w = wal()
    D, page, window = 64, 32, 2500 if L > 5000 else 100
    n = -(-L // page)
    cache = w.KvCache(normal(n, 1, page, D), normal(n, 1, page, D))
    table = torch.arange(n, device="cuda", dtype=torch.int32).repeat(2, 1)
    T = 2 * n_q
    q = normal(T, 4 * D)
    shape = (4, T, 2, n_q, L, window, 3)
    ws = torch.empty(max(512, cache.attend_workspace_bytes(*shape)), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 512 or L < 5000

    def call(start=(0, n_q, T), lens=(L, L - 5), tab=table):
        out = torch.full_like(q, SENTINEL)
        cache.attend(q, i32(start), i32(lens), tab, out, max_q=n_q, max_kv=L, window=window, sinks=3, ws=ws)
        try:
            w.attention.status(ws)
        except w.WalError as e:
            assert e.status == w.WAL_ERR_ARG
            return out, True
        return out, False
    ref, bad = call()
    assert not bad and torch.isfinite(ref).all()
    for kw in (dict(lens=(L, -1)), dict(lens=(L, L + 1)), dict(start=(0, n_q, n_q - 1)), dict(start=(0, n_q, T + 1))):
        out, bad = call(**kw)
        assert bad and torch.equal(out[:n_q], ref[:n_q]) and (out[n_q:] == SENTINEL).all()
    for at, counts in ((0, True), (1, False), (n - 1, True), ((L - 5 - n_q - window) // page - 1, False), ((L - 5 - n_q + 1 - window) // page, True)):
        tab = table.clone()
        tab[1, at] = n
        out, bad = call(tab=tab)
        assert bad == counts and torch.equal(out[:n_q], ref[:n_q]), at
        assert counts or torch.equal(out, ref)


@pytest.mark.parametrize("n_q", [1, 50])
def test_in_a_graph(n_q):
    """Replays read lengths and starts anew; two captured calls share a workspace in turn."""
    w = wal()
    D, page, L = 128, 64, 6000
    n = -(-L // page)
    cache = w.KvCache(normal(2 * n, 2, page, D), normal(2 * n, 2, page, D))
    table = torch.randperm(2 * n, device="cuda").int().view(2, n)
    q, start, lens = normal(2 * n_q, 8 * D), i32([0, n_q, 2 * n_q]), i32([L, L])
    ws = torch.empty(cache.attend_workspace_bytes(8, 2 * n_q, 2, n_q, L, 3000, 4), dtype=torch.uint8, device="cuda")
    out, out2, ref = (torch.empty_like(q) for _ in range(3))
    call = lambda out: cache.attend(q, start, lens, table, out, max_q=n_q, max_kv=L, window=3000, sinks=4, ws=ws)
    call(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
        call(out2)
    for a, b in ((L, L - 900), (n_q, 3000 + n_q), (70, L)):
        lens.copy_(i32([a, b]))
        g.replay()
        call(ref)
        assert torch.equal(out, ref) and torch.equal(out2, ref)
