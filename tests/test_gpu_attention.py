"""Attention over the paged cache and over packed prompts vs the FP64 oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao

from attn_util import TYPES, assert_close, attention_tolerance, bf16, random_cache
from gpu_util import needs_gpu, wal

pytestmark = [pytest.mark.gpu, needs_gpu]

SENTINEL = 77.0


def dev(x):
    return None if x is None else x.cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_paged(lens, n_q, heads, kv_heads, D, page, typ, seed=0, spread=1.0, lead=2, trail=3, pad=8, bounds=None,
              scale=None, ws=None):
    """One call over `lens` tokens held and `n_q` new ones each, with `lead` and
    `trail` rows of no sequence around them and `pad` extra columns."""
    w = wal()
    rng = np.random.default_rng(seed)
    tensors, table, ks, vs = random_cache(rng, lens, page, kv_heads, D, typ, spread)
    cache = w.KvCache(*[dev(t) for t in tensors])
    start = lead + np.concatenate([[0], np.cumsum(n_q)])
    T = int(start[-1]) + trail
    q = bf16(rng.normal(size=(T, heads * D)))
    Q = torch.full((T, heads * D + pad), float("nan"), dtype=torch.bfloat16)
    Q[:, :heads * D] = torch.from_numpy(q).bfloat16()
    Q = Q.cuda()
    O = torch.full((T, heads * D + pad), SENTINEL, dtype=torch.bfloat16, device="cuda")
    max_q, max_kv = bounds or (max(max(n_q), 1), max(max(lens), 1))
    if ws is None:
        nb = max(cache.attend_workspace_bytes(heads, T, len(lens), max_q, max_kv), 512)
        ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")  # nothing in it may count
    width = -(-max_kv // page)
    tab = np.full((len(lens), max(width, table.shape[1])), -9, np.int32)
    tab[:, :table.shape[1]] = table
    cache.attend(Q[:, :heads * D], i32(start), i32(lens), torch.from_numpy(tab).cuda(), O[:, :heads * D],
                 max_q=max_q, max_kv=max_kv, ws=ws, scale=scale)
    w.attention.status(ws)
    got = O.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == SENTINEL), "columns past the heads were written"
    assert np.all(got[:lead] == SENTINEL) and np.all(got[T - trail:] == SENTINEL), "rows of no sequence were written"
    sc = 1 / math.sqrt(D) if scale is None else scale
    for b, (k, v) in enumerate(zip(ks, vs)):
        qb = q[start[b]:start[b + 1]].reshape(-1, heads, D)
        if len(qb):
            o, a = ao.attend(qb, k, v, sc, heads // kv_heads)
            tol = attention_tolerance(o, a, qb, k, sc)
            assert_close(got[start[b]:start[b + 1], :heads * D].reshape(o.shape), o, tol, f"sequence {b}")
    return O


def run_prompt(lens, heads, kv_heads, D, seed=0, spread=1.0, lead=1, trail=2, pad=8, max_len=None):
    w = wal()
    rng = np.random.default_rng(seed)
    start = lead + np.concatenate([[0], np.cumsum(lens)])
    T = int(start[-1]) + trail
    x = {"q": bf16(rng.normal(size=(T, heads * D))), "k": bf16(rng.normal(size=(T, kv_heads * D)) * spread),
         "v": bf16(rng.normal(size=(T, kv_heads * D)))}
    t = {}
    for name, val in x.items():
        buf = torch.full((T, val.shape[1] + pad), float("nan"), dtype=torch.bfloat16)
        buf[lead:T - trail, :val.shape[1]] = torch.from_numpy(val[lead:T - trail]).bfloat16()
        t[name] = buf.cuda()[:, :val.shape[1]]
    O = torch.full((T, heads * D + pad), SENTINEL, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((512,), 0xFF, dtype=torch.uint8, device="cuda")
    w.attn_prompt(t["q"], t["k"], t["v"], i32(start), O[:, :heads * D], head_dim=D, max_len=max_len or max(max(lens), 1), ws=ws)
    w.attention.status(ws)
    got = O.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == SENTINEL)
    assert np.all(got[:lead] == SENTINEL) and np.all(got[T - trail:] == SENTINEL)
    for b, n in enumerate(lens):
        if n:
            qb, k, v = (x[name][start[b]:start[b + 1]].reshape(n, -1, D) for name in ("q", "k", "v"))
            o, a = ao.attend(qb, k, v, 1 / math.sqrt(D), heads // kv_heads)
            tol = attention_tolerance(o, a, qb, k, 1 / math.sqrt(D))
            assert_close(got[start[b]:start[b + 1], :heads * D].reshape(o.shape), o, tol, f"sequence {b}")
    return O


# ---- single tokens -----------------------------------------------------------

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("heads,kv_heads,D", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (16, 1, 64), (5, 1, 128), (40, 1, 128)])
def test_decode_head_layouts(heads, kv_heads, D, typ):
    run_paged([1, 16, 37, 300, 0, 129], [1] * 6, heads, kv_heads, D, 32, typ, seed=heads)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages(page, typ):
    run_paged([page - 1, page, page + 1, 3 * page + 5, 1], [1] * 5, 8, 2, 128, page, typ, seed=page, spread=3.0)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [15, 17, 63, 64, 65, 255, 256, 257, 1023, 2049, 5000])
def test_decode_lengths(n, typ):
    """Around the steps and splits of the keys, with peaked weights."""
    run_paged([n, max(1, n // 2)], [1, 1], 8, 2, 128, 16, typ, seed=n, spread=4.0)


def test_decode_loose_bounds():
    """max_q and max_kv far above what the batch has."""
    run_paged([5, 700, 64], [1, 1, 0], 8, 2, 128, 64, "bf16", bounds=(4, 20000))


# ---- several new tokens --------------------------------------------------------

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n_q,lens", [([2, 4, 3], [2, 100, 50]), ([8, 1, 5], [8, 1, 999]), ([16, 9, 0], [300, 9, 40]),
                                      ([70, 33, 1], [70, 400, 65]), ([129, 200], [129, 1000])])
def test_chunks(n_q, lens, typ):
    run_paged(lens, n_q, 8, 2, 128, 32, typ, seed=sum(n_q), spread=2.0)


@pytest.mark.parametrize("heads,kv_heads,D", [(6, 2, 64), (7, 1, 128), (4, 4, 128), (16, 16, 64), (33, 1, 64), (128, 1, 64)])
@pytest.mark.parametrize("typ", ["bf16", "int8", "e4m3"])
def test_chunk_head_layouts(heads, kv_heads, D, typ):
    run_paged([150, 20, 260], [40, 20, 1], heads, kv_heads, D, 16, typ, seed=heads + D, spread=2.0)


@pytest.mark.parametrize("typ", ["bf16", "e4m3"])
def test_chunk_over_long_cache(typ):
    run_paged([4100, 130], [60, 2], 4, 1, 128, 128, typ, seed=5, spread=3.0)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n_q", [3, 60])
def test_rows_without_keys(n_q, typ):
    """More new tokens than the sequence holds: the first see nothing and get zeros."""
    O = run_paged([1, 0, 2, n_q], [n_q] * 4, 8, 2, 128, 16, typ, seed=n_q)
    got = O.cpu().float()[2:]
    assert not got[:n_q - 1, :1024].any() and not got[n_q:2 * n_q, :1024].any()


@pytest.mark.parametrize("n_q", [1, 4, 64])
def test_scale_argument(n_q):
    for scale in (0.0, 0.5, -0.2):
        run_paged([90, 200], [n_q, n_q], 8, 2, 64, 32, "bf16", scale=scale, seed=n_q)


# ---- prompts -------------------------------------------------------------------

@pytest.mark.parametrize("heads,kv_heads,D", [(8, 2, 128), (4, 4, 64), (7, 1, 64), (3, 3, 128), (12, 4, 128)])
def test_prompt_head_layouts(heads, kv_heads, D):
    run_prompt([1, 100, 0, 257, 33], heads, kv_heads, D, seed=heads, spread=2.0)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 640])
def test_prompt_lengths(n):
    run_prompt([n, 3], 4, 2, 128, seed=n, spread=4.0)
    run_prompt([n], 2, 2, 64, seed=n, spread=4.0, lead=0, trail=0, pad=0)


def test_prompt_long():
    run_prompt([2500], 4, 1, 128, seed=1, spread=3.0)


# ---- non-finite and masked values ------------------------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_nonfinite_keys_stay_where_they_are(where, bad, D):
    """A non-finite K or V at token j of sequence 1: rows before j and the other
    sequences are as if it were not there; rows from j on follow the formula
    (not finite, for a value in V or a NaN in K)."""
    w = wal()
    rng = np.random.default_rng(11)
    lens, heads, kv = [70, 300, 50], 4, 2
    start = np.concatenate([[0], np.cumsum(lens)])
    T = start[-1]
    q, k, v = (bf16(rng.normal(size=(T, h * D))) for h in (heads, kv, kv))
    t = [torch.from_numpy(x).bfloat16().cuda() for x in (q, k, v)]
    ref = torch.empty_like(t[0])
    w.attn_prompt(*t, i32(start), ref, head_dim=D, max_len=300)
    j = start[1] + 150
    t[1 if where == "k" else 2][j, :D] = bad  # K/V head 0
    out = torch.empty_like(ref)
    w.attn_prompt(*t, i32(start), out, head_dim=D, max_len=300)
    r, o = ref.float().cpu(), out.float().cpu()
    hit = torch.zeros(T, heads * D, dtype=torch.bool)
    hit[j:start[2], :2 * D] = True
    # a row near the bad key may be computed another way: the weights' rounding
    # to bf16 (2^-8 of at most max |v| < 6) and two roundings of the output
    assert torch.all(torch.isfinite(o[~hit]))
    assert torch.all((o - r)[~hit].abs() <= 2.0 ** -7 * r[~hit].abs() + 6 * 2.0 ** -8)
    if where == "v" or bad != bad:
        assert not torch.isfinite(o[hit]).any() or where == "k"
        if bad != bad:
            assert torch.isnan(o[hit]).all()


@pytest.mark.parametrize("typ", ["bf16", "int8"])
@pytest.mark.parametrize("n_q", [4, 40])
def test_paged_nonfinite_future_keys(n_q, typ):
    """The last token's V (and its scale) is NaN: only the last new token's row may see it."""
    w = wal()
    rng = np.random.default_rng(12)
    lens = [100, 60]
    (k, v, ks, vs), table, kv, vv = random_cache(rng, lens, 16, 2, 128, typ)
    pg, off = table[0, 99 // 16], 99 % 16
    if typ == "bf16":
        v[pg, :, off] = float("nan")
    else:
        vs[pg, :, off] = float("nan")
    cache = w.KvCache(*[dev(t) for t in (k, v, ks, vs)])
    q = bf16(rng.normal(size=(2 * n_q, 8 * 128)))
    Q = torch.from_numpy(q).bfloat16().cuda()
    O = torch.empty_like(Q)
    cache.attend(Q, i32([0, n_q, 2 * n_q]), i32(lens), torch.from_numpy(table).cuda(), O, max_q=n_q, max_kv=100)
    got = O.cpu().double().numpy()
    assert np.isnan(got[n_q - 1]).all()
    for b in range(2):
        rows = slice(b * n_q, (b + 1) * n_q - (1 - b))
        qb = q[b * n_q:(b + 1) * n_q].reshape(n_q, 8, 128)
        vb = vv[b].copy()
        if b == 0:
            vb[-1] = 0
        o, a = ao.attend(qb, kv[b], vb, 128 ** -0.5, 4)
        tol = attention_tolerance(o, a, qb, kv[b], 128 ** -0.5)
        n = n_q - (1 - b)
        assert_close(got[rows].reshape(n, 8, 128), o[:n], tol[:n], f"sequence {b}")


@pytest.mark.parametrize("n_q", [1, 30])
def test_extreme_scores(n_q):
    """Scores around +-1e4 and at the lowest finite values: weights of exactly zero and one."""
    w = wal()
    D, L = 64, 80
    k = torch.zeros(5, 1, 16, D, dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    rng = np.random.default_rng(13)
    vals = bf16(rng.normal(size=(L, D)))
    for j in range(L):
        k[j // 16, 0, j % 16, 0] = -3.0e38 if j % 3 else 1.0e4 * (j % 5)
        v[j // 16, 0, j % 16] = torch.from_numpy(vals[j]).bfloat16()
    Q = torch.zeros(n_q, D, dtype=torch.bfloat16)
    Q[:, 0] = 1.0
    O = torch.empty(n_q, D, dtype=torch.bfloat16, device="cuda")
    w.KvCache(dev(k), dev(v)).attend(Q.cuda(), i32([0, n_q]), i32([L]), i32([[0, 1, 2, 3, 4]]), O, max_q=n_q, max_kv=L,
                                     scale=1.0)
    got = O.cpu().double().numpy()
    for i in range(n_q):
        lim = L - n_q + i + 1
        best = [j for j in range(lim) if j % 3 == 0]
        top = max(j % 5 for j in best)
        ref = np.mean([vals[j] for j in best if j % 5 == top], 0)
        size = np.mean([np.abs(vals[j]) for j in best if j % 5 == top], 0)
        assert np.all(np.abs(got[i] - ref) <= 2.0 ** -8 * (size + np.abs(ref)) * 1.01)


@pytest.mark.parametrize("n_q,L,typ", [(200, 700, "bf16"), (20, 700, "bf16"), (20, 700, "int8"), (20, 9000, "bf16"), (1, 900, "int8"), (300, 300, "bf16")])
def test_scores_that_jump(n_q, L, typ):
    """One key among the later ones tops all before it by hundreds of nats, for
    every other column of the batch's rows: its value alone remains."""
    w = wal()
    rng = np.random.default_rng(L + n_q)
    D, page = 64, 16
    (k, v, ks, vs), table, kv, vv = random_cache(rng, [L], page, 1, D, typ)
    jump = L - n_q // 2 - 1 if n_q > 1 else L - 5
    scale = 1.0 / D
    kv, vv = kv[0].copy(), vv[0]
    pg, off = table[0, jump // page], jump % page
    if typ == "bf16":
        k[pg, 0, off] = 1000.0
        kv[jump] = 1000.0
    else:
        k[pg, 0, off] = 100
        ks[pg, 0, off] = 10.0
        kv[jump] = 1000.0
    q = bf16(np.ones((n_q, 2 * D)) * np.where(np.arange(2 * D) < D, 1.0, -1.0) + 0.25 * rng.normal(size=(n_q, 2 * D)))
    Q = torch.from_numpy(q).bfloat16().cuda()
    O = torch.empty_like(Q)
    w.KvCache(*[dev(t) for t in (k, v, ks, vs)]).attend(Q, i32([0, n_q]), i32([L]), torch.from_numpy(table).cuda(), O,
                                                        max_q=n_q, max_kv=L, scale=scale)
    qb = q.reshape(n_q, 2, D)
    o, a = ao.attend(qb, kv, vv, scale, 2)
    assert_close(O.cpu().double().numpy().reshape(o.shape), o, attention_tolerance(o, a, qb, kv, scale))
    if n_q == L:
        O2 = torch.empty_like(Q)
        dense = [torch.from_numpy(x.reshape(L, D)).bfloat16().cuda() for x in (kv, vv)]
        w.attn_prompt(Q, *dense, i32([0, L]), O2, head_dim=D, max_len=L, scale=scale)
        assert_close(O2.cpu().double().numpy().reshape(o.shape), o, attention_tolerance(o, a, qb, kv, scale))


# ---- bad indexes -----------------------------------------------------------------

@pytest.mark.parametrize("n_q", [1, 40])
def test_bad_indexes_are_reported_and_harmless(n_q):
    w = wal()
    rng = np.random.default_rng(14)
    lens = [50, 60, 70]
    (k, v, ks, vs), table, kv, vv = random_cache(rng, lens, 16, 2, 64, "bf16")
    cache = w.KvCache(dev(k), dev(v))
    q = bf16(rng.normal(size=(3 * n_q, 4 * 64)))
    Q = torch.from_numpy(q).bfloat16().cuda()
    starts = [0, n_q, 2 * n_q, 3 * n_q]
    ws = torch.empty(max(512, cache.attend_workspace_bytes(4, 3 * n_q, 3, n_q, 80)), dtype=torch.uint8, device="cuda")

    def call(tab=table, kv_len=lens, q_start=starts):
        O = torch.full_like(Q, SENTINEL)
        cache.attend(Q, i32(q_start), i32(kv_len), torch.from_numpy(tab).cuda(), O, max_q=n_q, max_kv=80, ws=ws)
        try:
            w.attention.status(ws)
            return O.cpu().double().numpy(), False
        except w.WalError as e:
            assert e.status == w.WAL_ERR_ARG
            return O.cpu().double().numpy(), True

    fine, bad = call()
    assert not bad
    for page in (-1, cache.n_pages, 2 ** 31 - 1, -2 ** 31):  # one page of sequence 1: 0 and 2 are as before
        tab = table.copy()
        tab[1, 1] = page
        got, bad = call(tab=tab)
        assert bad and np.array_equal(got[:n_q], fine[:n_q]) and np.array_equal(got[2 * n_q:], fine[2 * n_q:])
    for length in (-1, 81, 2 ** 31 - 1):
        got, bad = call(kv_len=[50, length, 70])
        assert bad and np.all(got[n_q:2 * n_q] == SENTINEL)
        assert np.array_equal(got[:n_q], fine[:n_q]) and np.array_equal(got[2 * n_q:], fine[2 * n_q:])
    got, bad = call(q_start=[0, n_q, 2 * n_q, 3 * n_q + 1])
    assert bad and np.all(got[2 * n_q:] == SENTINEL) and np.array_equal(got[:2 * n_q], fine[:2 * n_q])
    got, bad = call(q_start=[-1, n_q, 2 * n_q, 3 * n_q])
    assert bad and np.all(got[:n_q] == SENTINEL) and np.array_equal(got[n_q:], fine[n_q:])
    got, bad = call()
    assert not bad and np.array_equal(got, fine)


# ---- streams, graphs, repetition ---------------------------------------------------

@pytest.mark.parametrize("n_q,typ", [(1, "int8"), (1, "bf16"), (50, "bf16"), (50, "e4m3")])
def test_graph_replay_reads_new_lengths(n_q, typ):
    """A captured call replayed with other lengths, on its own stream, twice the same bits."""
    w = wal()
    rng = np.random.default_rng(15)
    tensors, table, kv, vv = random_cache(rng, [900, 333], 64, 2, 128, typ)
    cache = w.KvCache(*[dev(t) for t in tensors])
    q = bf16(rng.normal(size=(2 * n_q, 8 * 128)))
    Q = torch.from_numpy(q).bfloat16().cuda()
    O = torch.empty_like(Q)
    start, lens = i32([0, n_q, 2 * n_q]), i32([900, 333])
    tab = torch.from_numpy(table).cuda()
    ws = torch.empty(cache.attend_workspace_bytes(8, 2 * n_q, 2, n_q, 900), dtype=torch.uint8, device="cuda")
    call = lambda: cache.attend(Q, start, lens, tab, O, max_q=n_q, max_kv=900, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    first = O.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    O.fill_(SENTINEL)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, first)
    lens.copy_(i32([700, 60]))
    g.replay()
    torch.cuda.synchronize()
    got = O.cpu().double().numpy().reshape(2, n_q, 8, 128)
    for b, n in enumerate((700, 60)):
        qb = q[b * n_q:(b + 1) * n_q].reshape(n_q, 8, 128)
        o, a = ao.attend(qb, kv[b][:n], vv[b][:n], 128 ** -0.5, 4)
        assert_close(got[b], o, attention_tolerance(o, a, qb, kv[b][:n], 128 ** -0.5), f"sequence {b}")


def test_two_streams_at_once():
    """Two calls with workspaces of their own on two streams give what each gives alone."""
    w = wal()
    rng = np.random.default_rng(16)
    tensors, table, _, _ = random_cache(rng, [3000, 2500], 64, 2, 128, "int8")
    cache = w.KvCache(*[dev(t) for t in tensors])
    tab, lens = torch.from_numpy(table).cuda(), i32([3000, 2500])
    args = []
    for n_q in (1, 40):
        Q = torch.from_numpy(bf16(rng.normal(size=(2 * n_q, 1024)))).bfloat16().cuda()
        args.append((Q, i32([0, n_q, 2 * n_q]), n_q))
    alone, streams = [], [torch.cuda.Stream() for _ in args]
    for Q, start, n_q in args:
        O = torch.empty_like(Q)
        cache.attend(Q, start, lens, tab, O, max_q=n_q, max_kv=3000)
        alone.append(O)
    torch.cuda.synchronize()
    outs = [torch.empty_like(Q) for Q, _, _ in args]
    torch.cuda.synchronize()
    for _ in range(20):
        for (Q, start, n_q), O, s in zip(args, outs, streams):
            cache.attend(Q, start, lens, tab, O, max_q=n_q, max_kv=3000, stream=s)
    torch.cuda.synchronize()
    for O, ref in zip(outs, alone):
        assert torch.equal(O, ref)


def test_large_offsets():
    """Pages whose elements lie past 2^32 bytes from the base."""
    w = wal()
    n_pages, page, heads, D = 70000, 64, 8, 128  # 9.2 GB in each of k and v
    cache = w.KvCache.empty(n_pages, page, heads, D)
    rng = np.random.default_rng(17)
    lens, picks = [100, 100], [[n_pages - 1, 3], [n_pages - 2, 36000]]
    vals = []
    for pg in picks:
        k, v = (bf16(rng.normal(size=(100, heads, D))) for _ in range(2))
        for j in range(100):
            cache.k[pg[j // page], :, j % page] = torch.from_numpy(k[j]).bfloat16().cuda()
            cache.v[pg[j // page], :, j % page] = torch.from_numpy(v[j]).bfloat16().cuda()
        vals.append((k, v))
    for n_q in (1, 40):
        q = bf16(rng.normal(size=(2 * n_q, heads * D)))
        O = torch.empty(2 * n_q, heads * D, dtype=torch.bfloat16, device="cuda")
        cache.attend(torch.from_numpy(q).bfloat16().cuda(), i32([0, n_q, 2 * n_q]), i32(lens), i32(picks), O, max_q=n_q, max_kv=128)
        got = O.cpu().double().numpy().reshape(2, n_q, heads, D)
        for b, (k, v) in enumerate(vals):
            qb = q[b * n_q:(b + 1) * n_q].reshape(n_q, heads, D)
            o, a = ao.attend(qb, k, v, D ** -0.5, 1)
            assert_close(got[b], o, attention_tolerance(o, a, qb, k, D ** -0.5), f"sequence {b}")
