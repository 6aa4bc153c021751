"""Attention of sequences that share their first tokens vs the FP64 oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao

from attn_util import TYPES, assert_close, attention_tolerance, bf16, random_cache
from gpu_util import needs_gpu, wal
from test_gpu_attention import SENTINEL, dev, i32
from test_gpu_attention_nonfinite import WITHIN, normal, us
from test_gpu_attention_timeout import POLLS, check as check_timeout

pytestmark = [pytest.mark.gpu, needs_gpu]


class Batch:
    """Sequences of `alone` (of no group), then `groups`, then `after` (of no group): a group is (shared tokens,
    [(new tokens, tokens behind the shared ones)]).  The shared pages are those of the group's first sequence."""

    def __init__(self, groups, alone=(), after=(), heads=8, kv_heads=2, D=128, page=32, typ="bf16", seed=0, spread=2.0, lead=2, trail=3):
        w = wal()
        rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.D, self.page, self.lead, self.trail = heads, kv_heads, D, page, lead, trail
        seqs = [(0, None, n, m) for n, m in alone]
        self.starts = [len(alone)]
        for g, (pre, members) in enumerate(groups):
            seqs += [(pre, len(alone) + sum(len(m) for _, m in groups[:g]), n, m) for n, m in members]
            self.starts.append(len(seqs))
        seqs += [(0, None, n, m) for n, m in after]
        # what each sequence holds itself: all of it, or what is behind the shared pages
        keep = [0 if first in (None, b) else pre // page * page for b, (pre, first, _, _) in enumerate(seqs)]
        lens = [pre + m for pre, _, _, m in seqs]
        tensors, own, ks, vs = random_cache(rng, [n - c for n, c in zip(lens, keep)], page, kv_heads, D, typ, spread)
        self.cache = w.KvCache(*[dev(t) for t in tensors])
        width = max(-(-max(lens) // page), 1)
        self.table = np.full((len(seqs), width), -9, np.int32)  # shared entries of all but a group's first stay that
        self.k, self.v = [], []
        for b, (pre, first, _, _) in enumerate(seqs):
            n = -(-(lens[b] - keep[b]) // page)
            self.table[b, keep[b] // page:keep[b] // page + n] = own[b, :n]
            for out, own_vals in ((self.k, ks), (self.v, vs)):
                head = out[first][:pre] if first not in (None, b) else own_vals[b][:pre]
                out.append(np.concatenate([head, own_vals[b][pre - keep[b]:]]))
        self.n_q, self.lens, self.prefix = [n for _, _, n, _ in seqs], lens, [pre for pre, _ in groups]
        self.pre = [pre for pre, _, _, _ in seqs]
        self.start = lead + np.concatenate([[0], np.cumsum(self.n_q)])
        self.T = int(self.start[-1]) + trail
        self.q = bf16(rng.normal(size=(self.T, heads * D)))
        self.Q = torch.full((self.T, heads * D + 8), float("nan"), dtype=torch.bfloat16)
        self.Q[:, :heads * D] = torch.from_numpy(self.q).bfloat16()
        self.Q = self.Q.cuda()
        self.bounds = dict(max_q=max(max(self.n_q), 1), max_kv=max(max(lens), 1), max_prefix=max(self.prefix),
                           max_own=max(1, max(n - p for n, p in zip(lens, self.pre))))
        self.args = dict(q_start=i32(self.start), kv_len=i32(lens), table=torch.from_numpy(self.table).cuda(),
                         group_start=i32(self.starts), prefix_len=i32(self.prefix))

    def ws(self, fill=0xFF):
        b = self.bounds
        n = self.cache.attend_shared_workspace_bytes(self.heads, self.T, len(self.lens), len(self.prefix), b["max_q"], b["max_prefix"], b["max_own"])
        return torch.full((n,), fill, dtype=torch.uint8, device="cuda")

    def call(self, ws=None, scale=None, out=None, stream=None, **change):
        if out is None:
            out = torch.full((self.T, self.heads * self.D + 8), SENTINEL, dtype=torch.bfloat16, device="cuda")
        a = {**self.args, **self.bounds, **change}
        self.cache.attend_shared(self.Q[:, :self.heads * self.D], out=out[:, :self.heads * self.D], scale=scale, ws=ws, stream=stream, **a)
        return out

    def rows(self, b):
        return slice(self.start[b], self.start[b + 1])

    def check(self, O, scale=None, skip=()):
        got = O.cpu().double().numpy()
        width = self.heads * self.D
        assert np.all(got[:, width:] == SENTINEL), "columns past the heads were written"
        assert np.all(got[:self.lead] == SENTINEL) and np.all(got[self.T - self.trail:] == SENTINEL), "rows of no sequence were written"
        sc = 1 / math.sqrt(self.D) if scale is None else scale
        for b, (k, v) in enumerate(zip(self.k, self.v)):
            qb = self.q[self.rows(b)].reshape(-1, self.heads, self.D)
            if b in skip:
                assert np.all(got[self.rows(b)] == SENTINEL), b
            elif len(qb):
                o, a = ao.attend(qb, k, v, sc, self.heads // self.kv_heads)
                assert_close(got[self.rows(b), :width].reshape(o.shape), o, attention_tolerance(o, a, qb, k, sc), f"sequence {b}")


def run(*args, scale=None, bounds=None, **kw):
    b = Batch(*args, **kw)
    b.bounds.update(bounds or {})
    wide = -(-b.bounds["max_kv"] // b.page) - b.table.shape[1]
    if wide > 0:
        b.args["table"] = torch.nn.functional.pad(b.args["table"], (0, wide), value=-9)
    ws = b.ws()
    O = b.call(ws, scale=scale)
    wal().attention.status(ws)
    b.check(O, scale)
    assert torch.equal(b.call(scale=scale), O)  # with scratch of its own
    return b, O


ONE = [(1, 1), (1, 40), (1, 17), (1, 300)]


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("pre", [1, 15, 16, 32, 33, 128, 129, 1000, 5000])
def test_prefix_lengths(pre, typ):
    """Prefixes that end inside a page take their last tokens from the first sequence's row."""
    run([(pre, ONE)], typ=typ, seed=pre)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("n", [1, 50])
def test_pages(n, page, typ):
    run([(3 * page, [(1, 1), (n, n + 5), (n, n + 2 * page + 1)]), (page + 7, [(n, n + page - 1), (1, page + 1)])], alone=[(1, 30)], after=[(n, 60)], page=page,
        typ=typ, D=64, seed=page)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("heads,kv_heads,D", [(4, 4, 64), (7, 1, 128), (16, 1, 64), (40, 1, 128), (128, 1, 64), (16, 16, 128)])
@pytest.mark.parametrize("n", [1, 9])
def test_head_layouts(n, heads, kv_heads, D, typ):
    run([(200, [(n, n + 3)] * 5), (64, [(n, n)])], heads=heads, kv_heads=kv_heads, D=D, page=16, typ=typ, seed=heads)


@pytest.mark.parametrize("typ", list(TYPES))
def test_groups_of_every_kind(typ):
    """A group of one, an empty one, one without a prefix, sequences without new tokens, more than a tile of rows."""
    run([(100, [(1, 5)]), (77, []), (0, [(1, 50), (2, 2)]), (300, [(0, 4), (3, 9), (0, 0)]), (500, [(1, 90)] * 70)], alone=[(0, 0), (2, 6)], typ=typ)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("own", [1, 2500])
def test_long(own, typ):
    run([(9000, [(1, own), (1, 3)] * 3), (4000, [(2, own + 1)] * 4)], typ=typ, D=64, page=64, seed=own)
    run([(3000, [(40, own + 40), (100, 100)])], heads=4, kv_heads=1, typ=typ, page=128, seed=own)


def test_bounds_and_scale():
    run([(100, ONE)], bounds=dict(max_q=4, max_kv=20000, max_prefix=9000, max_own=8000))
    run([(100, [(40, 60), (3, 3)])], bounds=dict(max_q=64, max_kv=20000, max_prefix=9000, max_own=8000))
    for scale in (0.0, 0.5, -0.2):
        run([(100, ONE)], D=64, scale=scale)
        run([(300, [(40, 60), (3, 3)])], D=64, scale=scale)


def test_no_prefix_at_all():
    """max_prefix 0: attention over the cache, as the other entry point computes it."""
    b, O = run([(0, ONE)])
    ref = torch.full_like(O, SENTINEL)
    b.cache.attend(b.Q[:, :1024], b.args["q_start"], b.args["kv_len"], b.args["table"], ref[:, :1024], max_q=1, max_kv=300)
    b.check(ref)


def test_many_sequences():
    rng = np.random.default_rng(3)
    groups = [(int(p), [(1, int(m)) for m in rng.integers(1, 40, n)]) for p, n in zip(rng.integers(1, 200, 40), rng.integers(1, 30, 40))]
    run(groups, heads=2, kv_heads=1, D=64, page=16)


def test_no_tokens():
    b = Batch([(40, [(0, 0), (0, 5)])], lead=0, trail=0)
    ws = b.ws()
    b.call(ws)
    wal().attention.status(ws)
    b.call()


# ---- non-finite values ---------------------------------------------------------------

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [1, 20])
def test_nonfinite_values_reach_only_who_sees_them(n, bad, typ):
    b = Batch([(150, [(n, n + 2), (n, n + 40)]), (90, [(n, n + 9), (1, 3)])], alone=[(1, 30)], typ=typ, D=64)
    ref = b.call()
    x = b.cache.v if typ == "bf16" else b.cache.v_scale

    def poison(row, j):
        page, off = b.table[row, j // b.page], j % b.page
        old = x[page, :, off].clone()
        x[page, :, off] = bad
        out = b.call()
        x[page, :, off] = old
        return out
    last = b.start[3] - 1
    # a token of the prefix, a sequence's own copy of it (which nobody looks at), its first and its last own token
    for row, j, hit in ((1, 149, slice(b.start[1], b.start[3])), (2, 149, slice(0, 0)), (2, 150, b.rows(2)), (2, b.lens[2] - 1, slice(last, last + 1)),
                        (0, 3, b.rows(0))):
        out = poison(row, j)
        seen = torch.zeros(b.T, dtype=torch.bool)
        seen[hit] = True
        o, r = out[:, :512].float().cpu(), ref[:, :512].float().cpu()
        assert not torch.isfinite(o[seen]).any()
        # a row near the bad key may be computed another way: the weights' and the output's roundings to bf16
        assert torch.all((o - r)[~seen].abs() <= 2.0 ** -7 * r[~seen].abs() + 6 * 2.0 ** -8)


def test_a_nan_in_the_prefix_takes_no_longer():
    b = Batch([(4000, [(1, 100)] * 20)], page=64)
    ws = b.ws()
    clean = us(lambda: b.call(ws))
    b.cache.v[b.table[0, 0], :, 0] = float("nan")
    took = us(lambda: b.call(ws))
    assert torch.isnan(b.call(ws)[b.lead:-b.trail, :1024]).all()
    assert took <= WITHIN * clean, f"{took:.0f} us against {clean:.0f}"


# ---- index values ----------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 30])
def test_reports(n):
    """What is out of range leaves its sequence or group out, and is recorded; what is not looked at is not."""
    w = wal()
    b = Batch([(100, [(n, n + 3), (n, n + 50)]), (64, [(1, 9), (1, 20), (n, n)])], alone=[(1, 40)], D=64)
    ws = b.ws()

    def call(skip, **change):
        O = b.call(ws, **change)
        with pytest.raises(w.WalError) as e:
            w.attention.status(ws)
        assert e.value.status == w.WAL_ERR_ARG
        b.check(O, skip=skip)
    s, L, P = list(b.start), list(b.lens), list(b.prefix)
    put = lambda x, i, v: i32(x[:i] + [v] + x[i + 1:])
    call([1], kv_len=put(L, 1, -1))
    call([2], kv_len=put(L, 2, b.bounds["max_kv"] + 1))
    call([4], kv_len=put(L, 4, 64))          # its new token would be part of the prefix
    call([2], max_own=n + 49)
    call([3, 4, 5], prefix_len=put(P, 1, 101))
    call([3, 4, 5], prefix_len=put(P, 1, -1))
    call([3, 4, 5], group_start=i32([1, 3, 7]))
    call(list(range(6)), group_start=i32([1, -1, 6]))
    call([0, 1, 2], group_start=i32([-1, 3, 6]))
    call(list(range(6)), q_start=i32([b.T + 1] * 7))
    for row, at, skip in ((5, 1, None), (2, 2, None), (1, 0, "all"), (0, 0, [0]), (2, 3, [2])):
        tab = b.args["table"].clone()
        tab[row, at] = b.cache.n_pages if at else -1
        O = b.call(ws, table=tab)
        if skip is None:  # pages of the prefix are those of the first sequence's row
            w.attention.status(ws)
            b.check(O)
        else:
            with pytest.raises(w.WalError):
                w.attention.status(ws)


def test_refuses_on_the_device_side_of_the_binding():
    w = wal()
    b = Batch([(100, [(1, 3)] * 3)], D=64)
    with pytest.raises(w.WalError) as e:
        b.call(b.ws()[:-1].clone())
    assert e.value.status == w.WAL_ERR_WORKSPACE
    with pytest.raises(w.WalError) as e:
        b.call(out=b.Q)
    assert e.value.status == w.WAL_ERR_ARG


# ---- waits, graphs, streams ----------------------------------------------------------------

@pytest.mark.parametrize("polls", POLLS)
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n,own", [(1, 30), (40, 900)])
def test_waits_that_run_out(n, own, typ, polls):
    """The prefix's launch (and, for chunks, the other) gives up: its rows are NaN or right, and the next call is clean."""
    b = Batch([(700, [(n, own)] * 6)], typ=typ, D=64, lead=0, trail=0, page=64)
    out = torch.empty(b.T, 8 * 64, dtype=torch.bfloat16, device="cuda")

    def call(ws):
        b.cache.attend_shared(b.Q[:, :512].contiguous(), out=out, ws=ws, **b.args, **b.bounds)
    check_timeout(call, out, b.ws(), 64, polls)


@pytest.mark.parametrize("n", [1, 25])
def test_in_a_graph(n):
    """Captured calls read lengths, groups and pages anew, and share a workspace in turn; calls on two streams do not."""
    b = Batch([(2000, [(n, n + 30)] * 5), (300, [(n, n + 70)] * 3)], page=64, typ="int8")
    b.bounds["max_own"] = 3000
    ws = b.ws()
    out, out2 = b.call(ws), b.call(ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(ws, out=out)
        b.call(ws, out=out2)
    for prefix, lens in (([2000, 300], b.lens), ([1984, 256], b.lens), ([64, 0], [v - 7 for v in b.lens])):
        b.args["prefix_len"].copy_(i32(prefix))
        b.args["kv_len"].copy_(i32(lens))
        b.args["table"].copy_(torch.from_numpy(np.where(b.table < 0, 0, b.table)).cuda())
        g.replay()
        ref = b.call(ws).view(torch.int16)  # some rows are NaN by slots that hold no token
        assert torch.equal(out.view(torch.int16), ref) and torch.equal(out2.view(torch.int16), ref)
    b.args["prefix_len"].copy_(i32(b.prefix)), b.args["kv_len"].copy_(i32(b.lens))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    spaces = b.ws(), b.ws()
    outs = [torch.full_like(out, SENTINEL) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        b.call(spaces[0], out=outs[0])
        b.call(spaces[1], out=outs[1], stream=side)
    torch.cuda.synchronize()
    b.check(outs[0])
    assert torch.equal(*outs)
