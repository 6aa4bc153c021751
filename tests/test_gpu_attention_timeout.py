"""Device waits of the attention kernels that run out (needs a B200).

The failure is made on the host: wal_debug_wait_polls limits the polls of every
wait.  With none, each wait gives up at once; with a few, wherever the data is
not there yet.  The call must end by itself, report WAL_ERR_TIMEOUT, leave NaN
in the rows it has no result for, and leave the context usable.  No GPU fault,
trap or endless wait is involved.
"""
import time

import pytest
import torch

from attn_util import TYPES
from gpu_util import needs_gpu, wal
from test_gpu_attention import i32
from test_gpu_attention_nonfinite import normal, splits

pytestmark = [pytest.mark.gpu, needs_gpu]

SENTINEL = 77.0


def recorded(ws):
    w = wal()
    try:
        w.attention.status(ws)
        return w.WAL_OK
    except w.WalError as e:
        return e.status


def check(call, out, ws, head_dim, polls, loses=True):
    """`call(ws)` writes every row of `out`: with that many polls, with a workspace and without, then as usual."""
    w = wal()
    rows = lambda: out.clone().view(-1, head_dim)
    call(ws)
    assert recorded(ws) == w.WAL_OK
    clean = rows()
    assert torch.isfinite(clean).all()
    for scratch in (ws, None):
        out.fill_(SENTINEL)
        torch.cuda.synchronize()
        before = w.wal_debug_wait_polls(polls)
        try:
            t0 = time.perf_counter()
            call(scratch)
            torch.cuda.synchronize()
            took = time.perf_counter() - t0
        finally:
            w.wal_debug_wait_polls(before)
        assert before == -1 and took < 1.0, f"the call took {took:.1f} s to give up"
        got = rows()
        lost = torch.isnan(got).all(-1)
        assert torch.equal(got[~lost], clean[~lost]), "a row is neither right nor NaN"
        if scratch is not None:
            status = recorded(ws)
            assert status in (w.WAL_OK, w.WAL_ERR_TIMEOUT)
            assert (status == w.WAL_ERR_TIMEOUT) or not lost.any()
            assert status == w.WAL_ERR_TIMEOUT or polls > 0 or not loses
        if polls == 0 and loses:
            assert lost.all()
    call(ws)
    assert recorded(ws) == w.WAL_OK and torch.equal(rows(), clean), "the call after it"


POLLS = [0, 1, 2, 5, 30]


@pytest.mark.parametrize("polls", POLLS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[3000], [1], [128, 40, 500, 1, 129, 256]])
def test_prompt(lens, D, polls):
    w = wal()
    T = sum(lens)
    q, k, v = normal(T, 8 * D), normal(T, 2 * D), normal(T, 2 * D)
    out, start = torch.empty_like(q), i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    check(lambda ws: w.attn_prompt(q, k, v, start, out, head_dim=D, max_len=max(lens), ws=ws), out, ws, D, polls)


def paged(typ, D, n_q, lens, page=32):
    """(call, out, workspace, splits, table) of a chunk, 8 q heads on 2."""
    w = wal()
    width, B, T = -(-max(lens) // page), len(lens), sum(n_q)
    shape = (width * B, 2, page, D)
    if typ == "bf16":
        cache = w.KvCache(normal(*shape), normal(*shape))
    else:
        code = lambda: torch.randint(0, 100, shape, device="cuda", dtype=torch.uint8).view(TYPES[typ])
        cache = w.KvCache(code(), code(), *[torch.full(shape[:3], 0.01, device="cuda") for _ in range(2)])
    table = torch.randperm(width * B, device="cuda").int().view(B, width)
    q = normal(T, 8 * D)
    out = torch.empty_like(q)
    start, kv_len = i32([sum(n_q[:i]) for i in range(B + 1)]), i32(lens)
    shape = (8, T, B, max(n_q), max(lens))
    ws = torch.empty(cache.attend_workspace_bytes(*shape), dtype=torch.uint8, device="cuda")
    call = lambda ws: cache.attend(q, start, kv_len, table, out, max_q=max(n_q), max_kv=max(lens), ws=ws)
    return call, out, ws, splits(cache, *shape), table


@pytest.mark.parametrize("polls", POLLS)
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q,lens,split", [([40, 9], [3000, 2500], True), ([600] * 30, [700] * 30, False), ([100, 20, 5], [120, 90, 60], False)])
def test_chunk(n_q, lens, split, D, typ, polls):
    call, out, ws, n, _ = paged(typ, D, n_q, lens)
    assert (n > 1) == split
    check(call, out, ws, D, polls)


@pytest.mark.parametrize("lens", [[3000, 2500], [100, 90]])
def test_a_timeout_outlives_a_bad_index(lens):
    """Both happen: the lost rows are what the status word tells of."""
    w = wal()
    call, out, ws, n, table = paged("bf16", 64, [40, 9], lens)
    assert (n > 1) == (max(lens) > 1000)
    table[1, 1] = -5
    call(ws)
    assert recorded(ws) == w.WAL_ERR_ARG
    w.wal_debug_wait_polls(0)
    try:
        call(ws)
        torch.cuda.synchronize()
    finally:
        w.wal_debug_wait_polls(-1)
    assert recorded(ws) == w.WAL_ERR_TIMEOUT


def test_single_tokens_have_no_such_waits():
    call, out, ws, _, _ = paged("int8", 128, [1, 1], [3000, 70])
    check(call, out, ws, 128, 0, loses=False)
