"""A serving step's operators at the edges of what their header allows (needs a B200)."""
import pytest
import torch

from attn_util import TYPES
from gpu_util import needs_gpu, wal
from test_gpu_attention import SENTINEL, i32
from test_gpu_shared import Batch
from test_gpu_window import run_paged

pytestmark = [pytest.mark.gpu, needs_gpu]


def recorded(b, skip=(), ws=None, **change):
    """A call that records WAL_ERR_ARG, leaves the sequences of `skip` unwritten and answers the others; the next
    one with the same workspace is clean."""
    w = wal()
    ws = b.ws() if ws is None else ws
    O = b.call(ws, **change)
    with pytest.raises(w.WalError) as e:
        w.attention.status(ws)
    assert e.value.status == w.WAL_ERR_ARG
    b.check(O, skip=skip)
    b.check(b.call(ws))
    w.attention.status(ws)


# ---- shared calls: malformed groups ----------------------------------------------------

@pytest.mark.parametrize("typ", ["bf16", "int8"])
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("starts", [[0, 5, 3, 8], [0, 5, 5, 3, 8], [0, 8, 0, 8], [4, 3, 8, 8], [0, 4, 8, 7], [0, 8, 8, 8, 5, 8, 8], [3, 8, 8, 0]])
def test_group_starts_that_fall(starts, n, typ):
    """Nobody knows whose the sequences between are, so all are left out, by every kernel: at 4 and at more than 16
    query rows a head, with neighbouring groups of different prefixes."""
    b = Batch([(500, [(n, n + 3), (n, n + 50), (1, 200)]), (96, [(1, 9), (1, 20), (n, n + 300), (n, n), (1, 700)])], D=64, typ=typ, seed=n)
    prefix = [500, 96, 32, 500, 0, 64][:len(starts) - 1]
    recorded(b, range(8), group_start=i32(starts), prefix_len=i32(prefix), max_own=b.bounds["max_kv"],
             ws=torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("n", [1, 30])
def test_sequences_behind_a_malformed_last_group(n):
    """They are in no group, whatever that one holds."""
    b = Batch([(100, [(n, n + 3), (n, n + 50)]), (64, [(1, 9), (n, n)])], alone=[(1, 40)], after=[(n, n + 33), (1, 1)], D=64)
    for bad in (-1, b.bounds["max_prefix"] + 1):
        recorded(b, [3, 4], prefix_len=i32([100, bad]))
    # one group, from -1 to 3: the sequences from 3 on share nothing, but what they hold behind a prefix of others is
    # not in their rows of the table
    b = Batch([(0, [(n, n + 3), (1, 50), (n, n)])], after=[(n, n + 33), (1, 1)], D=64)
    recorded(b, [0, 1, 2], group_start=i32([-1, 3]))


@pytest.mark.parametrize("n", [1, 30])
def test_malformed_groups_without_sequences(n):
    """Nothing is left out, and they are recorded."""
    b = Batch([(100, [(n, n + 3), (n, n + 50)]), (64, []), (32, [(1, 9), (n, n)]), (10, [])], alone=[(1, 40)], after=[(n, n + 33)], D=64)
    for at in (1, 3):
        for bad in (-1, b.bounds["max_prefix"] + 1):
            recorded(b, prefix_len=i32([100, 64, 32, 10][:at] + [bad] + [100, 64, 32, 10][at + 1:]))
    b = Batch([(0, []), (100, [(n, n + 3), (n, n + 50)]), (50, [])], D=64)
    recorded(b, group_start=i32([-1, 0, 2, 2]))
    recorded(b, group_start=i32([0, 0, 2, 3]))


# ---- shared calls: sequences that share nothing ---------------------------------------

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [1, 30])
def test_more_new_tokens_than_keys_without_a_prefix(n, typ):
    """As attend() answers them: the tokens before the first key see nothing and get zeros."""
    w = wal()
    b = Batch([(0, [(n + 4, 2), (3, 0), (1, 5)]), (100, [(n, n + 3), (1, 20)])], alone=[(n + 2, 1), (2, 0)], after=[(n + 9, n)], D=64, typ=typ)
    ws = b.ws()
    O = b.call(ws)
    w.attention.status(ws)
    b.check(O)
    ref = torch.full_like(O, SENTINEL)
    few = dict(q_start=b.args["q_start"][:6].contiguous(), kv_len=b.args["kv_len"][:5].contiguous(), table=b.args["table"][:5])
    b.cache.attend(b.Q[:, :512], out=ref[:, :512], max_q=b.bounds["max_q"], max_kv=b.bounds["max_kv"], **few)
    for seq, rows in ((0, n + 1), (1, 2), (2, n + 2), (3, 3)):
        at = slice(b.start[seq], b.start[seq] + rows)
        assert torch.all(O[at, :512] == 0) and torch.all(ref[at, :512] == 0)


@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("held", [0, 40, 100])
def test_idle_sequences_of_a_group(held, n):
    """A finished request that stays in its place, with less than the shared tokens or none: nothing to answer or record."""
    w = wal()
    b = Batch([(100, [(n, n + 3), (0, 7), (1, 50), (0, 0)]), (64, [(0, 20), (n, n)])], D=64)
    lens = [held if q == 0 else v for q, v in zip(b.n_q, b.lens)]
    ws = b.ws()
    O = b.call(ws, kv_len=i32(lens))
    w.attention.status(ws)
    b.check(O)


def test_many_groups():
    """More than a warp's probes squared; one out of range and one that falls among them."""
    w = wal()
    groups = [(3 + g % 40, [(1, 1 + g % 7)] * (g % 3)) for g in range(1500)]
    b = Batch(groups, alone=[(1, 9)], after=[(1, 4)], heads=2, kv_heads=1, D=64, page=16)
    ws = b.ws()
    O = b.call(ws)
    w.attention.status(ws)
    b.check(O)
    for g in (1023, 1499):
        recorded(b, range(b.starts[g], b.starts[g + 1]), ws, prefix_len=i32(b.prefix[:g] + [-1] + b.prefix[g + 1:]))
        recorded(b, range(len(b.lens)), ws, group_start=i32(b.starts[:g] + [b.starts[g + 1] + 1] + b.starts[g + 1:]))


# ---- windows ---------------------------------------------------------------------------

@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("window", [50, 4999, 5000, 100000])
def test_pages_of_idle_sequences_may_be_gone(window, n, typ):
    """A sequence without new tokens sees no page, with a window shorter than its context or not."""
    run_paged([5000, 3000, 700], [n, 0, n], window, 0, typ=typ, seed=window)
    run_paged([5000, 3000, 700], [n, 0, n], window, 5000, typ=typ, seed=window)
