"""Non-finite values and the attention kernels: what they reach, and what they cost (needs a B200)."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao

from attn_util import TYPES, assert_close, attention_tolerance, bf16, random_cache
from gpu_util import needs_gpu, wal
from test_gpu_attention import i32, run_paged

pytestmark = [pytest.mark.gpu, needs_gpu]


def us(call):
    """Median time of a call, of five after two."""
    times = []
    for _ in range(7):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times[2:])[2]


def normal(*shape):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


# A row is right as it stands when it is NaN by something that it sees: it costs a look at the at most 256 keys behind
# its last one, or at the 256 rows of its piece, which is less than the piece itself took.
WITHIN = 4.0


@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_with_a_nonfinite_first_token_takes_no_longer(where, D):
    """Every row sees the bad value, so nearly every row is NaN, and rightly so."""
    w = wal()
    T, heads, kv = 4096, 8, 2
    t = dict(q=normal(T, heads * D), k=normal(T, kv * D), v=normal(T, kv * D))
    out, start = torch.empty_like(t["q"]), i32([0, T])
    call = lambda: w.attn_prompt(t["q"], t["k"], t["v"], start, out, head_dim=D, max_len=T)
    clean = us(call)
    t[where][:1 if where != "q" else T] = float("nan")
    took = us(call)
    assert torch.isnan(out).all()
    assert took <= WITHIN * clean, f"{took:.0f} us against {clean:.0f}"


def test_prompt_of_nan_takes_no_longer():
    w = wal()
    T, D = 4096, 64
    q, k, v, start = normal(T, 8 * D), normal(T, 2 * D), normal(T, 2 * D), i32([0, T])
    out = torch.empty_like(q)
    call = lambda: w.attn_prompt(q, k, v, start, out, head_dim=D, max_len=T)
    clean = us(call)
    for x in (q, k, v):
        x.fill_(float("nan"))
    took = us(call)
    assert torch.isnan(out).all()
    assert took <= WITHIN * clean, f"{took:.0f} us against {clean:.0f}"


def paged(n_q, lens, heads, kv_heads, D, typ, page=64):
    """(call, out, cache, table) over random pages; `heads` q heads of `n_q` new tokens each."""
    w = wal()
    width = -(-max(lens) // page)
    n = width * len(lens)
    if typ == "bf16":
        cache = w.KvCache(normal(n, kv_heads, page, D), normal(n, kv_heads, page, D))
    else:
        code = lambda: torch.randint(0, 100, (n, kv_heads, page, D), device="cuda", dtype=torch.uint8).view(TYPES[typ])
        cache = w.KvCache(code(), code(), *[torch.full((n, kv_heads, page), 0.01, device="cuda") for _ in range(2)])
    table = torch.arange(n, device="cuda", dtype=torch.int32).view(len(lens), width)
    q = normal(n_q * len(lens), heads * D)
    out = torch.empty_like(q)
    start = i32([n_q * b for b in range(len(lens) + 1)])
    kv_len = i32(lens)
    return lambda: cache.attend(q, start, kv_len, table, out, max_q=n_q, max_kv=max(lens)), out, cache, table


def splits(cache, heads, T, B, max_q, max_kv):
    n = cache.attend_workspace_bytes(heads, T, B, max_q, max_kv)
    return max(1, (n - 512) // (T * heads * (8 + 4 * cache.head_dim)))


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("n_q,B,L,heads,split", [(4, 1, 20000, 8, True), (4, 200, 100, 8, False), (300, 1, 4000, 4, True),
                                                 (600, 30, 700, 16, False)])
def test_chunk_with_a_nonfinite_first_token_takes_no_longer(n_q, B, L, heads, split, typ):
    call, out, cache, table = paged(n_q, [L] * B, heads, 2, 64, typ)
    assert (splits(cache, heads, n_q * B, B, n_q, L) > 1) == split
    clean = us(call)
    first = table[:, 0].long()
    if typ == "bf16":
        cache.v[first, :, 0] = float("nan")
    else:
        cache.v_scale[first, :, 0] = float("nan")
    took = us(call)
    assert torch.isnan(out).all()
    assert took <= WITHIN * clean, f"{took:.0f} us against {clean:.0f}"


@pytest.mark.parametrize("D", [64, 128])
def test_seen_and_hidden_columns_are_told_apart(D):
    """A NaN in one column of V that every row sees, and one in another column that
    only the last token sees: the others keep their values in that one."""
    w = wal()
    T, heads, kv = 700, 4, 2
    q, k, v = normal(T, heads * D), normal(T, kv * D), normal(T, kv * D)
    ref, out, start = torch.empty_like(q), torch.empty_like(q), i32([0, T])
    w.attn_prompt(q, k, v, start, ref, head_dim=D, max_len=T)
    v[0, 3] = float("nan")
    v[T - 1, 5] = float("inf")
    w.attn_prompt(q, k, v, start, out, head_dim=D, max_len=T)
    hit = torch.zeros(T, heads * D, dtype=torch.bool, device="cuda")
    hit[:, 3] = hit[:, D + 3] = True
    assert torch.isnan(out[hit]).all()
    hit[T - 1, 5] = hit[T - 1, D + 5] = True
    assert not torch.isfinite(out[hit]).any()
    # a row may be done again another way: the weights' rounding to bf16 (2^-8 of at most max |v| < 6), two of the output
    r, o = ref.float(), out.float()
    assert torch.all((o - r)[~hit].abs() <= 2.0 ** -7 * r[~hit].abs() + 6 * 2.0 ** -8)


# ---- keys split over CTAs --------------------------------------------------------

BAD = [("bf16", "v", float("nan")), ("bf16", "v", float("inf")), ("bf16", "v", -float("inf")), ("bf16", "k", float("nan")),
       ("bf16", "k", float("inf")), ("int8", "vs", float("nan")), ("int8", "ks", float("nan")), ("e4m3", "vs", float("nan")),
       ("e4m3", "ks", float("nan")), ("e4m3", "code", None)]


@pytest.mark.parametrize("typ,where,bad", BAD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q", [4, 40])
def test_nonfinite_last_keys_where_keys_are_split(n_q, D, typ, where, bad):
    """The last two tokens' K or V (or scales) are not finite.  The new tokens of each
    sequence lie on both sides of a multiple of 128, one of which every border
    between splits is, so that some rows see nothing of the last split.  Rows
    before those two tokens are as if they were not there."""
    w = wal()
    rng = np.random.default_rng(n_q + D)
    heads, kv_heads, page = 4, 1, 16
    lens = [128 * m + n_q // 2 for m in range(4, 24)]
    (k, v, ks, vs), table, kv, vv = random_cache(rng, lens, page, kv_heads, D, typ)
    for b, n in enumerate(lens):
        for j in (n - 2, n - 1):
            at = (table[b, j // page], slice(None), j % page)
            if where == "code":
                v.view(torch.uint8)[at] = 0x7F if j % 2 else 0xFF
            else:
                dict(k=k, v=v, ks=ks, vs=vs)[where][at] = bad
    cache = w.KvCache(*[None if t is None else t.cuda() for t in (k, v, ks, vs)])
    T, max_kv = n_q * len(lens), max(lens)
    q = bf16(rng.normal(size=(T, heads * D)))
    Q = torch.from_numpy(q).bfloat16().cuda()
    O = torch.full_like(Q, 77.0)
    assert splits(cache, heads, T, len(lens), n_q, max_kv) > 1
    cache.attend(Q, i32(range(0, T + 1, n_q)), i32(lens), torch.from_numpy(table).cuda(), O, max_q=n_q, max_kv=max_kv)
    got = O.cpu().double().numpy().reshape(len(lens), n_q, heads, D)
    for b, n in enumerate(lens):
        qb = q[n_q * b:n_q * (b + 1)].reshape(n_q, heads, D)[:n_q - 2]
        o, a = ao.attend(qb, kv[b][:n - 2], vv[b][:n - 2], D ** -0.5, heads)
        assert_close(got[b, :n_q - 2], o, attention_tolerance(o, a, qb, kv[b][:n - 2], D ** -0.5), f"sequence {b}")
        if where == "code":
            continue  # what the NaN codes read as is not specified
        if where == "v" and bad == bad:  # infinity, or NaN under a weight of zero
            assert not np.isfinite(got[b, n_q - 2:]).any()
        else:  # an infinite K meets q of both signs: inf - inf
            assert np.isnan(got[b, n_q - 2:]).all()


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_rows_that_see_an_infinite_key(bad, D):
    """All columns of one K are infinite and q has both signs: the score is inf - inf."""
    w = wal()
    T, heads, kv, j = 300, 4, 2, 150
    q, k, v = normal(T, heads * D), normal(T, kv * D), normal(T, kv * D)
    ref, out, start = torch.empty_like(q), torch.empty_like(q), i32([0, T])
    w.attn_prompt(q, k, v, start, ref, head_dim=D, max_len=T)
    k[j, :D] = bad
    w.attn_prompt(q, k, v, start, out, head_dim=D, max_len=T)
    hit = torch.zeros(T, heads * D, dtype=torch.bool, device="cuda")
    hit[j:, :2 * D] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], ref[~hit])


@pytest.mark.parametrize("scale", [0.0, -0.2])
@pytest.mark.parametrize("typ", ["int8", "e4m3"])
@pytest.mark.parametrize("n_q", [1, 4, 64])
def test_zero_and_negative_scales_over_codes(n_q, typ, scale):
    run_paged([90, 200], [n_q, n_q], 8, 2, 64, 32, typ, scale=scale, seed=n_q)
    run_paged([1500, 2600], [n_q, n_q], 8, 2, 128, 32, typ, scale=scale, seed=n_q + 1)
