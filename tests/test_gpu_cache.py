"""Rotary positions and the paged cache (append, read back) vs the FP64 oracle (needs a B200)."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao

from attn_util import TYPES, bf16, pages_of
from gpu_util import needs_gpu, wal

pytestmark = [pytest.mark.gpu, needs_gpu]

F32 = 2.0 ** -24
SCALINGS = {"none": {}, "linear": dict(scaling="linear", factor=8.0),
            "parts": dict(scaling="parts", factor=4.0, original_len=4096.0, slow=1.0, fast=32.0)}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def turn_error(x, rot, mscale, layout):
    """Bound of the fp32 error of a rotated element: the angle is rounded to
    fp32 in half turns (at most pi 2^-24 radians), sincospif is good to 2 ulp
    and three products and a sum round: 2^-21 of |x1| + |x2| covers the sum."""
    e = np.zeros_like(x)
    n = rot // 2
    for i in range(n):
        lo, hi = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        e[..., lo] = e[..., hi] = (np.abs(x[..., lo]) + np.abs(x[..., hi])) * mscale * 2.0 ** -21
    return e


@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 64), (64, 16), (96, 32), (256, 256), (80, 80)])
@pytest.mark.parametrize("scaling", list(SCALINGS))
def test_rope(inp, layout, D, rot, scaling):
    w = wal()
    rng = np.random.default_rng(D + rot)
    T, heads, pad = 37, 5, 8
    x = rng.normal(size=(T, heads * D)) * np.exp(rng.normal(size=(T, 1)) * 3)
    X = torch.full((T, heads * D + pad), float("nan"), dtype=inp)
    X[:, :heads * D] = torch.from_numpy(x).to(inp)
    x = X[:, :heads * D].double().numpy().reshape(T, heads, D)
    pos = np.concatenate([[0, 1, 131071, 2 ** 31 - 1, -1, -5000, 2 ** 24 + 1], rng.integers(0, 40000, T - 7)]).astype(np.int32)
    Y = torch.full((T, heads * D + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    rope = w.Rope(D, rot, base=1e6, layout=layout, **SCALINGS[scaling])
    rope.apply(X.cuda()[:, :heads * D], torch.from_numpy(pos).cuda(), Y[:, :heads * D])
    got = Y.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == 5.0)
    f, m = ao.rope_freqs(rot, base=1e6, **SCALINGS[scaling])
    ref = ao.rotate(x, pos, f, m, layout)
    # the oracle's own angle p f is rounded to 2^-53 of itself, its f to a few 2^-53
    far = np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -50
    err = turn_error(x, rot, m, layout)
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * err + far * err * 2.0 ** 21
    assert np.all(np.abs(got[:, :heads * D].reshape(T, heads, D) - ref) <= tol)
    if inp == torch.bfloat16:  # in place
        Z = X[:, :heads * D].cuda().contiguous()
        rope.apply(Z, torch.from_numpy(pos).cuda(), Z)
        assert torch.equal(Z, Y[:, :heads * D])


def test_rope_one_row_and_none():
    w = wal()
    rope = w.Rope(64)
    for T in (0, 1):
        x = torch.ones(T, 64, device="cuda")
        y = torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
        rope.apply(x, torch.zeros(T, dtype=torch.int32, device="cuda"), y)
        assert torch.equal(y, torch.ones_like(y))


def raw(t):
    """Codes of an 8-bit tensor as float64 values."""
    t = t.cpu()
    return t.double().numpy() if t.dtype != torch.float8_e4m3fn else ao.e4m3_values(t.view(torch.uint8).numpy())


@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("heads,D,page,T,rot", [(8, 128, 16, 25, 128), (1, 64, 256, 1, 0), (5, 64, 32, 300, 32),
                                                (40, 128, 64, 9, 0), (3, 128, 128, 130, 64)])
def test_append(inp, typ, heads, D, page, T, rot):
    w = wal()
    rng = np.random.default_rng(T)
    n_pages = -(-T // page) + 3
    cache = w.KvCache.empty(n_pages, page, heads, D, dtype=TYPES[typ])
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x33)
    for t in (cache.k_scale, cache.v_scale):
        if t is not None:
            t.fill_(9.0)
    x = []
    for _ in range(2):
        y = rng.normal(size=(T, heads, D)) * np.exp(rng.normal(size=(T, heads, 1)) * 4)
        y[T // 2, 0] = 0.0
        y[0, heads - 1] = 1e-41 if inp == torch.float32 else 2.0 ** -130  # subnormal rows
        X = torch.full((T, heads * D + 8), float("nan"), dtype=inp)
        X[:, :heads * D] = torch.from_numpy(y.reshape(T, -1)).to(inp)
        x.append(X)
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    skip = np.zeros(T, bool)
    if T > 2:
        skip[1] = True
    pos = rng.integers(0, 30000, T).astype(np.int32)
    rope = w.Rope(D, rot, base=1e6) if rot else None
    used = np.where(skip, -1, slots).astype(np.int32)
    ws = torch.full((512,), 0xFF, dtype=torch.uint8, device="cuda")
    cache.append(x[0].cuda()[:, :heads * D], x[1].cuda()[:, :heads * D], torch.from_numpy(used).cuda(),
                 positions=torch.from_numpy(pos).cuda() if rot else None, rope=rope, ws=ws)
    w.attention.status(ws)
    live = ~skip
    for which, (X, codes, scale) in enumerate(zip(x, (cache.k, cache.v), (cache.k_scale, cache.v_scale))):
        val = X[:, :heads * D].double().numpy().reshape(T, heads, D)
        err = np.zeros_like(val)
        if rot and which == 0:
            f, m = ao.rope_freqs(rot, base=1e6)
            err = turn_error(val, rot, m, "half")
            val = ao.rotate(val, pos, f, m)
        at = (slots[live] // page, slice(None), slots[live] % page)
        got = raw(codes)[at]
        val, err = val[live], err[live]
        if typ == "bf16":
            assert np.all(np.abs(got - val) <= 2.0 ** -8 * np.abs(val) + 1.01 * err + 2.0 ** -134)
        else:
            sc = scale.cpu().numpy()[at].astype(np.float64)
            ref = ao.scales(val, typ)
            # the division rounds once; 2^-150: half the smallest fp32 step
            assert np.all(np.abs(sc - ref) <= ref * 1.01 * F32 + err.max(-1) / ao.QMAX[typ] + 2.0 ** -150)
            y = val / sc[..., None]
            # half a step of the code's own grid, the quotient's rounding, the rotation's error
            tol = ao.step(y, typ) / 2 * (1 + 1e-12) + np.abs(y) * 1.01 * F32 + 1.01 * err / sc[..., None]
            assert np.all(np.abs(got - y) <= tol)
            assert np.all(np.abs(got) <= ao.QMAX[typ])
            if not rot or which == 1:  # the same operations in fp32: the same codes, ties to even
                q = (X[live][:, :heads * D].float().view(-1, heads, D) / torch.from_numpy(sc).float()[..., None])
                same = q.round() if typ == "int8" else q.to(torch.float8_e4m3fn).float()
                assert np.array_equal(same.double().numpy(), got)
        # nothing else was written
        untouched = np.ones((n_pages, page), bool)
        untouched[slots[live] // page, slots[live] % page] = False
        b = codes.view(torch.uint8).cpu().numpy().reshape(n_pages, heads, page, -1).transpose(0, 2, 1, 3)
        assert np.all(b[untouched] == 0x33)
        if scale is not None:
            assert np.all(scale.cpu().numpy().transpose(0, 2, 1)[untouched] == 9.0)


@pytest.mark.parametrize("typ", ["int8", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_append_nonfinite_row_reads_back_as_nan(typ, bad):
    w = wal()
    cache = w.KvCache.empty(2, 16, 2, 64, dtype=TYPES[typ])
    x = torch.randn(4, 128, device="cuda")
    x[2, 70] = bad
    cache.append(x, x, i32([3, 4, 5, 6]))
    k, v = (torch.empty(7, 128, device="cuda") for _ in range(2))
    cache.read(i32([[0]]), i32([0, 7]), k, v, max_len=7)
    assert torch.isnan(k[5, 64:]).all() and torch.isnan(v[5, 64:]).all()
    assert torch.isfinite(k[[3, 4, 6]]).all() and torch.isfinite(k[5, :64]).all()


def test_append_bad_slots():
    w = wal()
    cache = w.KvCache.empty(2, 16, 1, 64)
    cache.k.zero_()
    cache.v.zero_()
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    x = torch.ones(6, 64, device="cuda")
    for slot in (32, -2, 2 ** 31 - 1, -2 ** 31):
        cache.append(x, x, i32([0, slot, -1, 5, 31, 7]), ws=ws)
        with pytest.raises(w.WalError) as e:
            w.attention.status(ws)
        assert e.value.status == w.WAL_ERR_ARG
    on = cache.k.float().sum(-1)[:, 0].reshape(-1) > 0
    assert on.nonzero().flatten().tolist() == [0, 5, 7, 31]
    cache.append(x[:1], x[:1], i32([-1]), ws=ws)
    w.attention.status(ws)  # a padded row alone is no error


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("heads,D,page", [(8, 128, 16), (1, 64, 256), (5, 128, 64)])
def test_read(heads, D, page, typ, out):
    from attn_util import random_cache
    w = wal()
    rng = np.random.default_rng(page)
    lens = [1, 0, 3 * page + 7, page, 15]
    tensors, table, ks, vs = random_cache(rng, lens, page, heads, D, typ)
    cache = w.KvCache(*[None if t is None else t.cuda() for t in tensors])
    start = 2 + np.concatenate([[0], np.cumsum(lens)])
    T = int(start[-1]) + 3
    K, V = (torch.full((T, heads * D + 8), 3.0, dtype=out, device="cuda") for _ in range(2))
    ws = torch.full((512,), 0xFF, dtype=torch.uint8, device="cuda")
    cache.read(torch.from_numpy(table).cuda(), i32(start), K[:, :heads * D], V[:, :heads * D], max_len=max(lens), ws=ws)
    w.attention.status(ws)
    for got, seqs in ((K, ks), (V, vs)):
        got = got.cpu().double().numpy()
        assert np.all(got[:, heads * D:] == 3.0) and np.all(got[:2] == 3.0) and np.all(got[T - 3:] == 3.0)
        ref = np.concatenate(seqs).reshape(-1, heads * D)
        # a code times an fp32 scale: one rounding to fp32, then one to bf16
        tol = np.abs(ref) * (F32 * 1.01 + (2.0 ** -8 if out == torch.bfloat16 else 0))
        assert np.all(np.abs(got[2:T - 3, :heads * D] - ref) <= tol)
    for page_id in (-1, cache.n_pages, 2 ** 31 - 1):
        bad = table.copy()
        bad[2, 1] = page_id
        K.fill_(3.0)
        cache.read(torch.from_numpy(bad).cuda(), i32(start), K[:, :heads * D], V[:, :heads * D], max_len=max(lens), ws=ws)
        with pytest.raises(w.WalError):
            w.attention.status(ws)
        rows = slice(int(start[2]) + page, int(start[2]) + 2 * page)
        assert not K[rows, :heads * D].any() and K[int(start[2]):rows.start, :heads * D].any()
    for starts in ([0, 1, 1, T + 1, T, T], [-1, 1, 1, 2, 3, 4], [5, 1, 1, 2, 3, 4], [0, 0, 0, 0, 0, max(lens) + 1]):
        cache.read(torch.from_numpy(table).cuda(), i32(starts), K[:, :heads * D], V[:, :heads * D], max_len=max(lens), ws=ws)
        with pytest.raises(w.WalError) as e:
            w.attention.status(ws)
        assert e.value.status == w.WAL_ERR_ARG


def test_append_in_graph_takes_new_slots():
    w = wal()
    cache = w.KvCache.empty(4, 16, 2, 64, dtype=torch.int8)
    rope = w.Rope(64)
    x, slots, pos = torch.randn(3, 128, device="cuda"), i32([0, 1, 2]), i32([0, 1, 2])
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    call = lambda: cache.append(x, x, slots, positions=pos, rope=rope, ws=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    first = cache.k[0, :, :3].clone()
    slots.copy_(i32([40, 41, -1]))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.k[2, :, 8:10], first[:, :2])


def test_other_device_values_and_streams():
    """Tensors used on a stream that is not current."""
    w = wal()
    s = torch.cuda.Stream()
    cache = w.KvCache.empty(4, 16, 2, 64)
    x = torch.randn(20, 128, device="cuda")
    torch.cuda.synchronize()
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    cache.append(x, x, slots, stream=s)
    k, v = (torch.empty(20, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(i32([[0, 1]]), i32([0, 20]), k, v, max_len=20, stream=s)
    s.synchronize()
    assert torch.equal(k, x.bfloat16()) and torch.equal(v, x.bfloat16())


@pytest.mark.parametrize("typ", list(TYPES))
def test_reading_one_half_moves_one_half(typ):
    """With a NULL K or V the other one is read as ever, in half the time."""
    w = wal()
    B, L, heads, D, page = 96, 4096, 8, 128, 64
    cache = w.KvCache.empty(B * L // page, page, heads, D, dtype=TYPES[typ])
    for t in (cache.k, cache.v):
        t.view(torch.uint8).random_(0, 0x40)
    for t in (cache.k_scale, cache.v_scale):
        if t is not None:
            t.uniform_(0.5, 1.5)
    table = torch.randperm(B * L // page, device="cuda").int().view(B, -1)
    start = i32([L * b for b in range(B + 1)])
    K, V, out = (torch.full((B * L, heads * D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    s = torch.cuda.current_stream().cuda_stream

    def read(k, v):
        ptr = lambda x: None if x is None else x.data_ptr()
        w.wal_kv_read(cache.desc, table.data_ptr(), table.shape[1], start.data_ptr(), B, L, ptr(k), ptr(v), w.WAL_BF16, B * L,
                      heads * D, heads * D, None, 0, s)

    def us(*args):
        times = []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            read(*args)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[4]

    both = us(K, V)
    # bytes in and out, of 8 (bf16) or 6 with both: 4 or 3 without the other half's, 6 or 4 with its reads
    limit = 0.625 * both
    for ref, args in ((K, (out, None)), (V, (None, out))):
        out.fill_(3.0)
        took = us(*args)
        assert torch.equal(out, ref)
        assert took <= limit, f"{took * 1e3:.0f} us against {both * 1e3:.0f} for both"
