"""The plan of a step, and norms of q and k heads with the rotation and the cache, vs the oracle (needs a B200)."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao, step_oracle as so

from attn_util import TYPES
from gpu_util import needs_gpu, wal
from test_gpu_cache import raw, turn_error

pytestmark = [pytest.mark.gpu, needs_gpu]


def dev(x):
    return torch.from_numpy(np.array(x, np.int32)).cuda()


class Plan:
    """A cache's sequences and free list on the host and, by `step`, on the device."""

    def __init__(self, rng, page, n_pages, B, width):
        w = wal()
        self.rng, self.page, self.n_pages, self.B, self.width = rng, page, n_pages, B, width
        self.cache = w.KvCache.empty(n_pages, page, 1, 64)
        self.table, self.lens = np.full((B, width), -1), np.zeros(B, int)
        self.free, self.n_free = rng.permutation(n_pages), n_pages

    def device(self, ld=None):
        ld = ld or self.width
        wide = torch.full((self.B, ld), -77, dtype=torch.int32, device="cuda")
        wide[:, :self.width] = dev(self.table)
        return dict(kv_len=dev(self.lens), table=wide[:, :self.width], free=dev(self.free), n_free=dev([self.n_free])), wide

    def step(self, new, T, in_place, ld=None, max_kv=None, status=None):
        w = wal()
        s, wide = self.device(ld)
        out = dict(q_start=dev([-5] * (self.B + 1)), positions=dev([-5] * T), slots=dev([-5] * T))
        ws = torch.full((512,), 255, dtype=torch.uint8, device="cuda")
        after = {} if in_place else dict(kv_len_out=dev([-5] * self.B), n_free_out=dev([-5]))
        self.cache.plan(dev(new), **s, **out, **after, max_kv=max_kv, ws=ws)
        ref = so.plan(list(new), self.lens.tolist(), self.table, self.free, self.n_free, T, self.page, self.n_pages,
                      max_kv or self.width * self.page)
        got = dict(out, table=s["table"], free=s["free"], kv_len=after.get("kv_len_out", s["kv_len"]), n_free=after.get("n_free_out", s["n_free"]))
        for name, want in ref.items():
            if name != "bad":
                assert np.array_equal(got[name].cpu().numpy().reshape(-1), np.reshape(want, -1)), name
        if not in_place:
            assert np.array_equal(s["kv_len"].cpu().numpy(), self.lens) and int(s["n_free"]) == self.n_free
        assert (wide[:, self.width:] == -77).all()
        if ref["bad"]:
            with pytest.raises(w.WalError) as e:
                w.attention.status(ws)
            assert e.value.status == w.WAL_ERR_ARG
        else:
            w.attention.status(ws)
        assert status is None or status == ref["bad"]
        self.table, self.lens, self.free, self.n_free = ref["table"], ref["kv_len"], ref["free"], ref["n_free"]


@pytest.mark.parametrize("page,B,width,most,T", [(16, 1, 4, 40, 64), (16, 3, 9, 60, 180), (64, 25, 20, 3, 75), (32, 300, 6, 50, 16000),
                                                 (256, 33, 3, 700, 9000), (16, 1024, 12, 9, 8192), (16, 1025, 12, 9, 8192), (32, 2500, 5, 40, 50001)])
def test_plan_steps(page, B, width, most, T):
    """Steps of growth, drops and ends from empty tables on, until pages or rows run short."""
    rng = np.random.default_rng(B)
    p = Plan(rng, page, max(4, B * width * 3 // 4), B, width)
    for i in range(8):
        new = rng.integers(0, most + 1, B)
        if i:
            drop = rng.random(B) < 0.3
            new = np.where(drop, -np.minimum(p.lens, rng.integers(0, most + 1, B)), new)
            new = np.where(rng.random(B) < 0.1, -p.lens, new)
        if i < 6:  # within the table
            new = np.minimum(new, width * page - p.lens)
        p.step(new, T, in_place=i % 2 == 0, ld=None if i % 3 else width + 5)


def test_plan_of_one_prompt():
    p = Plan(np.random.default_rng(0), 16, 3000, 1, 2500)
    p.step([33333], 40000, True, status=False)
    p.step([-33333], 3, False, status=False)
    p.step([16 * 2500 + 1], 1 << 17, False, status=True)
    p.step([16 * 2500], 1 << 17, False, status=False)
    p.step([0], 0, False, status=False)


def test_plan_of_many_sequences():
    rng = np.random.default_rng(5)
    p = Plan(rng, 16, 60000, 65535, 2)
    p.step(rng.integers(0, 4, 65535), 1 << 18, False)
    p.step(np.where(rng.random(65535) < 0.5, -p.lens, 20), 1 << 20, False)
    p.step(rng.integers(0, 3, 65535), 100, True, status=True)


@pytest.mark.parametrize("B", [6, 2000])
def test_plan_reports(B):
    """Values and ids out of range, a list that is not one, and shortages."""
    rng = np.random.default_rng(1)
    one = np.ones(B, int)

    def fresh():
        p = Plan(rng, 16, 4 * B, B, 3)
        p.step(rng.integers(1, 20, B), 30 * B, True, status=False)
        return p
    for change in (dict(lens=-1), dict(lens=49), dict(new=100), dict(new=-60), dict(new=2 ** 31 - 1), dict(new=-2 ** 31), dict(lens=2 ** 31 - 1)):
        p, new = fresh(), one.copy()
        if "lens" in change:
            p.lens[2] = change["lens"]
        else:
            new[2] = change["new"]
        p.step(new, 5 * B, False, status=True)
    for n_free in (-1, 4 * B + 1, 2 ** 31 - 1):
        p = fresh()
        p.n_free = n_free
        p.step(one, 5 * B, False, status=True)
    p = fresh()
    p.n_free = 4 * B - 1  # the given pages would not fit
    p.step(-p.lens, 5 * B, False, status=True)
    p = fresh()
    p.step(one, B // 2, False, status=True)
    p = fresh()
    p.n_free = 2
    p.step(one * 16, 16 * B, False, status=True)
    p = fresh()
    p.table[1, 0] = 4 * B
    p.lens[1] = 5
    p.step(one, B, False, status=True)
    p = fresh()
    p.table[1, 0], p.lens[1] = -3, 5
    p.step(np.where(np.arange(B) == 1, -5, 1), B, False, status=True)
    p = fresh()
    p.free[p.n_free - 1] = -2
    p.lens[0], p.lens[1:] = 16, 1
    p.step(one, B, False, status=True)
    p = fresh()
    p.lens[0] = 20
    p.step(one, B, False, max_kv=20, status=True)


@pytest.mark.parametrize("B,T", [(7, 9), (1500, 1600)])
def test_plan_in_a_graph(B, T):
    """A captured step in place: each replay goes on from the one before."""
    rng = np.random.default_rng(2)
    p = Plan(rng, 16, 6 * B, B, 8)
    p.step(rng.integers(0, 30, B), 30 * B, False, status=False)
    s, _ = p.device()
    new, out = dev([1] * B), dict(q_start=dev([0] * (B + 1)), positions=dev([0] * T), slots=dev([0] * T))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p.cache.plan(new, **s, **out)
    for step in range(40):
        n = rng.integers(-1, 3, B)
        n = np.maximum(n, -p.lens) if step % 2 else np.ones(B, int)
        n[np.cumsum(np.maximum(n, 0)) > T] = 0
        new.copy_(dev(n))
        g.replay()
        ref = so.plan(n.tolist(), p.lens.tolist(), p.table, p.free, p.n_free, T, p.page, p.n_pages, p.width * p.page)
        assert not ref["bad"]
        p.table, p.lens, p.free, p.n_free = ref["table"], ref["kv_len"], ref["free"], ref["n_free"]
    for name, want in ref.items():
        if name != "bad":
            assert np.array_equal({**s, **out}[name].cpu().numpy().reshape(-1), np.reshape(want, -1)), name


# ---- norms, rotation, cache -----------------------------------------------------------

def rows(rng, T, heads, D, inp, pad=0):
    """Head rows of very different sizes, in a wider buffer whose rest is NaN: (device view, float64 values)."""
    x = rng.normal(size=(T, heads, D)) * np.exp(rng.normal(size=(T, heads, 1)) * 3)
    X = torch.full((T, heads * D + pad), float("nan"), dtype=inp)
    X[:, :heads * D] = torch.from_numpy(x.reshape(T, -1)).to(inp)
    return X.cuda()[:, :heads * D], X[:, :heads * D].double().numpy().reshape(T, heads, D)


def weights(rng, D, typ):
    w = [torch.from_numpy(rng.normal(size=D)).to(typ) for _ in range(2)]
    return [x.cuda() for x in w], [x.double().numpy() for x in w]


def norm_error(y, D):
    """Bound of the fp32 error of a normalised element y: the sum of D squares (each with a product's and at most
    D / 16 + 16 sums' roundings, halved by the root), rsqrt (2 ulp), 1 / D, two products."""
    return np.abs(y) * ((D / 16 + 17) / 2 + 8) * 2.0 ** -24


def turned(x, pos, w, eps, D, rot, layout, scaling={}):
    """(values, error bound) of rotate(norm(x)) before the last rounding."""
    f, m = ao.rope_freqs(rot, base=1e6, **scaling) if rot else (np.zeros(0), 1.0)
    y = x if w is None else so.head_norm(x, w, eps)
    e = np.zeros_like(y) if w is None else norm_error(y, D)
    ref = ao.rotate(y, pos, f, m, layout)
    err = turn_error(y, rot, m, layout)
    far = np.abs(pos.astype(np.float64))[:, None, None] * 2.0 ** -50
    n = rot // 2  # an error of one element of a pair goes into both
    spread = e.copy()
    for i in range(n):
        lo, hi = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
        spread[..., lo] = spread[..., hi] = (e[..., lo] + e[..., hi]) * m
    return ref, 1.01 * (err + spread) + far * err * 2.0 ** 21


POS = np.array([0, 1, 131071, 2 ** 31 - 1, -1, -5000, 2 ** 24 + 1], np.int32)


@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("wt", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("layout,D,rot,heads,kv", [("half", 128, 128, 5, 1), ("interleaved", 128, 64, 4, 4), ("half", 64, 16, 7, 2),
                                                   ("interleaved", 96, 32, 3, 2), ("half", 256, 256, 2, 1), ("half", 80, 80, 3, 3), ("half", 16, 16, 9, 1)])
@pytest.mark.parametrize("T", [37, 700])
def test_qk_norm_rope(inp, wt, layout, D, rot, heads, kv, T):
    w = wal()
    rng = np.random.default_rng(D + rot + T)
    q, qv = rows(rng, T, heads, D, inp, 8)
    k, kvals = rows(rng, T, kv, D, inp, 16)
    pos = np.concatenate([POS, rng.integers(0, 40000, T - 7)]).astype(np.int32)
    eps = 1e-3
    norm, vals = None, [None, None]
    if wt is not None:
        dw, vals = weights(rng, D, wt)
        norm = w.HeadNorm(*dw, eps=eps)
    outs = [torch.full((T, n * D + 24), 5.0, dtype=torch.bfloat16, device="cuda") for n in (heads, kv)]
    rope = w.Rope(D, rot, base=1e6, layout=layout)
    rope.apply_qk(q, k, dev(pos), outs[0][:, :heads * D], outs[1][:, :kv * D], norm=norm)
    for out, x, wv, n in zip(outs, (qv, kvals), vals, (heads, kv)):
        got = out.cpu().double().numpy()
        assert np.all(got[:, n * D:] == 5.0)
        ref, err = turned(x, pos, wv, norm and np.float32(eps), D, rot, layout)
        assert np.all(np.abs(got[:, :n * D].reshape(ref.shape) - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)
    if norm is None:  # the rotation alone is the other entry point's
        y = torch.empty_like(outs[0])[:, :heads * D]
        rope.apply(q, dev(pos), y)
        assert torch.equal(y, outs[0][:, :heads * D])
    if inp == torch.bfloat16:  # in place
        zq, zk = q.contiguous(), k.contiguous()
        rope.apply_qk(zq, zk, dev(pos), zq, zk, norm=norm)
        assert torch.equal(zq, outs[0][:, :heads * D]) and torch.equal(zk, outs[1][:, :kv * D])


@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("heads,kv,D,page,T,rot,layout", [(32, 8, 128, 16, 25, 128, "half"), (1, 1, 64, 256, 1, 0, "half"), (10, 5, 64, 32, 700, 32, "interleaved"),
                                                          (3, 40, 128, 64, 9, 0, "half"), (6, 3, 128, 128, 130, 64, "half")])
@pytest.mark.parametrize("normed", [True, False])
def test_qkv_append(inp, typ, heads, kv, D, page, T, rot, layout, normed):
    w = wal()
    rng = np.random.default_rng(T + kv)
    n_pages = -(-T // page) + 3
    make = lambda: w.KvCache.empty(n_pages, page, kv, D, dtype=TYPES[typ])
    cache, other = make(), make()
    for c in (cache, other):
        for t in (c.k, c.v):
            t.view(torch.uint8).fill_(0x55)
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.fill_(0.125)
    x, xv = rows(rng, T, heads + 2 * kv, D, inp, 8)  # one buffer for q, k and v
    split = lambda t, f: (t[:, :heads * f], t[:, heads * f:(heads + kv) * f], t[:, (heads + kv) * f:])
    q, k, v = split(x, D)
    qv, kvals, vv = split(xv, 1)
    pos = np.resize(np.concatenate([POS, rng.integers(0, 40000, T)]), T).astype(np.int32)
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.2] = -1
    norm, vals, eps = None, [None, None], 1e-6
    if normed:
        dw, vals = weights(rng, D, torch.bfloat16)
        norm = w.HeadNorm(*dw, eps=eps)
    rope = w.Rope(D, rot, base=1e6, layout=layout) if rot else None
    out = torch.full((T, heads * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((512,), 255, dtype=torch.uint8, device="cuda")
    cache.append_qkv(q, k, v, dev(slots), out[:, :heads * D], positions=dev(pos), rope=rope, norm=norm, ws=ws)
    w.attention.status(ws)
    ref, err = turned(qv, pos, vals[0], np.float32(eps), D, rot, layout)
    got = out.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == 5.0)
    assert np.all(np.abs(got[:, :heads * D].reshape(ref.shape) - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)
    # V, and K without a norm, are what append stores, bit for bit
    other.append(k, v, dev(slots), positions=dev(pos), rope=rope)
    for name in ("k", "v", "k_scale", "v_scale"):
        a, b = getattr(cache, name), getattr(other, name)
        if a is not None and (name[0] == "v" or not normed):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    # K: half a step of the code, the quotient's rounding, the errors before it
    live = slots >= 0
    at = (slots[live] // page, slice(None), slots[live] % page)
    ref, err = (t[live] for t in turned(kvals, pos, vals[1], np.float32(eps), D, rot, layout))
    codes = raw(cache.k)
    if typ == "bf16":
        assert np.all(np.abs(codes[at] - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)
    else:
        sc = cache.k_scale.cpu().double().numpy()[at]
        top, slack = np.abs(ref).max(-1), err.max(-1)
        assert np.all(np.abs(sc - top / ao.QMAX[typ]) <= (slack + top * 2.0 ** -23) / ao.QMAX[typ])
        grid = ao.step((np.abs(ref) + err) / sc[..., None], typ) * sc[..., None]
        assert np.all(np.abs(codes[at] * sc[..., None] - ref) <= grid / 2 + np.abs(ref) * 2.0 ** -22 + err)
    untouched = np.ones((n_pages, page), bool)
    untouched[at[0], at[2]] = False
    bytes_ = cache.k.view(torch.uint8).cpu().numpy().transpose(0, 2, 1, 3)[untouched]
    assert np.all(bytes_ == 0x55)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
def test_norm_of_extreme_rows(typ, inp):
    """Rows of zeros, of the largest and smallest sizes, and with an infinity or a NaN."""
    w = wal()
    D, sizes = 128, [0.0, 1e38, 1e25, 1e-25, 1e-38, 1.0, float("inf"), float("nan")]
    rng = np.random.default_rng(0)
    x = rng.normal(size=(len(sizes), 1, D)) / 4
    x[:, :, 3] = 0.0
    for i, s in enumerate(sizes):
        if np.isfinite(s):
            x[i] *= s
        else:
            x[i, 0, 3] = s
    X = torch.from_numpy(x.reshape(len(sizes), D)).to(inp)
    x = X.double().numpy().reshape(x.shape)
    X = X.cuda()
    dw, vals = weights(rng, D, torch.float32)
    cache = w.KvCache.empty(1, 16, 1, D, dtype=TYPES[typ])
    out = torch.empty(len(sizes), D, dtype=torch.bfloat16, device="cuda")
    cache.append_qkv(X, X, X, dev(range(len(sizes))), out, norm=w.HeadNorm(*dw, eps=1e-6))
    got = out.cpu().double().numpy()
    ref = so.head_norm(x[:6], vals[0], np.float32(1e-6))[:, 0]
    tiny = 2.0 ** -133  # of bf16, where the values run out
    assert np.all(np.abs(got[:6] - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * norm_error(ref, D) + tiny)
    assert np.isnan(got[6, 3]) and np.all(np.delete(got[6], 3) == 0) and np.isnan(got[7]).all()
    k, v = (t[0, 0, :8].float().cpu().double().numpy() for t in (cache.k, cache.v))
    if typ != "bf16":
        k, v = k * cache.k_scale[0, 0, :8].cpu().double().numpy()[:, None], v * cache.v_scale[0, 0, :8].cpu().double().numpy()[:, None]
    ref = so.head_norm(x[:6], vals[1], np.float32(1e-6))[:, 0]
    for got, ref in ((k[:6], ref), (v[:6], x[:6, 0])):
        half = {"bf16": 2.0 ** -8 * np.abs(ref), "int8": np.abs(ref).max(-1, keepdims=True) / 254 * 1.001,
                "e4m3": np.maximum(np.abs(ref) * 2.0 ** -4, np.abs(ref).max(-1, keepdims=True) / 448 * 2.0 ** -10) * 1.001}[typ]
        low = tiny if typ == "bf16" else 2.0 ** -126 / 2  # half a step of the smallest scale
        assert np.all(np.abs(got - ref) <= half + 1.01 * norm_error(ref, D) + low)
    assert np.isnan(k[6:]).any(-1).all() and (typ == "bf16" or (np.isnan(k[6:]).all() and np.isnan(v[6:]).all()))


def test_qkv_append_reports():
    w = wal()
    cache = w.KvCache.empty(2, 16, 1, 64)
    x = torch.ones(3, 64, device="cuda")
    out = torch.empty(3, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    for bad in (32, -2, 2 ** 31 - 1):
        cache.k.zero_(), out.zero_()
        cache.append_qkv(x, x, x, dev([5, bad, -1]), out, ws=ws)
        assert (out == 1).all() and int(cache.k.count_nonzero()) == 64
        with pytest.raises(w.WalError) as e:
            w.attention.status(ws)
        assert e.value.status == w.WAL_ERR_ARG
    cache.append_qkv(x[:0], x[:0], x[:0], dev([]), out[:0], ws=ws)
    w.attention.status(ws)
