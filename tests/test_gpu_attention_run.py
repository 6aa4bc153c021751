"""The attention operators together, as a layer uses them, and batches of many sequences (needs a B200).

Each stage is compared with the FP64 oracle applied to what the stage before
it left in memory, so its tolerance is the operator's own.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import attn_oracle as ao
from wal_synth import gen_components

from attn_util import TYPES, assert_close, attention_tolerance, bf16
from gpu_util import assert_parity, device_matrix, needs_gpu, stream, wal
from test_gpu_attention import run_paged, run_prompt
from test_gpu_cache import i32, raw, turn_error

pytestmark = [pytest.mark.gpu, needs_gpu]


class Product:
    def __init__(self, N, K, k, r, index):
        self.c = gen_components(N, K, k, r, config_id=97, matrix_index=index)
        self.pm = device_matrix(self.c)

    def __call__(self, x, y):
        nb = self.pm.workspace_bytes(x.shape[0])
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        wal().wal_gemm_small_m(self.pm.desc, x.data_ptr(), x.shape[0], x.stride(0), y.data_ptr(), y.stride(0),
                               ws.data_ptr(), nb, stream())

    def check(self, x, y, what):
        bits = x.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)
        assert_parity(y.cpu().double().numpy(), oracle.matmul(self.c, bits), bits, self.c.alpha, what)


class Layer:
    """q, k, v products, rotary positions, the cache, attention, the o product."""

    def __init__(self, heads, kv_heads, D, typ, pages, page):
        w = wal()
        self.heads, self.kv_heads, self.D, hidden = heads, kv_heads, D, heads * D
        # one buffer for q, k and v, as the products of a fused projection would leave them
        self.proj = [Product(n * D, hidden, 8, 8, i) for i, n in enumerate((heads, kv_heads, kv_heads))]
        self.o = Product(hidden, hidden, 4, 8, 3)
        self.rope = w.Rope(D, base=5e5, layout="half")
        self.cache = w.KvCache.empty(pages, page, kv_heads, D, dtype=TYPES[typ])

    def buffers(self, T):
        new = lambda cols, dtype: torch.full((T, cols), float("nan"), dtype=dtype, device="cuda")
        h, kv = self.heads * self.D, self.kv_heads * self.D
        qkv = new(h + 2 * kv, torch.float32)
        return dict(qkv=qkv, q=qkv[:, :h], k=qkv[:, h:h + kv], v=qkv[:, h + kv:], qb=new(h, torch.bfloat16),
                    kb=new(kv, torch.bfloat16), att=new(h, torch.bfloat16), y=new(h, torch.float32))

    def before(self, x, b, pos, slots):
        for p, y in zip(self.proj, (b["q"], b["k"], b["v"])):
            p(x, y)
        self.rope.apply(b["q"], pos, b["qb"])
        self.cache.append(b["k"], b["v"], slots, positions=pos, rope=self.rope)

    def check(self, x, b, pos, slots, seqs, prompt=False):
        """seqs: (first row, rows, slots of all its tokens) of each sequence."""
        D, pos, slots = self.D, pos.cpu().numpy(), slots.cpu().numpy()
        for p, name in zip(self.proj, "qkv"):
            p.check(x, b[name], name)
        f, m = ao.rope_freqs(D, base=5e5)
        q, k, v = (b[name].cpu().double().numpy().reshape(len(pos), -1, D) for name in "qkv")
        ref, qb = ao.rotate(q, pos, f, m), b["qb"].cpu().double().numpy().reshape(q.shape)
        assert np.all(np.abs(qb - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * turn_error(q, D, m, "half"))
        live, page = slots >= 0, self.cache.page_size
        held = []
        for val, err, codes, scale in ((ao.rotate(k, pos, f, m), turn_error(k, D, m, "half"), self.cache.k, self.cache.k_scale),
                                       (v, np.zeros_like(v), self.cache.v, self.cache.v_scale)):
            at = lambda s: (s // page, slice(None), s % page)
            codes, sc = raw(codes), None if scale is None else scale.cpu().double().numpy()[..., None]
            got, val, err = codes[at(slots[live])], val[live], err[live]
            if sc is None:
                assert np.all(np.abs(got - val) <= 2.0 ** -8 * np.abs(val) + 1.01 * err)
            else:  # half a step of the code, the quotient's rounding, the rotation's error
                s = sc[at(slots[live])]
                grid = ao.step(val / s, "int8" if self.cache.k.dtype == torch.int8 else "e4m3")
                assert np.all(np.abs(got * s - val) <= s * grid / 2 * (1 + 1e-12) + np.abs(val) * 2.0 ** -23 + 1.01 * err)
                codes = codes * sc
            held.append([codes[at(s)] for _, _, s in seqs])
        if prompt:
            k, v = (b[n].cpu().double().numpy().reshape(len(pos), -1, D) for n in ("kb", "vb"))
            held = [[t[r:r + n] for r, n, _ in seqs] for t in (k, v)]
        att = b["att"].cpu().double().numpy().reshape(q.shape)
        for (r, n, _), k, v in zip(seqs, *held):
            if n:
                o, a = ao.attend(qb[r:r + n], k, v, D ** -0.5, self.heads // self.kv_heads)
                assert_close(att[r:r + n], o, attention_tolerance(o, a, qb[r:r + n], k, D ** -0.5), f"rows {r}")
        self.o.check(b["att"], b["y"], "o")


@pytest.mark.parametrize("typ,heads,kv_heads,D", [("bf16", 4, 1, 128), ("int8", 8, 2, 64), ("e4m3", 4, 4, 128)])
def test_layer(typ, heads, kv_heads, D):
    """Prompts, then a chunk of new tokens, then single tokens by a captured graph with a padded batch."""
    w = wal()
    rng = np.random.default_rng(D + heads)
    page, width, B = 32, 8, 4
    layer = Layer(heads, kv_heads, D, typ, B * width, page)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    tab = torch.from_numpy(table).cuda()
    slot = lambda b, p: table[b, p // page] * page + p % page
    lens = np.zeros(B, np.int64)  # the last place of the batch stays empty

    def tokens(n_new):
        """Positions and slots of the new tokens, and the sequences' tokens."""
        pos = np.concatenate([np.arange(lens[b], lens[b] + n) for b, n in enumerate(n_new)])
        slots = np.concatenate([slot(b, np.arange(lens[b], lens[b] + n)) for b, n in enumerate(n_new)])
        lens[:] += n_new
        start = np.concatenate([[0], np.cumsum(n_new)])
        return pos, slots, start, [(start[b], n, slot(b, np.arange(lens[b]))) for b, n in enumerate(n_new)]

    # a prompt each
    pos, slots, start, seqs = tokens([150, 37, 1, 0])
    x = torch.from_numpy(bf16(rng.normal(size=(len(pos), heads * D)))).bfloat16().cuda()
    b = layer.buffers(len(pos))
    layer.before(x, b, i32(pos), i32(slots))
    layer.rope.apply(b["k"], i32(pos), b["kb"])
    b["vb"] = b["v"].bfloat16()
    w.attn_prompt(b["qb"], b["kb"], b["vb"], i32(start), b["att"], head_dim=D, max_len=150)
    layer.o(b["att"], b["y"])
    layer.check(x, b, i32(pos), i32(slots), seqs, prompt=True)

    # more tokens of each
    pos, slots, start, seqs = tokens([20, 1, 33, 0])
    x = torch.from_numpy(bf16(rng.normal(size=(len(pos), heads * D)))).bfloat16().cuda()
    b = layer.buffers(len(pos))
    layer.before(x, b, i32(pos), i32(slots))
    layer.cache.attend(b["qb"], i32(start), i32(lens), tab, b["att"], max_q=33, max_kv=width * page)
    layer.o(b["att"], b["y"])
    layer.check(x, b, i32(pos), i32(slots), seqs)

    # single tokens: captured once, replayed with new values
    x, b = torch.zeros(B, heads * D, dtype=torch.bfloat16, device="cuda"), layer.buffers(B)
    pos_d, slots_d, lens_d, start_d = i32([0] * B), i32([-1] * B), i32([0] * B), i32(range(B + 1))

    def step():
        layer.before(x, b, pos_d, slots_d)
        layer.cache.attend(b["qb"], start_d, lens_d, tab, b["att"], max_q=1, max_kv=width * page)
        layer.o(b["att"], b["y"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        pos, slots, _, seqs = tokens([1, 1, 1, 0])
        seqs = seqs[:3] + [(3, 1, np.zeros(0, np.int64))]  # a row without a token: zeros
        pos_d.copy_(i32(np.append(pos, 0)))
        slots_d.copy_(i32(np.append(slots, -1)))
        lens_d.copy_(i32(lens))
        x.copy_(torch.from_numpy(bf16(rng.normal(size=(B, heads * D)))).bfloat16())
        x[3] = 0
        for t in b.values():
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert not b["att"][3].any()
        layer.check(x, b, pos_d, slots_d, seqs)


# ---- many sequences ----------------------------------------------------------

def test_prompt_many_sequences():
    """More sequences than a warp looks at once, more pieces than SMs, empty ones between."""
    rng = np.random.default_rng(70)
    lens = [int(n) for n in np.where(rng.random(75) < 0.2, 0, rng.integers(1, 400, 75))]
    run_prompt(lens, 6, 2, 64, seed=70, spread=2.0)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("most,max_kv", [(60, 700), (300, 400), (12, 3000)])
def test_chunks_many_sequences(most, max_kv, typ):
    rng = np.random.default_rng(most)
    lens = [int(n) for n in np.where(rng.random(70) < 0.15, 0, rng.integers(1, max_kv, 70))]
    n_q = [int(n) for n in np.where(rng.random(70) < 0.15, 0, rng.integers(1, most, 70))]
    run_paged(lens, n_q, 4, 1, 64, 16, typ, seed=most, spread=2.0)


def test_chunk_split_and_uneven():
    """Keys in splits for 40 sequences, most of them far shorter than the bound."""
    lens = [9000] + [3 + 11 * i for i in range(39)]
    run_paged(lens, [40] + [1 + i % 30 for i in range(39)], 4, 4, 64, 64, "bf16", seed=4, bounds=(50, 20000))


@pytest.mark.parametrize("typ", list(TYPES))
def test_decode_many_sequences(typ):
    rng = np.random.default_rng(90)
    lens = [int(n) for n in np.where(rng.random(130) < 0.1, 0, rng.integers(1, 600, 130))]
    run_paged(lens, [1] * 130, 4, 2, 128, 32, typ, seed=90, spread=2.0, bounds=(1, 4096))


def test_many_short_chunks():
    """Drafts of a few tokens for more sequences than the kernel has CTAs."""
    rng = np.random.default_rng(300)
    lens = [int(n) for n in rng.integers(0, 200, 300)]
    run_paged(lens, [int(n) for n in rng.integers(0, 9, 300)], 8, 2, 64, 16, "int8", seed=300, spread=2.0)


def test_long_prompt_with_a_nonfinite_last_value():
    """Thousands of keys are gone through again for each row beside the bad one, and nobody gives up waiting."""
    w = wal()
    rng = np.random.default_rng(31)
    T, D = 12000, 64
    q, k, v = (torch.from_numpy(rng.normal(size=(T, h * D)).astype(np.float32)).bfloat16().cuda() for h in (4, 1, 1))
    ref, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    w.attn_prompt(q, k, v, i32([0, T]), ref, head_dim=D, max_len=T, ws=ws)
    v[T - 1] = float("nan")
    w.attn_prompt(q, k, v, i32([0, T]), out, head_dim=D, max_len=T, ws=ws)
    w.attention.status(ws)
    assert torch.isnan(out[T - 1]).all()
    # done again in fp32: the weights' rounding (2^-8 of at most max |v| < 6) and two of the output
    r, o = ref[:T - 1].float(), out[:T - 1].float()
    assert torch.all((o - r).abs() <= 2.0 ** -7 * r.abs() + 6 * 2.0 ** -8)


def test_one_token_of_everything():
    """The smallest calls: one token, one head, one page."""
    for typ in TYPES:
        run_paged([1], [1], 1, 1, 64, 16, typ, lead=0, trail=0, pad=0)
    run_prompt([1], 1, 1, 64, lead=0, trail=0, pad=0)


def test_workspaces_are_checked_and_cleared():
    w = wal()
    cache = w.KvCache.empty(4, 16, 2, 64)
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    slots = i32([0, 1, 64])  # the last is out of range
    for ws in (torch.empty(512, dtype=torch.uint8), torch.empty(1024, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(512, device="cuda")):
        with pytest.raises(ValueError):
            cache.append(x, x, slots, ws=ws)
    with pytest.raises(ValueError):
        w.attention.status(torch.empty(256, dtype=torch.uint8, device="cuda"))
    ws = torch.full((512,), 0xFF, dtype=torch.uint8, device="cuda")
    cache.append(x, x, slots, ws=ws)
    with pytest.raises(w.WalError):
        w.attention.status(ws)
    none = x[:0]
    cache.read(i32([[0]]), i32([0, 0]), none, none, max_len=16, ws=ws)  # nothing to read: nothing recorded
    w.attention.status(ws)


def test_calls_without_tokens():
    """Empty batches change nothing, whatever the bounds."""
    w = wal()
    rope, cache = w.Rope(64), w.KvCache.empty(4, 16, 2, 64, dtype=torch.int8)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.zero_()
    x, none = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda"), i32([])
    kv, tab = x[:, :128], torch.zeros(3, 2048, dtype=torch.int32, device="cuda")
    ws = torch.full((512,), 0xFF, dtype=torch.uint8, device="cuda")
    for scratch in (None, ws):
        rope.apply(x, none, x)
        cache.append(kv, kv, none, positions=none, rope=rope, ws=scratch)
        cache.read(tab, i32([0, 0, 0, 0]), kv, kv, max_len=32768, ws=scratch)
        for max_q in (1, 500):
            cache.attend(x, i32([0, 0, 0, 0]), i32([5, 0, 9]), tab, x, max_q=max_q, max_kv=32768, ws=scratch)
        w.attn_prompt(x, kv, kv, i32([0, 0]), x, head_dim=64, max_len=100, ws=scratch)
    w.attention.status(ws)
    assert not cache.k.any() and not cache.k_scale.any()


def test_outputs_that_are_inputs_are_refused():
    """Rows are read after others are written, so nothing may be done in place."""
    w = wal()
    cache = w.KvCache.empty(4, 16, 2, 64)
    q, k, v = (torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    start = i32([0, 3])

    def refuses(call):
        with pytest.raises(w.WalError) as e:
            call()
        assert e.value.status == w.WAL_ERR_ARG

    for max_q in (3, 100):
        refuses(lambda: cache.attend(q, start, i32([3]), i32([[0]]), q, max_q=max_q, max_kv=16))
    for out in (q, k, v):
        refuses(lambda: w.attn_prompt(q, k, v, start, out, head_dim=64, max_len=3))
