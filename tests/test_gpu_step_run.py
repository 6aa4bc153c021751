"""The operators of a serving step together, as a server runs them (needs a B200): products, the plan of pages and
rows, norms and rotation into the cache, attention with a window or behind a shared prefix, the o product; eagerly
for prompts, then captured and replayed for single tokens, drafts, rejections and finished requests.

Each stage is compared with the FP64 oracle applied to what the stage before it left in memory, so its tolerance
is the operator's own.
"""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao, step_oracle as so

from attn_util import TYPES, assert_close, attention_tolerance, bf16
from gpu_util import needs_gpu, wal
from test_gpu_attention_run import Layer
from test_gpu_cache import raw
from test_gpu_step import dev, turned, weights

pytestmark = [pytest.mark.gpu, needs_gpu]

EPS = 1e-5


class Server(Layer):
    """A layer, its cache, and the state of B sequences, which only the device changes."""

    def __init__(self, rng, heads, kv_heads, D, typ, page, width, B, window=None, sinks=0):
        w = wal()
        self.n_pages = B * width * 2 // 3
        super().__init__(heads, kv_heads, D, typ, self.n_pages, page)
        self.rng, self.page, self.width, self.B, self.window, self.sinks = rng, page, width, B, window, sinks
        dw, self.w = weights(rng, D, torch.bfloat16)
        self.norm, self.rope = w.HeadNorm(*dw, eps=EPS), w.Rope(D, base=1e6)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.free, self.n_free = dev(rng.permutation(self.n_pages)), dev([self.n_pages])
        self.kv_len, self.n_new, self.q_start = dev([0] * B), dev([0] * B), dev([0] * (B + 1))
        self.groups = None  # (group_start, prefix_len)
        self.ws = torch.empty(512, dtype=torch.uint8, device="cuda")

    def buffers(self, T):
        b = super().buffers(T)
        b.update(x=torch.zeros(T, self.heads * self.D, dtype=torch.bfloat16, device="cuda"), att=torch.zeros_like(b["att"]),
                 pos=dev([-5] * T), slots=dev([-5] * T))
        return b

    def run(self, b, max_q):
        most = self.width * self.page
        for p, y in zip(self.proj, (b["q"], b["k"], b["v"])):
            p(b["x"], y)
        self.cache.plan(self.n_new, self.kv_len, self.table, self.free, self.n_free, self.q_start, b["pos"], b["slots"], ws=self.ws)
        self.cache.append_qkv(b["q"], b["k"], b["v"], b["slots"], b["qb"], positions=b["pos"], rope=self.rope, norm=self.norm)
        if self.groups:
            self.cache.attend_shared(b["qb"], self.q_start, self.kv_len, self.table, *self.groups, b["att"], max_q=max_q, max_kv=most,
                                     max_prefix=most, max_own=most)
        else:
            self.cache.attend(b["qb"], self.q_start, self.kv_len, self.table, b["att"], max_q=max_q, max_kv=most, window=self.window,
                              sinks=self.sinks)
        self.o(b["att"], b["y"])

    def before(self, b, new):
        """The inputs of a step, and the plan that it should make."""
        host = lambda t: t.cpu().numpy()
        T = len(b["x"])
        self.n_new.copy_(dev(new))
        b["x"].copy_(torch.from_numpy(bf16(self.rng.normal(size=(T, self.heads * self.D)))))
        b["att"].zero_()
        return so.plan(list(new), host(self.kv_len).tolist(), host(self.table), host(self.free), int(self.n_free), T, self.page, self.n_pages,
                       self.width * self.page)

    def check_step(self, b, plan, short=False):
        w, D = wal(), self.D
        assert plan["bad"] == short
        if short:
            with pytest.raises(w.WalError):
                w.attention.status(self.ws)
        else:
            w.attention.status(self.ws)
        for name, t in (("q_start", self.q_start), ("positions", b["pos"]), ("slots", b["slots"]), ("kv_len", self.kv_len),
                        ("n_free", self.n_free), ("table", self.table), ("free", self.free)):
            assert np.array_equal(t.cpu().numpy().reshape(-1), np.reshape(plan[name], -1)), name
        for p, name in zip(self.proj, "qkv"):
            p.check(b["x"], b[name], name)
        pos, slots = plan["positions"], plan["slots"]
        q, k, v = (b[name].cpu().double().numpy().reshape(len(pos), -1, D) for name in "qkv")
        ref, err = turned(q, pos, self.w[0], np.float32(EPS), D, D, "half")
        qb = b["qb"].cpu().double().numpy().reshape(q.shape)
        assert np.all(np.abs(qb - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)
        live, typ = slots >= 0, {v: k for k, v in TYPES.items()}[self.cache.k.dtype]
        at = (slots[live] // self.page, slice(None), slots[live] % self.page)
        held = []
        for (ref, err), codes, scale in ((turned(k, pos, self.w[1], np.float32(EPS), D, D, "half"), self.cache.k, self.cache.k_scale),
                                         ((v, np.zeros_like(v)), self.cache.v, self.cache.v_scale)):
            ref, err, val = ref[live], err[live], raw(codes)
            if scale is None:
                assert np.all(np.abs(val[at] - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)
            else:  # half a step of the code, the quotient's rounding, the errors before it
                sc = scale.cpu().double().numpy()
                grid = ao.step((np.abs(ref) + err) / sc[at][..., None], typ) * sc[at][..., None]
                val = val * sc[..., None]
                assert np.all(np.abs(val[at] - ref) <= grid / 2 + np.abs(ref) * 2.0 ** -22 + err)
            held.append(val)
        att = b["att"].cpu().double().numpy().reshape(q.shape)
        first, table = plan["q_start"], plan["table"]
        assert np.all(att[first[-1]:] == 0), "rows behind the last sequence were written"
        for i, L in enumerate(plan["kv_len"]):
            n = first[i + 1] - first[i]
            if n:
                j = np.arange(L)
                K, V = (t[table[i, j // self.page], :, j % self.page] for t in held)
                sees = so.window_sees(n, L, self.window or L, self.sinks)
                rows = slice(first[i], first[i + 1])
                o, a = so.attend(qb[rows], K, V, D ** -0.5, self.heads // self.kv_heads, sees)
                assert_close(att[rows], o, attention_tolerance(o, a, qb[rows], K, D ** -0.5), f"sequence {i}")
        self.o.check(b["att"], b["y"], "o")

    def steps(self, T, max_q, news):
        """Captured once, replayed for each of `news`."""
        b = self.buffers(T)
        self.n_new.zero_()
        self.run(b, max_q)  # warm-up: nobody gets anything
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run(b, max_q)
        for new in news:
            plan = self.before(b, new() if callable(new) else new)
            g.replay()
            self.check_step(b, plan)

    def once(self, new, T, max_q, short=False):
        b = self.buffers(T)
        plan = self.before(b, new)
        self.run(b, max_q)
        self.check_step(b, plan, short)


@pytest.mark.parametrize("typ,heads,kv_heads,D,window,sinks", [("bf16", 4, 1, 128, 50, 4), ("int8", 8, 2, 64, 33, 0), ("e4m3", 4, 4, 128, 70, 20),
                                                               ("e4m3", 2, 2, 64, None, 0)])
def test_serving_with_a_window(typ, heads, kv_heads, D, window, sinks):
    B = 5
    s = Server(np.random.default_rng(D + heads), heads, kv_heads, D, typ, 16, 16, B, window, sinks)
    s.once([150, 37, 1, 0, 60], 251, 150)
    s.once([20, 0, 33, 70, 0], 130, 128)
    lens = lambda: s.kv_len.cpu().numpy()
    # single tokens, drafts and what is rejected of them, a finished request and one in its place
    s.steps(12, 4, [[1] * B, [4, 1, 0, 1, 2], [-3, 1, 1, 1, -2], lambda: [1, -lens()[1], 1, 0, 1], [1, 4, 1, 2, 1], [1, 1, 1, 1, 0]])
    assert lens()[1] == 5
    s.once([-int(n) for n in lens()], 3, 1)  # all pages come back
    assert int(s.n_free) == s.n_pages and sorted(s.free.cpu().tolist()) == list(range(s.n_pages))
    s.once([200, 250, 200, 200, 200], 1050, 256, short=True)  # more than there are pages


@pytest.mark.parametrize("typ,heads,kv_heads,D", [("bf16", 4, 1, 128), ("int8", 8, 2, 64), ("e4m3", 16, 4, 64)])
@pytest.mark.parametrize("prefix", [48, 41])
def test_serving_behind_a_prefix(typ, heads, kv_heads, D, prefix):
    """One sequence fills the prefix's pages; the others' tables get them too, and go on in pages of their own."""
    B, page = 7, 16
    s = Server(np.random.default_rng(prefix + heads), heads, kv_heads, D, typ, page, 16, B)
    s.once([prefix] + [0] * (B - 1), prefix + 1, 64)
    whole = prefix // page  # pages that every sequence may read; the tokens behind them are each sequence's own
    s.table[1:, :whole] = s.table[:1, :whole]
    s.kv_len.fill_(whole * page)
    if prefix % page:  # give the first sequence's rest of a page back to the list
        s.free[int(s.n_free)] = s.table[0, whole]
        s.n_free += 1
    s.groups = dev([0, B]), dev([whole * page])
    s.once([30, 9, 1, 0, 64, 17, 2], 130, 64)
    lens = lambda: s.kv_len.cpu().numpy()
    s.steps(16, 4, [[1, 1, 1, 3, 1, 1, 1], [4, 1, 2, 1, 0, 1, 1], [-2, 1, -1, 1, 1, 1, 1], [1, 1, 1, 1, 1, 1, 0]])
    # one finishes, down to the shared tokens, and another request starts behind the same prefix
    s.steps(16, 4, [lambda: [1, 1, 1, 1, whole * page - lens()[4], 1, 1], [1, 1, 1, 1, 4, 1, 1]])
    assert lens()[4] == whole * page + 4
    s.groups = dev([0, 3, B]), dev([whole * page, page])  # fewer shared tokens, in groups: the same answers
    s.steps(16, 4, [[1] * B])


def test_plan_arrays_of_any_alignment():
    """Rows of positions and slots that do not start on 16 bytes, and every length of their end."""
    w = wal()
    rng = np.random.default_rng(0)
    cache = w.KvCache.empty(64, 16, 1, 64)
    for T in range(1, 14):
        for lead in (1, 2, 3):
            new, lens = rng.integers(0, 3, 5), rng.integers(0, 20, 5)
            need = -(-(lens + new) // 16)
            table, at = np.full((5, 4), -1), 0
            for i, n in enumerate(-(-lens // 16)):
                table[i, :n] = np.arange(at, at + n)
                at += n
            free = np.concatenate([np.arange(at, 64), np.zeros(at, int)])
            ref = so.plan(list(new), list(lens), table, free, 64 - at, T, 16, 64, 64)
            pos, slots = dev([-5] * (T + lead + 2)), dev([-5] * (T + lead + 2))
            kv_len, tab, fr, nf, q = dev(lens), dev(table), dev(free), dev([64 - at]), dev([-5] * 6)
            cache.plan(dev(new), kv_len, tab, fr, nf, q, pos[lead:lead + T], slots[lead:lead + T])
            for name, t in (("positions", pos[lead:lead + T]), ("slots", slots[lead:lead + T]), ("kv_len", kv_len), ("table", tab), ("free", fr),
                            ("n_free", nf), ("q_start", q)):
                assert np.array_equal(t.cpu().numpy().reshape(-1), np.reshape(ref[name], -1)), (name, T, lead)
            for t in (pos, slots):
                assert (t[:lead] == -5).all() and (t[lead + T:] == -5).all()
            assert need.max() <= 4


@pytest.mark.parametrize("B", [31, 32, 33, 511, 512, 513, 1024, 1025, 16384, 16385])
def test_plan_sizes_of_a_warp_and_a_cta(B):
    """Sequences around what a warp's probes, a CTA and a cluster take; most of them want nothing."""
    w = wal()
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B)
    new = np.where(rng.random(B) < 0.1, rng.integers(1, 60, B), 0)
    new = np.where(rng.random(B) < 0.1, -rng.integers(0, lens + 1), new)
    pages = -(-lens // 16)
    n_pages, width = int(pages.sum() + 4 * B), 10
    deal, at = rng.permutation(n_pages), 0
    table = np.full((B, width), -1)
    for i, n in enumerate(pages):
        table[i, :n] = deal[at:at + n]
        at += n
    free = np.concatenate([deal[at:], np.zeros(at, int)])
    T = int(np.maximum(new, 0).sum()) + 7
    ref = so.plan(list(new), list(lens), table, free, n_pages - at, T, 16, n_pages, 160)
    cache = w.KvCache.empty(n_pages, 16, 1, 64)
    kv_len, tab, fr, nf, q, pos, slots = dev(lens), dev(table), dev(free), dev([n_pages - at]), dev([-5] * (B + 1)), dev([-5] * T), dev([-5] * T)
    cache.plan(dev(new), kv_len, tab, fr, nf, q, pos, slots)
    for name, t in (("positions", pos), ("slots", slots), ("kv_len", kv_len), ("table", tab), ("free", fr), ("n_free", nf), ("q_start", q)):
        assert np.array_equal(t.cpu().numpy().reshape(-1), np.reshape(ref[name], -1)), name
