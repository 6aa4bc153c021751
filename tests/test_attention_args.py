"""Refusals of the rotary, cache and attention entry points, and their host-side helpers (CPU only)."""
import math

import numpy as np
import pytest
import torch

import ternary_sparse_binary_b200 as wal
from oracle import attn_oracle as ao

P = 1 << 20  # an aligned address nobody follows: every call below stops before the device


def cache(**kw):
    d = dict(n_pages=4, page_size=16, n_heads=2, head_dim=64, type=wal.WAL_KV_INT8, k=P, v=P, k_scale=P, v_scale=P)
    d.update(kw)
    return wal.wal_kv_cache(**d)


def rope(**kw):
    d = dict(head_dim=64, rot_dim=64, layout=0, mscale=1.0, freq=P)
    d.update(kw)
    return wal.wal_rope_plan(**d)


def refuses(status, fn, *args):
    with pytest.raises(wal.WalError) as e:
        fn(*args)
    assert e.value.status == status, e.value


def args(defaults, kw):
    assert set(kw) <= set(defaults)
    return [kw.get(k, v) for k, v in defaults.items()]


BAD_CACHE = [(dict(n_pages=0), wal.WAL_ERR_SHAPE), (dict(n_heads=0), wal.WAL_ERR_SHAPE), (dict(page_size=8), wal.WAL_ERR_UNSUPPORTED),
             (dict(page_size=48), wal.WAL_ERR_UNSUPPORTED), (dict(page_size=512), wal.WAL_ERR_UNSUPPORTED),
             (dict(head_dim=96), wal.WAL_ERR_UNSUPPORTED), (dict(head_dim=256), wal.WAL_ERR_UNSUPPORTED),
             (dict(type=3), wal.WAL_ERR_ARG), (dict(n_pages=2 ** 31 - 1), wal.WAL_ERR_UNSUPPORTED),
             (dict(k=None), wal.WAL_ERR_ARG), (dict(v=None), wal.WAL_ERR_ARG), (dict(k_scale=None), wal.WAL_ERR_ARG),
             (dict(k=P + 8), wal.WAL_ERR_ARG), (dict(v_scale=P + 4), wal.WAL_ERR_ARG), (dict(n_heads=2000), wal.WAL_ERR_UNSUPPORTED)]

ROPE = dict(rope=rope(), X=P, x_type=0, T=3, n_heads=2, ldx=128, positions=P, Y=P + 4096, ldy=128, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(rope=rope(rot_dim=0)), wal.WAL_ERR_SHAPE), (dict(rope=rope(rot_dim=80)), wal.WAL_ERR_SHAPE),
    (dict(rope=rope(rot_dim=24)), wal.WAL_ERR_UNSUPPORTED), (dict(rope=rope(rot_dim=63)), wal.WAL_ERR_SHAPE),
    (dict(rope=rope(head_dim=272, rot_dim=64)), wal.WAL_ERR_UNSUPPORTED), (dict(rope=rope(layout=2)), wal.WAL_ERR_ARG),
    (dict(rope=rope(freq=None)), wal.WAL_ERR_ARG), (dict(rope=rope(freq=P + 4)), wal.WAL_ERR_ARG),
    (dict(x_type=2), wal.WAL_ERR_ARG), (dict(T=-1), wal.WAL_ERR_SHAPE), (dict(n_heads=0), wal.WAL_ERR_SHAPE),
    (dict(ldx=127), wal.WAL_ERR_ARG), (dict(ldx=130), wal.WAL_ERR_ARG), (dict(ldy=132), wal.WAL_ERR_ARG),
    (dict(X=None), wal.WAL_ERR_ARG), (dict(Y=None), wal.WAL_ERR_ARG), (dict(positions=None), wal.WAL_ERR_ARG),
    (dict(X=P + 4), wal.WAL_ERR_ARG), (dict(Y=P), wal.WAL_ERR_ARG), (dict(positions=P + 2), wal.WAL_ERR_ARG),
    (dict(x_type=1, Y=P, ldx=136), wal.WAL_ERR_ARG)])
def test_rope_refuses(kw, status):
    refuses(status, wal.wal_rope, *args(ROPE, kw))


APPEND = dict(cache=cache(), K=P, V=P, in_type=0, T=3, ldk=128, ldv=128, slots=P, positions=P, rope=rope(), ws=P,
              ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE] + [
    (dict(rope=rope(head_dim=128)), wal.WAL_ERR_SHAPE), (dict(in_type=5), wal.WAL_ERR_ARG), (dict(T=-1), wal.WAL_ERR_SHAPE),
    (dict(ldk=124), wal.WAL_ERR_ARG), (dict(ldv=129), wal.WAL_ERR_ARG), (dict(in_type=1, ldk=132), wal.WAL_ERR_ARG),
    (dict(K=None), wal.WAL_ERR_ARG), (dict(V=P + 1), wal.WAL_ERR_ARG), (dict(slots=None), wal.WAL_ERR_ARG),
    (dict(positions=None), wal.WAL_ERR_ARG), (dict(ws_bytes=511), wal.WAL_ERR_WORKSPACE)])
def test_append_refuses(kw, status):
    refuses(status, wal.wal_kv_append, *args(APPEND, kw))


READ = dict(cache=cache(), table=P, ld_table=4, start=P, B=2, max_len=64, K=P, V=P, out_type=1, T=9, ldk=128, ldv=128,
            ws=P, ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE] + [
    (dict(table=None), wal.WAL_ERR_ARG), (dict(start=None), wal.WAL_ERR_ARG), (dict(ld_table=3), wal.WAL_ERR_ARG),
    (dict(B=0), wal.WAL_ERR_SHAPE), (dict(B=65536), wal.WAL_ERR_SHAPE), (dict(max_len=0), wal.WAL_ERR_SHAPE),
    (dict(T=-1), wal.WAL_ERR_SHAPE), (dict(out_type=2), wal.WAL_ERR_ARG), (dict(ldk=120), wal.WAL_ERR_ARG),
    (dict(V=P + 2), wal.WAL_ERR_ARG), (dict(ws_bytes=0), wal.WAL_ERR_WORKSPACE)])
def test_read_refuses(kw, status):
    refuses(status, wal.wal_kv_read, *args(READ, kw))


PAGED = dict(cache=cache(), Q=P, n_heads=4, T=6, ldq=256, q_start=P, kv_len=P, table=P, ld_table=4, B=2, max_q=3, max_kv=64,
             scale=0.125, O=P, ldo=256, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE if c != dict(n_heads=2000)] + [
    (dict(n_heads=3), wal.WAL_ERR_SHAPE), (dict(n_heads=0), wal.WAL_ERR_SHAPE), (dict(n_heads=258, ldq=16512, ldo=16512), wal.WAL_ERR_UNSUPPORTED),
    (dict(T=-1), wal.WAL_ERR_SHAPE), (dict(B=0), wal.WAL_ERR_SHAPE), (dict(B=65536), wal.WAL_ERR_SHAPE),
    (dict(max_q=0), wal.WAL_ERR_SHAPE), (dict(max_kv=0), wal.WAL_ERR_SHAPE), (dict(ld_table=3), wal.WAL_ERR_ARG),
    (dict(ldq=248), wal.WAL_ERR_ARG), (dict(ldo=260), wal.WAL_ERR_ARG), (dict(Q=None), wal.WAL_ERR_ARG), (dict(O=P + 8), wal.WAL_ERR_ARG),
    (dict(q_start=None), wal.WAL_ERR_ARG), (dict(kv_len=P + 2), wal.WAL_ERR_ARG), (dict(table=None), wal.WAL_ERR_ARG),
    (dict(scale=math.inf), wal.WAL_ERR_ARG), (dict(scale=math.nan), wal.WAL_ERR_ARG), (dict(ws=None, max_kv=20000, ld_table=2000), wal.WAL_ERR_WORKSPACE),
    (dict(ws_bytes=256), wal.WAL_ERR_WORKSPACE), (dict(ws_bytes=4096, max_kv=20000, ld_table=2000), wal.WAL_ERR_WORKSPACE)])
def test_paged_refuses(kw, status):
    refuses(status, wal.wal_attn_paged, *args(PAGED, kw))


PROMPT = dict(Q=P, K=P, V=P, n_heads=4, n_kv_heads=2, head_dim=64, T=6, ldq=256, ldk=128, ldv=128, start=P, B=2, max_len=6,
              scale=0.125, O=P, ldo=256, ws=P, ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_heads=5), wal.WAL_ERR_SHAPE), (dict(n_kv_heads=0), wal.WAL_ERR_SHAPE), (dict(head_dim=32), wal.WAL_ERR_UNSUPPORTED),
    (dict(T=-1), wal.WAL_ERR_SHAPE), (dict(B=0), wal.WAL_ERR_SHAPE), (dict(max_len=0), wal.WAL_ERR_SHAPE),
    (dict(ldq=252), wal.WAL_ERR_ARG), (dict(ldk=120), wal.WAL_ERR_ARG), (dict(ldv=132), wal.WAL_ERR_ARG), (dict(ldo=0), wal.WAL_ERR_ARG),
    (dict(K=None), wal.WAL_ERR_ARG), (dict(V=P + 2), wal.WAL_ERR_ARG), (dict(start=None), wal.WAL_ERR_ARG),
    (dict(scale=-math.inf), wal.WAL_ERR_ARG), (dict(ws_bytes=511), wal.WAL_ERR_WORKSPACE)])
def test_prompt_refuses(kw, status):
    refuses(status, wal.wal_attn_prompt, *args(PROMPT, kw))


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour on a host without a GPU")
def test_valid_calls_need_a_gpu():
    """Every argument in order: the calls go as far as the missing device and no further."""
    for fn, defaults in ((wal.wal_rope, ROPE), (wal.wal_kv_append, APPEND), (wal.wal_kv_read, READ),
                         (wal.wal_attn_paged, PAGED), (wal.wal_attn_prompt, PROMPT)):
        refuses(wal.WAL_ERR_CUDA, fn, *defaults.values())


def test_workspace_bytes():
    c = cache()
    assert wal.wal_attn_paged_workspace_bytes(c, 4, 6, 2, 3, 64) >= 512
    assert wal.wal_attn_paged_workspace_bytes(c, 3, 6, 2, 3, 64) == 0
    assert wal.wal_attn_paged_workspace_bytes(cache(head_dim=32), 4, 6, 2, 3, 64) == 0


def test_cache_sizes():
    assert wal.wal_kv_cache_sizes(4, 16, 2, 64, wal.WAL_KV_BF16) == [16384, 16384, 0, 0]
    assert wal.wal_kv_cache_sizes(4, 16, 2, 64, wal.WAL_KV_INT8) == [8192, 8192, 512, 512]
    assert wal.wal_kv_cache_sizes(2 ** 21, 256, 64, 128, wal.WAL_KV_E4M3)[0] == 2 ** 42


@pytest.mark.parametrize("rot", [2, 64, 128, 256])
@pytest.mark.parametrize("kw", [{}, dict(scaling="linear", factor=8.0),
                                dict(scaling="parts", factor=40.0, original_len=4096.0, slow=1.0, fast=32.0)])
def test_frequencies_match_the_oracle(rot, kw):
    out = np.zeros(rot // 2, np.uint64)
    code = dict(none=0, linear=1, parts=2)[kw.get("scaling", "none")]
    m = wal.wal_rope_freqs(rot, 1e6, code, kw.get("factor", 1.0), kw.get("original_len", 0.0), kw.get("slow", 1.0),
                           kw.get("fast", 32.0), out.ctypes.data)
    f, ms = ao.rope_freqs(rot, base=1e6, **kw)
    assert m == np.float32(ms)
    got = out.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
    # the oracle's double pow, product and quotient round a few times (2^-53 each), and base^-x amplifies the
    # rounding of its exponent x ln(base) < 14 times; the fixed point rounds f / 2 pi to half of 2^-64, 2 pi 2^-65 here
    assert np.all(np.abs(got - f) <= f * 40 * 2.0 ** -53 + 2 * math.pi * 2.0 ** -65)


@pytest.mark.parametrize("a", [(0, 1e4, 0, 1, 0, 1, 32), (3, 1e4, 0, 1, 0, 1, 32), (258, 1e4, 0, 1, 0, 1, 32)])
def test_frequencies_refuse_shapes(a):
    refuses(wal.WAL_ERR_SHAPE, wal.wal_rope_freqs, *a, np.zeros(200, np.uint64).ctypes.data)


@pytest.mark.parametrize("a", [(64, 1.0, 0, 1, 0, 1, 32), (64, math.nan, 0, 1, 0, 1, 32), (64, 1e4, 3, 1, 0, 1, 32),
                               (64, 1e4, 1, 0.5, 0, 1, 32), (64, 1e4, 2, 4, 0, 1, 32), (64, 1e4, 2, 4, 4096, 32, 32),
                               (64, 1e4, 2, math.inf, 4096, 1, 32)])
def test_frequencies_refuse_arguments(a):
    refuses(wal.WAL_ERR_ARG, wal.wal_rope_freqs, *a, np.zeros(200, np.uint64).ctypes.data)


def test_binding_checks_tensors():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(4, 2, 16)
    wal.KvCache(k, k, s, s)
    for bad in ((k, k), (k, k, s, s.double()), (k, k.float(), s, s), (k, k[:, :, :8], s, s), (k[..., :32], k[..., :32], s, s),
                (k.transpose(1, 2), k.transpose(1, 2), s.transpose(1, 2), s.transpose(1, 2))):
        with pytest.raises(ValueError):
            wal.KvCache(*bad)
    c = wal.KvCache(k, k, s, s)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    x = torch.zeros(3, 128)
    for call in (lambda: c.append(x, x[:2], i(0, 1, 2)), lambda: c.append(x, x, i(0, 1, 2).long()),
                 lambda: c.append(x, x, i(0, 1, 2)),  # not on a GPU
                 lambda: c.attend(x, i(0, 3), i(3), i(0)[None], x, 3, 3),
                 lambda: wal.attn_prompt(x.bfloat16(), x.bfloat16(), x.bfloat16(), i(0, 3), x.bfloat16(), 48, 3),
                 lambda: c.read(i(0)[None], i(0, 3), x, x[:, ::2], 3)):
        with pytest.raises(ValueError):
            call()


def test_a_narrow_slice_of_a_page_table_is_refused():
    """The bound on the lengths reaches past the table's columns, into a wider table that it is a slice of."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c = wal.KvCache(k, k)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    wide = torch.zeros(2, 8, dtype=torch.int32)
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for n in (1, 3, 7):
        table = wide[:, 8 - n:]
        with pytest.raises(ValueError, match="cover"):
            c.attend(x, i(0, 1, 2), i(1, 1), table, x, max_q=1, max_kv=16 * n + 1)
        with pytest.raises(ValueError, match="cover"):
            c.read(table, i(0, 1, 2), x, x, max_len=16 * n + 1)
        with pytest.raises(ValueError, match="device"):  # as far as the table goes: the next check
            c.attend(x, i(0, 1, 2), i(1, 1), table, x, max_q=1, max_kv=16 * n)


def test_lengths_past_32_bits_of_arithmetic_are_refused():
    """The kernels add splits and steps to a key's number: a bound near 2^31 would wrap them."""
    wide = dict(cache=cache(n_pages=2 ** 22, page_size=256, n_heads=1, type=wal.WAL_KV_BF16), n_heads=1, ldq=64, ldo=64,
                ld_table=2 ** 23)
    for n_kv in (2 ** 30 + 1, 2 ** 31 - 1):
        for max_q in (1, 3):
            refuses(wal.WAL_ERR_UNSUPPORTED, wal.wal_attn_paged, *args(PAGED, dict(wide, max_kv=n_kv, max_q=max_q)))
            assert wal.wal_attn_paged_workspace_bytes(wide["cache"], 1, 6, 2, max_q, n_kv) == 0
    assert wal.wal_attn_paged_workspace_bytes(wide["cache"], 1, 6, 2, 3, 2 ** 30) >= 512
    refuses(wal.WAL_ERR_UNSUPPORTED, wal.wal_attn_prompt, *args(PROMPT, dict(n_heads=1, n_kv_heads=1, T=2 ** 30 + 1, max_len=2 ** 31 - 300)))
    # a loose bound is no reason: no sequence has more tokens than the call
    if not torch.cuda.is_available():
        refuses(wal.WAL_ERR_CUDA, wal.wal_attn_prompt, *args(PROMPT, dict(n_heads=1, n_kv_heads=1, max_len=2 ** 31 - 300)))


def test_numbers_past_32_bits_are_refused():
    """Strides and bounds of which the library would see the low 32 bits only."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c = wal.KvCache(k, k)
    i = lambda *v: torch.tensor(v, dtype=torch.int32)
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    far = torch.empty(3, 2 ** 32 + 128, dtype=torch.bfloat16, device="meta")[:, :128]
    table = i(0, 1)[None]
    for call in (lambda: wal.Rope(64, device="cpu").apply(far, i(0, 1, 2), x), lambda: wal.Rope(64, device="cpu").apply(x, i(0, 1, 2), far),
                 lambda: c.append(far, x, i(0, 1, 2)), lambda: c.append(x, far, i(0, 1, 2)),
                 lambda: c.read(table, i(0, 3), far, x, 3), lambda: c.read(table, i(0, 3), x, far, 3),
                 lambda: c.attend(far, i(0, 3), i(3), table, x, 3, 3), lambda: c.attend(x, i(0, 3), i(3), table, far, 3, 3),
                 lambda: c.attend(x, i(0, 3), i(3), table, x, 2 ** 32 + 3, 3),
                 lambda: c.attend(x, i(0, 1, 3), i(1, 2), torch.empty(2, 2 ** 32 + 2, dtype=torch.int32, device="meta")[:, :2], x, 3, 3),
                 lambda: c.attend_workspace_bytes(2, 3, 1, 3, 2 ** 32 + 3), lambda: c.attend_workspace_bytes(2, 3, 1, 2 ** 32 + 3, 3),
                 lambda: wal.attn_prompt(x, far, x, i(0, 3), x, 64, 3), lambda: wal.attn_prompt(x, x, far, i(0, 3), x, 64, 3),
                 lambda: wal.attn_prompt(x, x, x, i(0, 3), x, 64, 2 ** 32 + 3)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("shapes", [[(n, n, 1, 32768) for n in range(1, 65)], [(T, 4, T, 16384) for T in (1, 16, 64, 256, 512, 1024, 4096)]])
def test_a_workspace_serves_every_shape_whose_size_it_has(shapes):
    """Sizes rise and fall with the batch; the largest of them serves all, and each is exact."""
    c = cache(n_pages=1 << 16, page_size=64, n_heads=8, head_dim=128)
    call = dict(cache=c, n_heads=32, ldq=4096, ldo=4096, ld_table=512)
    need = [wal.wal_attn_paged_workspace_bytes(c, 32, *s) for s in shapes]
    assert need != sorted(need)  # a smaller batch may need more
    for (T, B, max_q, max_kv), n in zip(shapes, need):
        kw = dict(call, T=T, B=B, max_q=max_q, max_kv=max_kv)
        refuses(wal.WAL_ERR_WORKSPACE, wal.wal_attn_paged, *args(PAGED, dict(kw, ws_bytes=n - 1)))
        if not torch.cuda.is_available():
            for enough in (n, max(need)):
                refuses(wal.WAL_ERR_CUDA, wal.wal_attn_paged, *args(PAGED, dict(kw, ws_bytes=enough)))
