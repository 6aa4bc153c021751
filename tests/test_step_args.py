"""Refusals of the step's entry points (CPU only)."""
import numpy as np
import pytest
import torch

import ternary_sparse_binary_b200 as wal

from test_attention_args import BAD_CACHE, P, args, cache, refuses, rope

ARG, SHAPE, UNSUPPORTED, WORKSPACE = wal.WAL_ERR_ARG, wal.WAL_ERR_SHAPE, wal.WAL_ERR_UNSUPPORTED, wal.WAL_ERR_WORKSPACE


def norm(**kw):
    d = dict(head_dim=64, type=wal.WAL_BF16, eps=1e-6, q_weight=P, k_weight=P)
    d.update(kw)
    return wal.wal_head_norm(**d)


PLAN = dict(cache=cache(), n_new=P, kv_len=P + 64, B=3, table=P, ld_table=4, max_kv=64, free_pages=P, n_free=P + 128, T=9, q_start=P,
            positions=P, slots=P, kv_len_out=P + 64, n_free_out=P + 128, ws=P, ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE] + [
    (dict(B=0), SHAPE), (dict(B=65536), SHAPE), (dict(T=-1), SHAPE), (dict(T=2 ** 31 - 1), UNSUPPORTED), (dict(max_kv=0), SHAPE),
    (dict(max_kv=2 ** 30 + 1, ld_table=2 ** 30), UNSUPPORTED), (dict(max_kv=65), ARG), (dict(ws_bytes=511), WORKSPACE),
    (dict(kv_len_out=P), ARG), (dict(n_free_out=P), ARG), (dict(n_free_out=P + 64), ARG), (dict(n_free=P + 64), ARG)] + [
    (dict(**{name: None}), ARG) for name in ("n_new", "kv_len", "table", "free_pages", "n_free", "q_start", "positions", "slots",
                                             "kv_len_out", "n_free_out")] + [
    (dict(**{name: P + 2}), ARG) for name in ("n_new", "kv_len", "table", "free_pages", "n_free", "q_start", "positions", "slots")])
def test_plan_refuses(kw, status):
    refuses(status, wal.wal_kv_plan, *args(PLAN, kw))


BAD_NORM = [(dict(head_dim=128), SHAPE), (dict(type=2), ARG), (dict(eps=0.0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
            (dict(eps=float("inf")), ARG), (dict(q_weight=None), ARG), (dict(k_weight=None), ARG), (dict(k_weight=P + 2), ARG)]
BAD_ROPE = [(dict(rot_dim=0), SHAPE), (dict(rot_dim=24), UNSUPPORTED), (dict(layout=2), ARG), (dict(freq=None), ARG)]

ROWS = dict(norm=norm(), rope=rope(), Q=P, K=P + 512, x_type=0, T=3, n_heads=4, n_kv_heads=2, ldq=256, ldk=128, positions=P, Yq=P + 4096,
            ldyq=256, Yk=P + 8192, ldyk=128, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(norm=norm(**n)), s) for n, s in BAD_NORM] + [(dict(rope=rope(**r)), s) for r, s in BAD_ROPE] + [
    (dict(T=-1), SHAPE), (dict(n_heads=0), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(n_heads=65537, ldq=65537 * 64), UNSUPPORTED),
    (dict(x_type=2), ARG), (dict(ldq=255), ARG), (dict(ldq=258), ARG), (dict(ldk=124), ARG), (dict(ldyq=260), ARG), (dict(ldyk=120), ARG),
    (dict(Q=None), ARG), (dict(K=P + 4), ARG), (dict(Yq=None), ARG), (dict(Yk=None), ARG), (dict(positions=None), ARG),
    (dict(positions=P + 1), ARG), (dict(Yq=P), ARG), (dict(Yk=P + 512), ARG), (dict(x_type=1, Yq=P, ldq=264), ARG),
    (dict(x_type=1, Yq=P + 512), ARG), (dict(x_type=1, Yk=P), ARG), (dict(Yk=P + 4096), ARG)])
def test_qk_norm_rope_refuses(kw, status):
    refuses(status, wal.wal_qk_norm_rope, *args(ROWS, kw))


APPEND = dict(cache=cache(), norm=norm(), rope=rope(), Q=P, K=P + 512, V=P + 1024, in_type=0, T=3, n_heads=4, ldq=256, ldk=128, ldv=128,
              slots=P, positions=P, Yq=P + 4096, ldy=256, ws=P, ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE] + [
    (dict(norm=norm(**n)), s) for n, s in BAD_NORM] + [(dict(rope=rope(**r)), s) for r, s in BAD_ROPE] + [
    (dict(rope=rope(head_dim=128)), SHAPE), (dict(in_type=5), ARG), (dict(T=-1), SHAPE), (dict(n_heads=0), SHAPE),
    (dict(n_heads=65537, ldq=65537 * 64, ldy=65537 * 64), UNSUPPORTED), (dict(ldq=252), ARG), (dict(ldk=130), ARG), (dict(ldv=120), ARG), (dict(ldy=250), ARG),
    (dict(Q=None), ARG), (dict(K=None), ARG), (dict(V=P + 8), ARG), (dict(Yq=None), ARG), (dict(slots=None), ARG), (dict(positions=None), ARG),
    (dict(Yq=P), ARG), (dict(in_type=1, Yq=P + 512), ARG), (dict(in_type=1, Yq=P + 1024), ARG), (dict(in_type=1, Yq=P, ldy=264), ARG),
    (dict(ws_bytes=511), WORKSPACE)])
def test_qkv_append_refuses(kw, status):
    refuses(status, wal.wal_qkv_append, *args(APPEND, kw))


PAGED = dict(cache=cache(), Q=P, n_heads=4, T=3, ldq=256, q_start=P, kv_len=P, table=P, ld_table=4, B=2, max_q=2, max_kv=64, window=10,
             sinks=2, scale=0.1, O=P + 4096, ldo=256, ws=P, ws_bytes=1 << 30, stream=None)
BAD_ATTN = [(dict(n_heads=5), SHAPE), (dict(T=-1), SHAPE), (dict(B=0), SHAPE), (dict(B=65536), SHAPE), (dict(max_q=0), SHAPE), (dict(max_kv=0), SHAPE),
            (dict(max_kv=65), ARG), (dict(max_kv=2 ** 30 + 1), UNSUPPORTED), (dict(scale=float("nan")), ARG), (dict(Q=None), ARG), (dict(Q=P + 8), ARG),
            (dict(O=None), ARG), (dict(O=P), ARG), (dict(ldq=255), ARG), (dict(ldo=248), ARG), (dict(q_start=None), ARG), (dict(kv_len=P + 2), ARG),
            (dict(table=None), ARG)]


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE] + BAD_ATTN + [
    (dict(window=0), SHAPE), (dict(window=-5), SHAPE), (dict(sinks=-1), SHAPE), (dict(ws_bytes=511), WORKSPACE)])
def test_paged_window_refuses(kw, status):
    if kw == dict(O=P):
        status = ARG if torch.cuda.is_available() else wal.WAL_ERR_CUDA
    refuses(status, wal.wal_attn_paged_window, *args(PAGED, kw))


PROMPT = dict(Q=P, K=P, V=P, n_heads=4, n_kv_heads=2, head_dim=64, T=3, ldq=256, ldk=128, ldv=128, start=P, B=2, max_len=64, window=10, sinks=2,
              scale=0.1, O=P + 4096, ldo=256, ws=P, ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(window=0), SHAPE), (dict(sinks=-1), SHAPE), (dict(n_heads=5), SHAPE), (dict(head_dim=96), UNSUPPORTED), (dict(T=-1), SHAPE), (dict(B=0), SHAPE),
    (dict(max_len=0), SHAPE), (dict(scale=float("inf")), ARG), (dict(Q=None), ARG), (dict(K=P + 8), ARG), (dict(V=None), ARG), (dict(ldk=120), ARG),
    (dict(start=None), ARG), (dict(ws_bytes=511), WORKSPACE)])
def test_prompt_window_refuses(kw, status):
    refuses(status, wal.wal_attn_prompt_window, *args(PROMPT, kw))


SHARED = dict(cache=cache(), Q=P, n_heads=4, T=3, ldq=256, q_start=P, kv_len=P, table=P, ld_table=4, B=2, group_start=P, prefix_len=P, G=1, max_q=2,
              max_kv=64, max_prefix=32, max_own=32, scale=0.1, O=P + 4096, ldo=256, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("kw,status", [(dict(cache=cache(**c)), s) for c, s in BAD_CACHE] + [x for x in BAD_ATTN if x[0] != dict(O=P)] + [
    (dict(G=0), SHAPE), (dict(G=65536), SHAPE), (dict(max_prefix=-1), SHAPE), (dict(max_prefix=65), SHAPE), (dict(max_own=0), SHAPE),
    (dict(max_own=2 ** 30 + 1), UNSUPPORTED), (dict(group_start=None), ARG), (dict(prefix_len=P + 2), ARG), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=600), WORKSPACE)])
def test_shared_refuses(kw, status):
    refuses(status, wal.wal_attn_paged_shared, *args(SHARED, kw))


def test_workspace_sizes_are_those_that_the_calls_want():
    c = cache(n_pages=1 << 16, type=wal.WAL_KV_BF16, k_scale=None, v_scale=None)
    for T, B, max_q, max_kv in ((1, 1, 1, 64), (3, 3, 1, 30000), (90, 2, 50, 30000), (4000, 2, 2000, 4000)):
        for window, sinks in ((1, 0), (900, 4), (2000, 300), (40000, 0)):
            n = wal.wal_attn_paged_window_workspace_bytes(c, 4, T, B, max_q, max_kv, window, sinks)
            assert n >= 512
            kw = dict(cache=c, T=T, B=B, max_q=max_q, max_kv=max_kv, ld_table=2000, window=window, sinks=sinks, ws_bytes=n - 1)
            refuses(WORKSPACE, wal.wal_attn_paged_window, *args(PAGED, kw))
            if window >= max_kv:
                assert n == wal.wal_attn_paged_workspace_bytes(c, 4, T, B, max_q, max_kv)
        for G, pre, own in ((1, 0, 64), (2, 8000, 100), (3, 64, max_kv)):
            n = wal.wal_attn_paged_shared_workspace_bytes(c, 4, T, B, G, max_q, pre, own)
            kw = dict(cache=c, T=T, B=B, G=G, max_q=max_q, max_kv=30000, ld_table=2000, max_prefix=pre, max_own=own, ws_bytes=n - 1)
            refuses(WORKSPACE, wal.wal_attn_paged_shared, *args(SHARED, kw))
    for bad in (dict(window=0), dict(sinks=-1), dict(n_heads=3), dict(max_kv=0)):
        kw = dict(n_heads=4, T=3, B=2, max_q=2, max_kv=64, window=9, sinks=0)
        assert wal.wal_attn_paged_window_workspace_bytes(c, *{**kw, **bad}.values()) == 0
    for bad in (dict(G=0), dict(max_prefix=-1), dict(max_own=0), dict(n_heads=3)):
        kw = dict(n_heads=4, T=3, B=2, G=1, max_q=2, max_prefix=64, max_own=9)
        assert wal.wal_attn_paged_shared_workspace_bytes(c, *{**kw, **bad}.values()) == 0


def test_bindings_refuse():
    """What the library cannot see; every call stops before the device."""
    f = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    c, r = wal.KvCache.empty(4, 16, 2, 64, device="cpu"), wal.Rope(64, device="cpu")
    n = wal.HeadNorm(f(64), f(64))
    for bad in ((f(64), f(128)), (f(64), f(64, dtype=torch.float32)), (f(64, dtype=torch.float16),) * 2, (f(2, 32),) * 2, (f(128)[::2],) * 2):
        with pytest.raises(ValueError):
            wal.HeadNorm(*bad)
    qk = dict(q=f(3, 256), k=f(3, 128), positions=i(3), q_out=f(3, 256), k_out=f(3, 128), norm=n)
    for kw in (dict(k=f(3, 128, dtype=torch.float32)), dict(k=f(4, 128)), dict(q_out=f(3, 128)), dict(k_out=f(3, 64)), dict(q=f(3, 250)),
               dict(q_out=f(3, 256, dtype=torch.float32)), dict(q=f(256, 3).T), {}):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            r.apply_qk(**{**qk, **kw})
    qkv = dict(q=f(3, 256), k=f(3, 128), v=f(3, 128), slots=i(3), q_out=f(3, 256), positions=i(3), rope=r, norm=n)
    for kw in (dict(v=f(3, 128, dtype=torch.float32)), dict(k=f(3, 64)), dict(v=f(2, 128)), dict(q_out=f(3, 128)), dict(q=f(3, 250), q_out=f(3, 250)),
               dict(positions=None), dict(slots=i(3), q=f(256, 3).T), {}):
        with pytest.raises(ValueError):
            c.append_qkv(**{**qkv, **kw})
    plan = dict(n_new=i(2), kv_len=i(2), table=i(2, 4), free=i(4), n_free=i(1), q_start=i(3), positions=i(5), slots=i(5))
    for kw in (dict(table=i(3, 4)), dict(table=i(2, 8)[:, ::2]), dict(max_kv=65), dict(max_kv=2 ** 31), {}):
        with pytest.raises(ValueError):
            c.plan(**{**plan, **kw})
    att = dict(q=f(3, 256), q_start=i(3), kv_len=i(2), table=i(2, 4), out=f(3, 256), max_q=2, max_kv=64)
    for kw in (dict(window=0), dict(window=4, sinks=-1), dict(window=4, max_kv=65), dict(window=4, q=f(3, 250)), dict(window=4)):
        with pytest.raises(ValueError):
            c.attend(**{**att, **kw})
    share = dict(att, group_start=i(2), prefix_len=i(1), max_prefix=16, max_own=48)
    for kw in (dict(max_kv=65), dict(out=f(3, 128)), dict(max_own=2 ** 31), dict(max_prefix=2 ** 31), {}):
        with pytest.raises(ValueError):
            c.attend_shared(**{**share, **kw})
    prompt = dict(q=f(3, 256), k=f(3, 128), v=f(3, 128), start=i(2), out=f(3, 256), head_dim=64, max_len=3)
    for kw in (dict(window=0), dict(window=4, sinks=-1), dict(window=4)):
        with pytest.raises(ValueError):
            wal.attn_prompt(**{**prompt, **kw})
