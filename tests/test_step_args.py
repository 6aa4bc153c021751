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
