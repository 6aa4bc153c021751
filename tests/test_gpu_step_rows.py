"""Norms, rotation and cache of many tokens: odd counts, more items than threads (needs a B200).

More than 592 tokens go to CTAs of at most 128 threads, bf16 rows two tokens at a time: an odd count leaves a CTA with
one, and a token of more than 128 items of 16 elements takes several rounds."""
import numpy as np
import pytest
import torch

import test_gpu_step as step
from attn_util import TYPES
from gpu_util import needs_gpu, wal

pytestmark = [pytest.mark.gpu, needs_gpu]

# q heads, k heads, D: 320 and 640 items of rows (384 and 960 of a cache's), and counts that are no multiple of the threads
SHAPES = [(32, 8, 128), (40, 40, 128), (9, 4, 128), (20, 11, 64)]


@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,D", SHAPES + [(20, 11, 48)])
@pytest.mark.parametrize("T", [592, 593, 701])
def test_rows(inp, heads, kv, D, T):
    """Against the oracle, and bf16 rows in place."""
    layout = "half" if T != 701 else "interleaved"
    step.test_qk_norm_rope(inp, torch.bfloat16, layout, D, D if T != 593 else 16, heads, kv, T)
    step.test_qk_norm_rope(inp, None, layout, D, D, heads, kv, T)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,D", SHAPES)
@pytest.mark.parametrize("T", [592, 593, 701])
def test_append(inp, typ, heads, kv, D, T):
    step.test_qkv_append(inp, typ, heads, kv, D, 32, T, D if T != 701 else 16, "half" if T != 701 else "interleaved", T != 592)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("inp", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,D", SHAPES)
@pytest.mark.parametrize("skip", ["last", "all but the last", "all"])
def test_slots_of_the_last_rows(inp, typ, heads, kv, D, skip):
    """A CTA's one or two tokens, some of them without a slot: q is written all the same, the cache is what append stores."""
    w = wal()
    T, page = 593, 16
    rng = np.random.default_rng(heads)
    x, xv = step.rows(rng, T, heads + 2 * kv, D, inp, 8)
    q, k, v = x[:, :heads * D], x[:, heads * D:(heads + kv) * D], x[:, (heads + kv) * D:]
    slots = rng.permutation((T // page + 2) * page)[:T].astype(np.int32)
    if skip == "last":
        slots[-1] = -1
    else:
        slots[:-1 if skip == "all but the last" else T] = -1
    pos = rng.integers(0, 40000, T).astype(np.int32)
    rope = w.Rope(D, base=1e6)
    caches = [w.KvCache.empty(T // page + 2, page, kv, D, dtype=TYPES[typ]) for _ in range(2)]
    for c in caches:
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.view(torch.uint8).fill_(0x55)
    out = torch.full((T, heads * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((512,), 255, dtype=torch.uint8, device="cuda")
    caches[0].append_qkv(q, k, v, step.dev(slots), out[:, :heads * D], positions=step.dev(pos), rope=rope, ws=ws)
    w.attention.status(ws)
    caches[1].append(k, v, step.dev(slots), positions=step.dev(pos), rope=rope)
    for name in ("k", "v", "k_scale", "v_scale"):
        a, b = (getattr(c, name) for c in caches)
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    ref, err = step.turned(xv[:, :heads], pos, None, None, D, D, "half")
    got = out.cpu().double().numpy()
    assert np.all(got[:, heads * D:] == 5.0)
    assert np.all(np.abs(got[:, :heads * D].reshape(ref.shape) - ref) <= 2.0 ** -8 * (np.abs(ref) + err) + err)
