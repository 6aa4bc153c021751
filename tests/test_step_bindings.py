"""Arguments that the bindings of a serving step would hand on wrongly (CPU only)."""
import pytest
import torch

import ternary_sparse_binary_b200 as wal

f = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype)
i = lambda *shape: torch.zeros(shape, dtype=torch.int32)
WIDE = torch.empty((2, 1 << 28), dtype=torch.int32, device="meta")  # 2^32 tokens in pages of 16
ATTEND = dict(q=f(3, 256), q_start=i(3), kv_len=i(2), table=i(2, 4), out=f(3, 256), max_q=2, max_kv=64)


def cache():
    return wal.KvCache.empty(4, 16, 2, 64, device="cpu")


def refused(match, call, **kw):
    with pytest.raises(ValueError, match=match):
        call(**kw)


@pytest.mark.parametrize("max_kv", [2 ** 31, 2 ** 32, 2 ** 32 - 5])
@pytest.mark.parametrize("ws", [None, torch.zeros(4096, dtype=torch.uint8)])
def test_bounds_past_32_bits(max_kv, ws):
    """A table may cover them; the library would see their low 32 bits."""
    c, wide = cache(), dict(ATTEND, table=WIDE, max_kv=max_kv, ws=ws)
    refused("fit", c.attend, **wide)
    refused("fit", c.attend, **wide, window=9)
    refused("fit", c.attend_shared, **wide, group_start=i(2), prefix_len=i(1), max_prefix=16, max_own=48)
    refused("fit", c.read, table=WIDE, start=i(3), k_out=f(3, 128), v_out=f(3, 128), max_len=max_kv, ws=ws)


def test_sinks_are_checked_without_a_window_too():
    c = cache()
    refused("sinks", c.attend, **ATTEND, sinks=-1)
    refused("sinks", c.attend_workspace_bytes, n_heads=4, T=3, B=2, max_q=2, max_kv=64, sinks=-1)
    refused("sinks", wal.attn_prompt, q=f(3, 256), k=f(3, 128), v=f(3, 128), start=i(2), out=f(3, 256), head_dim=64, max_len=3, sinks=-1)
    # without a window every key is seen, the first ones among them: the size is that of the call without them
    assert c.attend_workspace_bytes(4, 3, 2, 2, 64, sinks=4) == c.attend_workspace_bytes(4, 3, 2, 2, 64)
