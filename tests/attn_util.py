"""Inputs and tolerances of the attention tests."""
import numpy as np
import torch

from oracle import attn_oracle as ao

TYPES = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def bf16(x):
    """float64 -> the nearest bf16 values, as float64."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().double().numpy()


def pages_of(rng, lens, page, spare=3):
    """A page table that deals pages out in random order: (table [B, most], number of pages)."""
    need = [-(-n // page) for n in lens]
    deal = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1)), -7, np.int32)  # entries nobody may look at
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = deal[at:at + n]
        at += n
    return table, sum(need) + spare


def random_cache(rng, lens, page, heads, D, typ, spread=1.0, garbage=True):
    """A cache of sequences of `lens` tokens.  Returns (tensors on the CPU:
    k, v, k_scale, v_scale), the table and the float64 values k, v of every
    sequence.  Slots of no token hold NaN (bf16), any code and NaN scales."""
    table, n_pages = pages_of(rng, lens, page)
    shape = (n_pages, heads, page, D)
    out, vals = [], []
    for mul in (spread, 1.0):
        if typ == "bf16":
            x = torch.full(shape, float("nan") if garbage else 0.0, dtype=torch.bfloat16)
            x_val, scale = None, None
        else:
            codes = rng.integers(-127, 128, shape) if typ == "int8" else rng.integers(0, 254, shape) // 2 * 2 % 252
            if typ == "e4m3":
                codes = np.where(rng.random(shape) < 0.5, codes % 127, 128 + codes % 127)  # finite codes only
                x_val, norm = ao.e4m3_values(codes), 150.0
            else:
                x_val, norm = codes.astype(np.float64), 73.0
            scale = (mul / norm * np.exp(rng.normal(size=shape[:3]) * 0.3)).astype(np.float32)
            raw = torch.from_numpy(codes.astype(np.uint8))
            x = raw.view(TYPES[typ]) if typ == "e4m3" else torch.from_numpy(codes.astype(np.int8))
        used = np.zeros(shape[:3], bool)
        seqs = []
        for b, n in enumerate(lens):
            pos = np.arange(n)
            pg, off = table[b, pos // page], pos % page
            if typ == "bf16":
                val = bf16(rng.normal(size=(n, heads, D)) * mul)
                if n:
                    x[torch.from_numpy(pg.astype(np.int64)), :, torch.from_numpy(off)] = torch.from_numpy(val).bfloat16()
            else:
                val = x_val[pg, :, off] * scale[pg, :, off].astype(np.float64)[..., None]
            used[pg, :, off] = True
            seqs.append(val.reshape(n, heads, D))
        if scale is not None and garbage:
            scale = np.where(used, scale, np.float32("nan")).astype(np.float32)
        out.append((x, None if scale is None else torch.from_numpy(scale)))
        vals.append(seqs)
    (k, ks), (v, vs) = out
    return (k, v, ks, vs), table, vals[0], vals[1]


def attention_tolerance(o, a, q, k, scale):
    """Largest error of one output.  Every softmax weight is rounded to bf16
    (half a step, 2^-8; the fp16 weights of single tokens over codes are nearer)
    and carries the error of its score: D fp32 products and sums (2^-23 each,
    the tensor core may truncate) of size sum |q||k|, a product with the scale,
    and exp2 (2^-21 in all); l and the accumulator are fp32 sums over the keys
    (2^-23 each); the output is rounded to bf16.  Beside these nothing counts:
    q as fp16 is exact but for values 2^-24 below its row's largest."""
    n, heads, D = q.shape
    L = k.shape[0]
    group = heads // k.shape[1]
    size = np.stack([(np.abs(q[:, h]) @ np.abs(k[:, h // group]).T).max(1) if L else np.zeros(n) for h in range(heads)], 1)
    ds = abs(scale) * size * (D + 8) * 2.0 ** -23
    w = 2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -21 + 2 * L * 2.0 ** -23
    return (a * w) * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(o) + 1e-30


def assert_close(got, ref, tol, what=""):
    assert np.all(np.isfinite(got)), f"{what}: {np.count_nonzero(~np.isfinite(got))} outputs not finite"
    worst = float(np.max(np.abs(got - ref) / tol, initial=0.0))
    assert worst <= 1.0, f"{what}: error {worst:.3f} of the tolerance"
