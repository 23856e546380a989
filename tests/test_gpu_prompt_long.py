"""Chunk attention over more keys than L2 holds, where the work is taken in several
rounds, against 64-bit rows.

Tolerance (half a step of a rounding: bf16 2^-8, fp32 2^-24): probabilities rounded to
bf16 (2^-8 of sum p |v|), the output rounded (2^-8), the scores' fp32 error (a sum of d
products loses at most d 2^-24 of sum |q k|, which moves every p by that much), and at most
2000 additions of partial sums one after the other (2000 2^-24 of sum p |v|).
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_prompt import PAGE, B_, built, heads, i32, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

LONG = [  # rows, lengths, hq, hkv, d, rows of the call
    ([1100, 1, 930], [50001, 3001, 49007], 16, 4, 128, 2040),  # cut within heads and between requests
    ([900, 33, 1100], [99990, 99000, 40], 8, 8, 64, 2048),     # one long request of eight heads
    ([257], [4010000], 1, 1, 64, 2050),    # two units, each over hundreds of ranges
    ([1, 257, 0, 2], [777, 4000123, 0, 130], 2, 1, 64, 1100),  # the same behind single rows, 128 rows to a unit
]


@pytest.mark.parametrize("ns,ctx,hq,hkv,d,T", LONG)
def test_chunk_over_more_keys_than_l2(ns, ctx, hq, hkv, d, T):
    B = B_()
    need = [(n + PAGE - 1) // PAGE for n in ctx]
    pages, width = sum(need), max(need)
    g = torch.Generator(device="cuda").manual_seed(d + hkv)
    perm = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((len(ns), width), -7, dtype=torch.int32, device="cuda")
    ids = list(perm.split(need))
    pool = torch.empty(1, pages, 2, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
    pool.normal_(generator=g)
    for r, p in enumerate(ids):
        table[r, :need[r]] = p.int()
        # column c of V is large in the c-th of d stretches: a stretch left out or taken twice shows
        at = torch.arange(need[r] * PAGE, device="cuda") * d // max(1, ctx[r])
        big = torch.nn.functional.one_hot(at.clamp(max=d - 1), d).to(torch.bfloat16) * d
        pool[0, p, 1] += big.view(need[r], 1, PAGE, d)
    kv = B.DflashKV(pool=pool.data_ptr(), page_table=table.data_ptr(), n_pages=pages, max_pages=width,
                    n_rows=len(ns), dtype=0, scales=None)
    q = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out, lse = torch.full_like(q, 7.0), torch.full((T, hq), 7.0, device="cuda")
    start = np.concatenate([[0], np.cumsum(ns)])
    hd = heads(1, hq, hkv, d)
    ws = workspace(B.dflash_attention_chunk_bytes(hd, len(ns), T))
    args = (hd, 0, q, i32(start), len(ns), T, True, 0.0, kv, i32(ctx), out, lse, ws)
    B.dflash_attention_chunk(*args)
    assert B.dflash_get_status(ws) == (0, 0)
    first = out.clone()
    B.dflash_attention_chunk(*args)
    assert torch.equal(first, out)
    assert torch.all(out[start[-1]:] == 7.0) and torch.all(lse[start[-1]:] == 7.0)
    scale, G = 1.0 / math.sqrt(d), hq // hkv
    for r, n in enumerate(ns):
        if n == 0:
            continue
        rows = sorted({i for i in (0, 1, n // 3, n // 2, 63, 64, 127, 128, 255, 256, n - 1) if i < n})
        keys = pool[0, ids[r]].transpose(0, 1).transpose(1, 2).reshape(2, hkv, -1, d)[:, :, :ctx[r]]
        limits = torch.tensor([ctx[r] - n + i + 1 for i in rows], device="cuda")
        hidden = torch.arange(ctx[r], device="cuda")[None] >= limits[:, None]
        for h in range(hq):
            k, v = (x.double() for x in keys[:, h // G])
            qs = q[int(start[r]) + torch.tensor(rows, device="cuda"), h].double()
            s = (qs @ k.T * scale).masked_fill(hidden, -math.inf)
            want = torch.logsumexp(s, 1)
            p = torch.exp(s - want[:, None]).masked_fill(hidden, 0.0)     # (some rows see nothing)
            o, size = p @ v, p @ v.abs()
            worst = scale * float((qs.abs() @ k.abs().T).max())
            delta = (d + 16) * 2.0 ** -24 * worst + 2.0 ** -20
            tol = (2.0 ** -8 + 2 * delta + 2000 * 2.0 ** -24) * (size + o.abs())
            at = int(start[r]) + torch.tensor(rows, device="cuda")
            assert bool(torch.all((out[at, h].double() - o).abs() <= tol)), (r, h)
            gl, seen = lse[at, h].double(), limits > 0
            assert bool(torch.all(gl[~seen] == -math.inf))
            gl, want = gl[seen], want[seen]
            assert bool(torch.all((gl - want).abs() <= delta + (2.0 ** -21 + 2000 * 2.0 ** -24) * (1 + want.abs())))
