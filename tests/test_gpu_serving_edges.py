"""Serving operators on the GPU: calls that their documentation allows and
that once gave wrong results."""
import numpy as np
import pytest
import torch

from test_gpu_serving import PAGE, B_, attention_case, built, check_attention  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- attention
NOT_FINITE = [  # batch, n, group, hq, hkv, d, prefix per group, ctx
    (2, 5, 2, 8, 4, 64, [160], [165, 400]),                 # small tiles
    (3, 2, 1, 4, 4, 128, [0] * 3, [2, 17, 300]),
    (2, 32, 1, 4, 4, 128, [0, 0], [130, 20]),               # 31 such keys, on three pages; rows before the start
    (3, 16, 3, 8, 2, 128, [300], [316, 700, 421]),          # large tiles, 64 rows; the keys span two chunks of 128
    (2, 9, 2, 12, 2, 64, [2048], [2300, 2057]),             # 54 rows
    (2, 32, 1, 8, 1, 64, [0, 0], [500, 141]),               # 256 rows: two tiles over the same keys
    (1, 32, 1, 16, 1, 128, [0], [5000]),                    # 512 rows, many ranges
    (6, 16, 6, 16, 2, 128, [640], [656 + 23 * i for i in range(6)]),   # 128 rows, a shared prefix of 768
]


@pytest.mark.parametrize("batch,n,group,hq,hkv,d,prefix,ctx", NOT_FINITE)
def test_attention_keys_that_only_later_rows_see_may_hold_anything(batch, n, group, hq, hkv, d, prefix, ctx):
    """An infinity or NaN in K or V of a block row's own position changes no
    bit of the rows before it, nor of other heads and requests; the rows that
    see it in V are not finite."""
    B = B_()
    s = attention_case(batch, n, group, hq, hkv, d, True, prefix, ctx, seed=n)
    check_attention(s, batch, n, hq, d, True, ctx)
    out, lse, pool = s["out"].clone(), s["lse"].clone(), s["c"].pool.clone()
    G = hq // hkv
    bad = [float("nan"), float("inf"), float("-inf")]
    tries = 0
    for r in range(batch):
        for back in sorted({1, n // 2, n - 1}):             # key ctx - back: of block row n - back
            pos = ctx[r] - back
            if back < 1 or pos < 0:
                continue
            for plane in (0, 1):
                h, col = (r + back) % hkv, (7 * back + 3 * r) % d
                s["c"].pool.copy_(pool)
                s["c"].pool[0, s["ids"][r][pos // PAGE], plane, h, pos % PAGE, col] = bad[tries % 3]
                tries += 1
                B.dflash_attention_prefix(*s["args"])
                sees = torch.zeros(batch, n, hq, dtype=torch.bool, device="cuda")
                sees[r, n - back:, h * G:(h + 1) * G] = True
                assert torch.equal(s["out"][~sees], out[~sees]), (r, back, plane)
                assert torch.equal(s["lse"][~sees], lse[~sees]), (r, back, plane)
                if plane == 1:
                    assert not torch.isfinite(s["out"][sees]).all(-1).any(), (r, back)
    assert tries > 0 and B.dflash_get_status(s["ws"]) == (0, 0)
