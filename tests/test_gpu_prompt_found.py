"""Operators of a long prompt on the GPU: cases found by reading the kernels.

Tolerances as in test_gpu_prompt.py, whose cases and comparisons these are."""
import math

import numpy as np
import pytest
import torch

from test_gpu_prompt import B_, Cache, PAGE, built, check_chunk, chunk_case, heads, i32, workspace  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_pieces_beside_those_whose_v_is_not_finite(d):
    """Requests of which every row sees every key (a single row, whole chunks of keys), each
    behind one with a V that is not finite at a key of its last row: what was found in a
    piece stays that piece's."""
    B = B_()
    many = 600
    ns = [3 if r % 2 == 0 else 1 for r in range(many)]
    ctx = [100 + r % 28 if r % 2 == 0 else 128 * (1 + r % 3) for r in range(many)]
    s = chunk_case(ns, ctx, 8, 2, d, seed=d)
    for r in range(0, many, 2):
        page, slot = divmod(ctx[r] - 1, PAGE)
        s["c"].pool[0, s["c"].ids[r][page], 1, :, slot, r % d] = math.nan
    for _ in range(3):
        s["out"].fill_(7.0)
        B.dflash_attention_chunk(*s["args"])
        torch.cuda.synchronize()
        last = torch.tensor([int(s["start"][r]) + 2 for r in range(0, many, 2)], device="cuda")
        assert not torch.isfinite(s["out"][last]).all(-1).any()
        check_chunk(s, 8, d, requests=range(1, many, 2))
