"""Serving calls that are refused on the host (no GPU)."""
import numpy as np
import pytest

from block_diffusion_speculative_fuse_gb300 import _build, binding as B
from block_diffusion_speculative_fuse_gb300.generate import sample_generate


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return B.load()


class Runner:
    """What sample_generate may look at before it does any work."""
    batch, max_len, device = 2, 16, "no such device"


def test_sampled_generation_refuses_more_positions_than_the_runner_has():
    with pytest.raises(B.DflashError) as e:
        sample_generate(Runner(), np.zeros((2, 10), np.int32), 8, np.zeros((2, 8)))
    assert e.value.code == -3


@pytest.mark.parametrize("prompts,u", [((1, 4), (1, 3)), ((3, 4), (3, 3)), ((2, 0), (2, 3)), ((2, 4), (1, 3)),
                                       ((2, 4), (3, 3)), ((2, 4), (2, 2)), ((2, 4), (6,))])
def test_sampled_generation_refuses_shapes_the_target_would_misread(prompts, u):
    """The target's forward reads and writes rows for all of the runner's requests."""
    with pytest.raises(ValueError):
        sample_generate(Runner(), np.zeros(prompts, np.int32), 3, np.zeros(u))


@pytest.mark.parametrize("batch,n,group,hq,hkv,d,rows", [
    # rows of partial results: all units', and the largest unit's for each worker
    (1024, 16, 1, 32, 8, 128, 1024 * 8 * 64 + 152 * 64),                       # large tiles, 64 rows a request
    (32, 16, 32, 32, 8, 128, 8 * 8 * 256 + 32 * 8 * 64 + 152 * 256),           # and a prefix of 2048 rows
    (32, 1, 32, 32, 8, 128, 8 * 128 + 152 * 128 + 32 * 8 * 4 + 1216 * 4),      # a large list and a small one
])
def test_attention_workspace_holds_the_units_own_rows(batch, n, group, hq, hkv, d, rows):
    heads = B.DflashHeads(n_layers=1, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=16, kv_terms=1)
    size = B.dflash_attention_prefix_bytes(heads, batch, n, group)
    partials = rows * (d + 2) * 4
    assert partials < size < partials + (1 << 17)      # and the header, the lists' offsets, alignment
