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
