"""Operators of a long prompt without a GPU: refusals and bounds found by reading."""
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from block_diffusion_speculative_fuse_gb300 import _build, binding as B
from block_diffusion_speculative_fuse_gb300.device import PagedKV
from test_prompt_abi_cpu import chunk, evict, mass
from test_serving_abi_cpu import cache, heads


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return B.load()


# ------------------------------------------------- eviction between two caches
def paged(n_pages=4, dtype="bf16", **kw):
    shape = dict(n_layers=2, n_kv_heads=2, head_dim=64, kv_terms=1)
    shape.update(kw)
    return PagedKV(SimpleNamespace(**shape), np.zeros((2, 2), np.int32), n_pages, device="cpu", dtype=dtype)


def test_evict_to_refuses_caches_of_another_geometry(monkeypatch):
    """The call has one geometry for both caches: a second one would be written by the first's
    strides."""
    calls = []
    monkeypatch.setattr(B, "dflash_kv_evict", lambda *a: calls.append(a))
    i, m = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, 32)
    for src, dst in ((dict(), dict(n_layers=1)), (dict(), dict(n_layers=3)), (dict(kv_terms=2), dict()),
                     (dict(), dict(kv_terms=2)), (dict(), dict(n_kv_heads=1)), (dict(), dict(head_dim=128)),
                     (dict(head_dim=128), dict()), (dict(), dict(dtype="e4m3")), (dict(dtype="e4m3"), dict())):
        with pytest.raises(ValueError):
            paged(**src).evict_to(paged(**dst), 0, i, i, m, i, None)
    assert not calls
    for kw in (dict(), dict(kv_terms=2), dict(dtype="e4m3")):     # another number of pages is another cache's right
        paged(**kw).evict_to(paged(n_pages=9, **kw), 1, i, i, m, i, None)
    assert len(calls) == 3


def test_evict_refuses_more_heads_than_a_grid_has_rows(lib):
    """An error launches nothing: one head more than the copy's grid takes is refused before the
    choice has written its outputs."""
    many = dict(n_q_heads=65536, n_kv_heads=65536)
    assert evict(lib, hd=heads(**many), dst=cache(pool=1 << 40)) == -2
    assert evict(lib, hd=heads(n_q_heads=65535, n_kv_heads=65535), dst=cache(pool=1 << 40), size=0) == -3
    hd = heads(**many)
    assert lib.dflash_kv_evict_bytes(ctypes.byref(hd), 4, 8) == 0


def test_evict_refuses_two_pools_that_share_their_scales(lib):
    """E4M3 caches apart from each other have scales apart from each other too (2 layers of 8
    pages, 2 planes, 2 heads and 16 positions: 4096 bytes)."""
    src = cache(dtype=1, scales=1 << 30)
    size = 2 * 8 * 2 * 2 * 16 * 4
    for at, code in (((1 << 30), -1), ((1 << 30) + size - 16, -1), ((1 << 30) - size + 16, -1),
                     ((1 << 30) + size, -3), ((1 << 30) - size, -3)):
        assert evict(lib, src=src, dst=cache(pool=1 << 40, dtype=1, scales=at), size=0) == code, at - (1 << 30)


# ------------------------------------------------------- bounds that the header states
def test_chunk_workspace_by_tiles(lib):
    """At most 41 MB for fewer than 8 tiles of rows, 324 MB from 32 tiles on."""
    for hq, hkv, d in ((32, 8, 128), (15, 3, 128), (2, 2, 128), (16, 1, 64)):
        hd = heads(n_q_heads=hq, n_kv_heads=hkv, head_dim=d)
        tokens = 128 // (hq // hkv)
        size = lambda T: lib.dflash_attention_chunk_bytes(ctypes.byref(hd), 3, T)  # noqa: E731
        assert size(8 * tokens - 1) <= 41e6
        for tiles, phases in ((1, 1), (8, 2), (16, 4), (32, 8), (1000, 8)):
            # two slots of 256 rows, or of a single tile's, for each of 152 workers and round
            rows = 2 * 152 * phases * (256 if tiles > 1 else tokens * (hq // hkv))
            assert rows * (d + 2) * 4 <= size(tiles * tokens) - (1 << 16) <= rows * (d + 2) * 4 + 4 * 8 * 152 * 32
        assert size(32 * tokens - 1) < size(32 * tokens) == size(10000 * tokens) <= 324e6


def test_chunk_refuses_work_by_the_stated_formula(lib):
    """(T / (2 * (128 / G)) + batch) * n_kv_heads * (max_pages / 2 + 11) = 2^30, short tables too."""
    for max_pages, batch, hq, hkv in ((1, 4, 1024, 1024), (10, 5, 64, 64), (21, 100, 24, 8), (1 << 20, 3, 32, 8), (1 << 26, 7, 3, 1)):
        G = hq // hkv
        units = int((1 << 30) // (hkv * (max_pages / 2 + 11)))      # the largest count below the bound
        units -= units * hkv * (max_pages / 2 + 11) >= 1 << 30
        if units < batch:
            T, codes = 1, (-2, -2)
        else:
            T, codes = (units - batch + 1) * 2 * (128 // G) - 1, (-3, -2)   # the last row count with these units
        for t, code in zip((T, T + 1), codes):
            hd, kv = heads(n_q_heads=hq, n_kv_heads=hkv), cache(max_pages=max_pages, n_rows=batch)
            assert chunk(lib, hd=hd, kv=kv, batch=batch, T=t, ldq=hq * 64, ldo=hq * 64, size=0) == code, (max_pages, t)


def test_mass_refuses_work_by_the_stated_formula(lib):
    """batch * n_kv_heads * (max_pages / 16 + 1) = 2^30."""
    hd = heads(n_q_heads=65536, n_kv_heads=65536)
    for max_pages, code in ((239, -3), (240, -2)):
        kv = cache(max_pages=max_pages, n_rows=1024)
        assert mass(lib, hd=hd, kv=kv, batch=1024, ldq=65536 * 64, size=0) == code, max_pages
