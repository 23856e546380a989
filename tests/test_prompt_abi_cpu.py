"""Refusals of the operators of a long prompt, before anything is launched, and of
score_sequences (no GPU)."""
import ctypes
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from block_diffusion_speculative_fuse_gb300 import _build, binding as B
from block_diffusion_speculative_fuse_gb300.generate import score_sequences
from test_serving_abi_cpu import P, WS, WS_N, cache, heads

BIG = 1 << 40
ODD = ctypes.c_void_p(0x1008)       # not 16-byte aligned
ODDER = ctypes.c_void_p(0x1002)     # not 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return B.load()


def chunk(lib, hd=None, layer=0, q=P, ldq=512, start=P, batch=4, T=9, causal=1, scale=0.0, kv=None, ctx=P,
          out=ctypes.c_void_p(0x9000), ldo=512, lse=P, ws=WS, size=BIG):
    hd, kv = hd or heads(), kv or cache()
    return lib.dflash_attention_chunk(ctypes.byref(hd), layer, q, ldq, start, batch, T, causal, scale,
                                      ctypes.byref(kv), ctx, out, ldo, lse, ws, size, None)


COMMON = [  # shared by the chunk attention and the mass
    (dict(batch=0), -1), (dict(T=0), -1), (dict(causal=2), -1), (dict(scale=-1.0), -1), (dict(scale=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(q=None), -1), (dict(q=ODD), -1), (dict(ldq=504), -1), (dict(ldq=516), -1),
    (dict(start=None), -1), (dict(start=ODDER), -1), (dict(ctx=None), -1), (dict(ctx=ODDER), -1), (dict(lse=ODDER), -1),
    (dict(layer=2), -1), (dict(layer=-1), -1), (dict(kv=cache(n_rows=3)), -3), (dict(kv=cache(pool=0x1008)), -1),
    (dict(kv=cache(dtype=1, scales=0x1000)), -2), (dict(hd=heads(kv_terms=2)), -2), (dict(hd=heads(head_dim=96)), -2),
    (dict(hd=heads(page_size=32)), -2), (dict(hd=heads(n_q_heads=7)), -2), (dict(hd=heads(n_layers=0)), -1),
    (dict(T=(1 << 30) + 1), -2), (dict(kv=cache(n_pages=1 << 30)), -2), (dict(kv=cache(max_pages=(1 << 26) + 1)), -2),
    (dict(ldq=1 << 38), -2), (dict(ws=None), -1), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), -1),
    (dict(size=WS_N - 1), -3)]


def test_chunk_refuses(lib):
    for kw, code in COMMON + [(dict(out=None), -1), (dict(out=ODD), -1), (dict(out=P), -1), (dict(ldo=448), -1), (dict(ldo=516), -1),
                              (dict(kv=cache(max_pages=1 << 26, n_rows=1 << 20), batch=1 << 20), -2)]:
        assert chunk(lib, **kw) == code, kw
    hd = heads()
    need = lib.dflash_attention_chunk_bytes(ctypes.byref(hd), 4, 9)
    assert need > WS_N and chunk(lib, size=need - 1) == -3
    assert lib.dflash_attention_chunk_bytes(ctypes.byref(hd), 1000, 9) == need          # the rows decide
    assert lib.dflash_attention_chunk_bytes(ctypes.byref(hd), 4, 10000) > need
    assert lib.dflash_attention_chunk_bytes(ctypes.byref(hd), 0, 9) == 0
    assert lib.dflash_attention_chunk_bytes(ctypes.byref(hd), 4, 0) == 0
    assert lib.dflash_attention_chunk_bytes(None, 4, 9) == 0


def mass(lib, hd=None, layer=0, q=P, ldq=512, start=P, batch=4, T=9, last=0, causal=1, scale=0.0, kv=None, ctx=P,
         lse=P, sums=P, ldm=64, add=1, ws=WS, size=BIG):
    hd, kv = hd or heads(), kv or cache()
    return lib.dflash_attention_mass(ctypes.byref(hd), layer, q, ldq, start, batch, T, last, causal, scale,
                                     ctypes.byref(kv), ctx, lse, sums, ldm, add, ws, size, None)


def test_mass_refuses(lib):
    for kw, code in COMMON + [(dict(lse=None), -1), (dict(sums=None), -1), (dict(sums=ODDER), -1), (dict(ldm=0), -1),
                              (dict(last=-1), -1), (dict(add=2), -1), (dict(kv=cache(n_rows=2000), batch=1025), -2),
                              (dict(kv=cache(max_pages=1 << 26, n_rows=1024), batch=1024), -2)]:
        assert mass(lib, **kw) == code, kw
    hd = heads()
    assert lib.dflash_attention_mass_bytes(ctypes.byref(hd), 4, 9) == WS_N
    assert lib.dflash_attention_mass_bytes(ctypes.byref(hd), 1025, 9) == 0
    assert lib.dflash_attention_mass_bytes(ctypes.byref(hd), 4, 0) == 0


def evict(lib, hd=None, layer=0, src=None, dst=None, batch=4, ctx=P, keep=P, sink=0, recent=0, sums=P, ldm=64,
          kept=P, ldk=8, new=ctypes.c_void_p(0x8000), out=ctypes.c_void_p(0x9000), ws=WS, size=BIG):
    hd = hd or heads()
    src, dst = src or cache(), dst or cache()
    return lib.dflash_kv_evict(ctypes.byref(hd), layer, ctypes.byref(src), ctypes.byref(dst), batch, ctx, keep, sink,
                               recent, sums, ldm, kept, ldk, new, out, ws, size, None)


def test_evict_refuses(lib):
    far = cache(pool=0x1000 + 16 * 8)           # inside the first pool
    for kw, code in ((dict(batch=0), -1), (dict(sink=-1), -1), (dict(recent=-1), -1), (dict(ctx=None), -1),
                     (dict(keep=ODDER), -1), (dict(sums=None), -1), (dict(kept=None), -1), (dict(new=ODDER), -1),
                     (dict(out=P), -1), (dict(new=P), -1), (dict(ldm=0), -1), (dict(ldk=0), -1), (dict(layer=2), -1),
                     (dict(dst=cache(n_rows=3)), -3), (dict(src=cache(n_rows=3)), -3), (dict(dst=far), -1),
                     (dict(src=far), -1), (dict(dst=cache(n_pages=7)), -1),                 # one pool, two sizes
                     (dict(dst=cache(pool=1 << 30, dtype=1, scales=0x1000)), -1),
                     (dict(src=cache(dtype=1, scales=0x1000), dst=cache(dtype=1, scales=0x2000)), -1),
                     (dict(hd=heads(head_dim=96)), -2), (dict(ldm=(1 << 30) + 1), -2),
                     (dict(src=cache(n_rows=70000), dst=cache(n_rows=70000), batch=65536), -2),
                     (dict(ws=None), -1), (dict(size=WS_N), -3)):
        assert evict(lib, **kw) == code, kw
    hd = heads()
    need = lib.dflash_kv_evict_bytes(ctypes.byref(hd), 4, 8)
    assert need > WS_N and evict(lib, size=need - 1) == -3
    for bad in ((0, 8), (65536, 8), (4, 0)):
        assert lib.dflash_kv_evict_bytes(ctypes.byref(hd), *bad) == 0


def score(lib, z=P, ld=100, rows=2, vocab=100, dt=1, T=P, ids=P, lp=P, rank=P, ent=P, n=3, ti=P, tl=P, ws=WS, size=WS_N):
    return lib.dflash_score_tokens(z, ld, rows, vocab, dt, T, ids, lp, rank, ent, n, ti, tl, ws, size, None)


def test_score_refuses(lib):
    for kw, code in ((dict(z=None), -1), (dict(z=ODDER), -1), (dict(z=ctypes.c_void_p(0x1001), dt=0), -1),
                     (dict(ld=99), -1), (dict(rows=0), -1), (dict(vocab=0), -1), (dict(dt=2), -1), (dict(T=ODDER), -1),
                     (dict(ids=None), -1), (dict(ids=None, lp=None), -1), (dict(n=-1), -1), (dict(ti=None), -1),
                     (dict(tl=None), -1), (dict(ent=ODDER), -1), (dict(n=65), -2), (dict(vocab=393217, ld=393217), -2),
                     (dict(rows=(1 << 24) + 1), -2), (dict(ws=None), -1), (dict(size=WS_N - 1), -3)):
        assert score(lib, **kw) == code, kw
    assert lib.dflash_score_tokens_bytes(5, 100, 64) == WS_N
    for bad in ((0, 5, 1), (5, 393217, 1), (5, 5, 65), (5, 5, -1)):
        assert lib.dflash_score_tokens_bytes(*bad) == 0


def test_binding_refuses_tensors_the_library_would_misread(lib):
    x = torch.zeros(4, 8, 64, dtype=torch.bfloat16)      # not on a CUDA device
    i, f = torch.zeros(5, dtype=torch.int32), torch.zeros(4, 8)
    with pytest.raises(B.DflashError):
        B.dflash_attention_chunk(heads(), 0, x, i, 4, 4, True, 0.0, cache(), i[:4], x, f, x)
    with pytest.raises(B.DflashError):
        B.dflash_attention_mass(heads(), 0, x, i, 4, 4, 0, True, 0.0, cache(), i[:4], f, torch.zeros(4, 2, 8), True, x)
    with pytest.raises(B.DflashError):
        B.dflash_kv_evict(heads(), 0, cache(), cache(), 4, i, i, 0, 0, torch.zeros(4, 2, 8), None, None, None, x)
    with pytest.raises(B.DflashError):
        B.dflash_score_tokens(f, 4, 8, None, i[:4], None, None, None, 0, None, None, f)
    for fn, args in ((B.dflash_attention_chunk_bytes, (heads(), 0, 5)), (B.dflash_attention_mass_bytes, (heads(), 5, 0)),
                     (B.dflash_kv_evict_bytes, (heads(), 5, 0)), (B.dflash_score_tokens_bytes, (5, 5, 65))):
        with pytest.raises(B.DflashError):
            fn(*args)


@pytest.mark.parametrize("tokens,kw", [(np.zeros((2, 5), np.int32), {}), (np.zeros((3, 1), np.int32), {}),
                                       (np.zeros(3, np.int32), {}), (np.zeros((3, 5), np.int32), dict(chunk=0))])
def test_score_sequences_refuses_shapes_the_target_would_misread(tokens, kw):
    runner = SimpleNamespace(batch=3, max_len=100)
    with pytest.raises(ValueError):
        score_sequences(runner, tokens, **kw)


def test_score_sequences_refuses_more_positions_than_the_runner_has():
    with pytest.raises(B.DflashError) as e:
        score_sequences(SimpleNamespace(batch=2, max_len=8), np.zeros((2, 10), np.int32))
    assert e.value.code == -3
