"""Refusals of the serving operators, before anything is launched (no GPU)."""
import ctypes
import math

import pytest
import torch

from oracle import serving as O
from block_diffusion_speculative_fuse_gb300 import _build, binding as B

P = ctypes.c_void_p(0x1000)     # never dereferenced: every call below fails its checks
WS = ctypes.c_void_p(1 << 20)
WS_N = 1 << 16


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return B.load()


def heads(**kw):
    d = dict(n_layers=2, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, kv_terms=1)
    d.update(kw)
    return B.DflashHeads(**d)


def cache(**kw):
    d = dict(pool=0x1000, page_table=0x1000, n_pages=8, max_pages=4, n_rows=4, dtype=0, scales=None)
    d.update(kw)
    return B.DflashKV(**d)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot", [0, 16, 64, 128])
def test_rope_init_matches_the_oracle(lib, scaling, rot):
    r = B.dflash_rope_init(rot, rot == 64, base=5e5, scaling=scaling, factor=3.5, orig_ctx=4096)
    f, mag = O.rope_freqs(rot, 5e5, scaling, 3.5, 4096) if rot else ([], None)
    assert r.rot_dim == rot and r.interleaved == int(rot == 64)
    for p in range(rot // 2):
        assert math.isclose(r.inv_freq[p], f[p], rel_tol=1e-12)
    if rot:
        assert math.isclose(r.mscale, mag, rel_tol=1e-15)


def test_rope_init_refuses(lib):
    ok = dict(rot_dim=64, base=1e4, scaling="yarn", factor=2.0, orig_ctx=4096)
    for bad, code in ((dict(rot_dim=24), -2), (dict(rot_dim=144), -2), (dict(rot_dim=-16), -2),
                      (dict(base=1.0), -1), (dict(base=math.nan), -1), (dict(factor=0.5), -1),
                      (dict(factor=math.inf), -1), (dict(orig_ctx=0), -1), (dict(beta_slow=0.0), -1),
                      (dict(beta_fast=1.0), -1), (dict(scaling="other"), -1)):
        with pytest.raises(B.DflashError) as e:
            B.dflash_rope_init(**{**ok, **bad})
        assert e.value.code == code, bad


def append(lib, hd=None, rope=None, layer=0, q=P, ldq=512, k=P, ldk=128, v=P, ldv=128, dt=0, qn=None,
           kn=None, eps=1e-6, req=P, pos=P, T=3, qo=ctypes.c_void_p(0x9000), ldqo=512, kv=None, ws=WS, n=WS_N):
    hd, kv = hd or heads(), kv or cache()
    rope = rope or B.dflash_rope_init(64)
    return lib.dflash_kv_rope_append(ctypes.byref(hd), ctypes.byref(rope), layer, q, ldq, k, ldk, v, ldv,
                                     dt, qn, kn, eps, req, pos, T, qo, ldqo, ctypes.byref(kv), ws, n, None)


def test_append_refuses(lib):
    odd = ctypes.c_void_p(0x1008)
    neg = B.dflash_rope_init(64)
    neg.inv_freq[3] = -1.0
    inf = B.dflash_rope_init(64)
    inf.mscale = math.inf
    for kw, code in ((dict(hd=heads(head_dim=80)), -2), (dict(hd=heads(page_size=32)), -2),
                     (dict(hd=heads(n_q_heads=7)), -2), (dict(hd=heads(n_q_heads=64)), -2),
                     (dict(hd=heads(kv_terms=3)), -2), (dict(hd=heads(n_layers=0)), -1),
                     (dict(layer=2), -1), (dict(layer=-1), -1), (dict(k=None), -1), (dict(v=odd), -1),
                     (dict(ldk=120), -1), (dict(ldv=132), -1), (dict(ldq=504), -1), (dict(qo=None), -1),
                     (dict(q=None), -1), (dict(qo=P, ldqo=520), -1), (dict(qo=P, dt=1), -1),
                     (dict(dt=2), -1), (dict(T=0), -1), (dict(eps=math.nan), -1), (dict(kn=odd), -1),
                     (dict(rope=B.dflash_rope_init(128)), -2), (dict(rope=neg), -1), (dict(rope=inf), -1),
                     (dict(kv=cache(dtype=2)), -1), (dict(kv=cache(dtype=1)), -1),
                     (dict(kv=cache(pool=0x1008)), -1), (dict(kv=cache(n_rows=0)), -1),
                     (dict(kv=cache(dtype=1, scales=0x1000), hd=heads(kv_terms=2)), -2),
                     (dict(kv=cache(max_pages=(1 << 26) + 1)), -2),
                     (dict(ws=None), -1), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), -1), (dict(n=1024), -3)):
        assert append(lib, **kw) == code, kw
    assert lib.dflash_kv_rope_append(None, None, 0, P, 512, P, 128, P, 128, 0, None, None, 0.0, P, P, 3, P,
                                     512, None, WS, WS_N, None) == -1


def attend(lib, hd=None, layer=0, q=P, batch=4, n=2, group=2, causal=1, scale=0.0, kv=None, ctx=P, pre=P,
           out=P, lse=P, ws=WS, size=1 << 40):
    hd, kv = hd or heads(), kv or cache()
    return lib.dflash_attention_prefix(ctypes.byref(hd), layer, q, batch, n, group, causal, scale,
                                       ctypes.byref(kv), ctx, pre, out, lse, ws, size, None)


def test_attention_refuses(lib):
    for kw, code in ((dict(batch=0), -1), (dict(group=3), -1), (dict(group=0), -1), (dict(n=0), -1),
                     (dict(n=33), -1), (dict(batch=1026, group=2), -1), (dict(causal=2), -1),
                     (dict(scale=-1.0), -1), (dict(scale=math.nan), -1), (dict(q=None), -1),
                     (dict(out=ctypes.c_void_p(0x1008)), -1), (dict(ctx=None), -1), (dict(pre=None), -1),
                     (dict(layer=2), -1), (dict(kv=cache(n_rows=3)), -3),
                     (dict(kv=cache(dtype=1, scales=0x1000)), -2), (dict(hd=heads(kv_terms=2)), -2),
                     (dict(hd=heads(head_dim=96)), -2),
                     (dict(kv=cache(max_pages=1 << 26, n_rows=1024), batch=1024, n=1), -2),
                     (dict(ws=ctypes.c_void_p((1 << 20) + 128)), -1), (dict(size=WS_N), -3)):
        assert attend(lib, **kw) == code, kw
    hd = heads()
    need = lib.dflash_attention_prefix_bytes(ctypes.byref(hd), 4, 2, 2)
    assert need > WS_N and attend(lib, size=need - 1) == -3
    assert lib.dflash_attention_prefix_bytes(ctypes.byref(hd), 4, 2, 3) == 0
    assert lib.dflash_attention_prefix_bytes(None, 4, 2, 2) == 0


def sample(lib, z=P, ld=100, rows=2, vocab=100, T=P, k=P, p=P, m=P, a=P, tok=P, kept=P, lp=P, ws=WS, n=WS_N):
    return lib.dflash_sample_filtered(z, ld, rows, vocab, T, k, p, m, a, tok, kept, lp, ws, n, None)


def test_sample_refuses(lib):
    for kw, code in ((dict(z=None), -1), (dict(ld=99), -1), (dict(rows=0), -1), (dict(vocab=0), -1),
                     (dict(T=None), -1), (dict(a=None), -1), (dict(a=ctypes.c_void_p(0x1004)), -1),
                     (dict(tok=None), -1), (dict(kept=ctypes.c_void_p(0x1002)), -1),
                     (dict(vocab=393217, ld=393217), -2), (dict(rows=(1 << 24) + 1), -2),
                     (dict(ws=None), -1), (dict(n=WS_N - 1), -3)):
        assert sample(lib, **kw) == code, kw
    assert lib.dflash_sample_filtered_bytes(0, 5) == 0
    assert lib.dflash_sample_filtered_bytes(5, 393217) == 0
    assert lib.dflash_sample_filtered_bytes(5, 100) == WS_N


def test_binding_refuses_tensors_the_library_would_misread(lib):
    t = torch.zeros(4, 100)          # not on a CUDA device
    with pytest.raises(B.DflashError):
        B.dflash_sample_filtered(t, 4, 100, t[:, 0], None, None, None, t[:, 0], t[:, 0], None, None, t)
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(B.DflashError):
        B.dflash_kv_rope_append(heads(), B.dflash_rope_init(64), 0, x, x[:, :2], x[:, :2], None, None, 2, x,
                                cache(), None)
    with pytest.raises(B.DflashError):
        B.dflash_attention_prefix(heads(), 0, x, 4, 2, 3, True, 0.0, cache(), None, None, x, None, None)
