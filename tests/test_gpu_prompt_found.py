"""Operators of a long prompt on the GPU: cases found by reading the kernels.

Tolerances as in test_gpu_prompt.py, whose cases and comparisons these are."""
import math

import numpy as np
import pytest
import torch

from test_gpu_prompt import (PAGE, B_, Cache, built, check_chunk, chunk_case, heads, i32, logits,  # noqa: F401
                             mass_case, workspace)

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


def test_mass_of_a_key_that_very_many_rows_see():
    """24576 rows of 16 heads to one: the first half of them gives key 0 about all of their weight,
    the second half 0.0015 each, less than half a step of the sum that is there by then.

    Tolerance, relative: scores are exact here (one product, scale 1).  The exponent is at most
    13 (log2 e) from two products rounded to 2^-24 and one sum, its constants to 2^-24: 4 * 19 * 2^-24
    ln 2 < 53 * 2^-24 of the weight, which exp2 rounds by 2^-22 more.  A tile's 128 weights
    add up over 34 additions at most, the tiles' sums as if once."""
    B = B_()
    n, ctx, G, d = 24576, 256, 16, 64
    c = Cache(1, 1, d, [ctx], spoil=False)
    c.pool[0, :, 0] = 0.0
    c.pool[0, c.ids[0][0], 0, 0, 0, 0] = 1.0             # key 0 is e_0, the others none
    q = torch.zeros(n, G, d, dtype=torch.bfloat16, device="cuda")
    q[:n // 2, :, 0], q[n // 2:, :, 0] = 12.0, -0.9609375
    lse = torch.log(torch.exp(q[:, :, 0].double()) + ctx - 1).float()
    mass = torch.zeros(1, 1, ctx, device="cuda")
    hd = heads(1, G, 1, d)
    ws = workspace(B.dflash_attention_mass_bytes(hd, 1, n))
    B.dflash_attention_mass(hd, 0, q, i32([0, n]), 1, n, 0, False, 1.0, c.kv, i32([ctx]), lse, mass, False, ws)
    assert B.dflash_get_status(ws) == (0, 0)
    want = torch.exp(-lse.double()).sum().expand(ctx).clone()
    want[0] = torch.exp(q[:, :, 0].double() - lse.double()).sum()
    err = ((mass[0, 0].double() - want).abs() / want).max()
    assert float(err) <= (53 + 4 + 34 + 4) * 2.0 ** -24, float(err) * 2.0 ** 24


@pytest.mark.parametrize("ns,ctx,hq,hkv,d", [([5, 40, 3], [165, 300, 30], 8, 2, 64), ([300], [300], 2, 2, 128),
                                             ([33, 1], [4000, 2500], 4, 1, 128), ([1], [3001], 8, 1, 64)])
def test_lse_and_masses_do_not_depend_on_v(ns, ctx, hq, hkv, d):
    """A V that is not finite makes the rows that see it NaN and leaves their lse, and all
    masses, as they are, wherever the position is."""
    B = B_()
    s = mass_case(ns, ctx, hq, hkv, d, seed=4)
    lse, mass = s["lse"].clone(), s["mass"].clone()
    for r, (n, m) in enumerate(zip(ns, ctx)):
        for pos in sorted({m - n // 2 - 1, m - 1, m // 3}):
            page, slot = divmod(pos, PAGE)
            at = s["c"].pool[0, s["c"].ids[r][page], 1, :, slot]
            before = at.clone()
            at.fill_(math.nan if pos % 2 else math.inf)
            s["out"].fill_(7.0)
            B.dflash_attention_chunk(*s["args"])
            B.dflash_attention_mass(*s["mass_args"])
            a = int(s["start"][r])
            first = max(0, pos - (m - n))               # the first row that sees it
            assert not torch.isfinite(s["out"][a + first:a + n]).any(), (r, pos)
            assert torch.isfinite(s["out"][a:a + first]).all(), (r, pos)
            assert torch.equal(s["lse"], lse) and torch.equal(s["mass"], mass), (r, pos)
            at.copy_(before)


def test_masses_by_the_lse_of_rows_that_saw_a_bad_key():
    """A K that is not finite spoils its own mass alone by a finite lse.  The one that the
    attention leaves for the rows that see it spoils those of the whole head, none of another."""
    B = B_()
    s = mass_case([5, 40, 3], [165, 300, 30], 8, 2, 64, seed=4)
    pool, lse, mass = s["c"].pool.clone(), s["lse"].clone(), s["mass"].clone()
    for bad in (math.nan, math.inf):
        s["c"].pool.copy_(pool)
        s["c"].pool[0, s["c"].ids[1][3], 0, 1, 7] = bad          # position 55, which all 40 rows see
        B.dflash_attention_chunk(*s["args"])
        B.dflash_attention_mass(*s["mass_args"])
        spoilt = torch.zeros_like(mass, dtype=torch.bool)
        spoilt[1, 1, :300] = True
        assert torch.isnan(s["mass"][spoilt]).all()
        assert torch.equal(s["mass"][~spoilt], mass[~spoilt])
        args = list(s["mass_args"])
        args[11] = lse
        B.dflash_attention_mass(*args)
        other = torch.ones_like(spoilt)
        other[1, 1, 55] = False
        assert torch.equal(s["mass"][other], mass[other])


def test_score_records_which_of_the_two_it_was():
    """Ids beyond the vocabulary alone are site 572, bad rows alone 571; with both, one of them."""
    B = B_()
    ws = workspace()
    lp = torch.zeros(3, device="cuda")
    for ids, bad, sites in (([1, 300, 2], False, (572,)), ([2 ** 31 - 1, 1, 1], False, (572,)), ([1, 2, 3], True, (571,)),
                            ([1, 300, 2], True, (571, 572))):
        z = logits(3, 300)
        if bad:
            z[2, 7] = math.nan
        B.dflash_workspace_init(ws)
        B.dflash_score_tokens(z, 3, 300, None, i32(ids), lp, None, None, 0, None, None, ws)
        status, site = B.dflash_get_status(ws)
        assert status == -1 and site in sites, (ids, bad, site)


def test_calls_at_once_on_two_streams():
    """Each with a workspace of its own: the same bits as one after the other."""
    B = B_()
    cases = [mass_case(ns, ctx, 8, 2, d, seed=d) for ns, ctx, d in
             (([300, 1, 45], [4000, 900, 45], 64), ([1, 70], [9000, 300], 128))]
    z = logits(40, 50000)
    ids, wss = i32(np.arange(40) * 7), [workspace(), workspace()]
    lps = [torch.zeros(40, device="cuda") for _ in range(2)]

    def call(i, stream=None):
        B.dflash_attention_chunk(*cases[i]["args"], stream=stream)
        B.dflash_attention_mass(*cases[i]["mass_args"], stream=stream)
        B.dflash_score_tokens(z, 40, 50000, None, ids, lps[i], None, None, 0, None, None, wss[i], stream=stream)
    for i in range(2):
        call(i)
    torch.cuda.synchronize()
    want = [[cases[i][k].clone() for k in ("out", "lse", "mass")] + [lps[i].clone()] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip([cases[i][k] for k in ("out", "lse", "mass")] + [lps[i]], want[i]):
            assert torch.equal(a, b), i
        assert all(B.dflash_get_status(ws) == (0, 0) for ws in (cases[i]["ws"], wss[i], cases[i]["mass_args"][-1]))


def test_decoding_on_from_an_evicted_cache():
    """New rows go on from the old length's angles and behind the positions that are left, on the
    device throughout: q and k are rotated as the q heads of an append into a scratch cache (a
    page per request, which every entry of its table names), and stored by one without a
    rotation.  Against rows rotated in 64 bits (an angle to 2^-19 of the pair, k's and q's
    rounding to bf16 2^-8)."""
    B = B_()
    from oracle import serving as O
    from types import SimpleNamespace
    from block_diffusion_speculative_fuse_gb300.device import PagedKV
    hq, hkv, d, batch, layer = 8, 2, 64, 2, 1
    shape = SimpleNamespace(n_layers=2, n_kv_heads=hkv, head_dim=d, kv_terms=1)
    lens, keep, steps = [150, 61], [48, 40], 5
    big = PagedKV(shape, np.random.default_rng(0).permutation(20).reshape(2, 10), 20)
    small = PagedKV(shape, np.arange(8).reshape(2, 4), 8)
    scratch = PagedKV(SimpleNamespace(n_layers=1, n_kv_heads=hkv, head_dim=d, kv_terms=1),
                      np.repeat([[0], [1]], 10, 1), 2)
    g = torch.Generator(device="cuda").manual_seed(6)
    rope, none = B.dflash_rope_init(d, base=1e4), B.dflash_rope_init(0)
    f, mag = O.rope_freqs(d, 1e4)
    ws = big.chunk_workspace(hq, batch, 256)
    seq = [torch.randn(n + steps, hq + 2 * hkv, d, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    for r, n in enumerate(lens):
        x = seq[r][:n]
        big.append_rotated(rope, layer, None, x[:, hq:hq + hkv].contiguous(), x[:, hq + hkv:].contiguous(), i32([r] * n),
                           i32(np.arange(n)), ws)
    mass = torch.rand(batch, hkv, 160, generator=g, device="cuda")
    kept, new_len = torch.zeros(batch, hkv, 48, dtype=torch.int32, device="cuda"), i32([0, 0])
    big.evict_to(small, layer, i32(lens), i32(keep), mass, kept, small.evict_workspace(batch), new_len=new_len)
    pos, req, start = i32(lens), i32([0, 1]), i32([0, 1, 2])
    for i in range(steps):
        x = torch.stack([seq[r][lens[r] + i] for r in range(batch)])
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:].contiguous()
        qk = torch.empty(batch, hq + hkv, d, dtype=torch.bfloat16, device="cuda")
        scratch.append_rotated(rope, 0, x[:, :hq + hkv], k, v, req, pos, ws, q_out=qk)
        small.append_rotated(none, layer, None, qk[:, hq:], v, req, new_len, ws)
        new_len += 1
        pos += 1
        out = torch.zeros(batch, hq, d, dtype=torch.bfloat16, device="cuda")
        small.attend_chunk(layer, qk[:, :hq], start, new_len, out, ws)
        at = [lens[r] + i for r in range(batch)]
        qr, kr = (O.rotate(t.double().cpu().numpy(), at, f, mag, False) for t in (q, k))
        size = math.sqrt(2) * max(float(q.abs().max()), float(k.abs().max()))
        assert np.all(np.abs(qk[:, :hq].double().cpu().numpy() - qr) <= 2.0 ** -8 * np.abs(qr) + 2.0 ** -18 * size)
        for r in range(batch):
            kk, vv = (t.double().cpu().numpy() for t in small.read_logical(layer, r, keep[r] + i + 1))
            assert np.all(np.abs(kk[-1] - kr[r]) <= 2.0 ** -8 * np.abs(kr[r]) + 2.0 ** -18 * size)
            assert np.array_equal(vv[-1], v[r].double().cpu().numpy())
            o, _, mag_v = O.attend(qk[r:r + 1, :hq].double().cpu().numpy(), kk, vv, 0.125, [keep[r] + i + 1])
            assert np.all(np.abs(out[r:r + 1].double().cpu().numpy() - o) <= 2.0 ** -7 * (mag_v + np.abs(o)) + 1e-6)
    # what was kept lies before them as it lay in the old cache
    for r in range(batch):
        old, left = big.read_logical(layer, r, lens[r]), small.read_logical(layer, r, keep[r])
        for h in range(hkv):
            for a, b in zip(old, left):
                assert torch.equal(b[:, h].cpu(), a[kept[r, h, :keep[r]].long().cpu(), h].cpu())
    assert B.dflash_get_status(ws) == (0, 0)
