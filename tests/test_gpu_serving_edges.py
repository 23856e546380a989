"""Serving operators on the GPU: calls that their documentation allows and
that once gave wrong results."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import serving as O
from test_gpu_serving import (PAGE, B_, attention_case, built, check_attention, check_rows,  # noqa: F401
                              heads, i32, workspace)

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


# ----------------------------------------------------------------- sampling
CANCEL = [  # largest logit, temperature, min_p (found by search): m + T ln min_p is 0 in double precision
    ("0x1.3c68dep+1", "0x1.19999ap-1", "0x1.6e0b3p-7"), ("0x1.1df886p+3", "0x1.8p-1", "0x1.c0b5c6p-18"),
    ("0x1.94c292p+0", "0x1.733334p+0", "0x1.58250cp-2"), ("0x1.c47a38p+2", "0x1.e66666p-1", "0x1.3345a6p-11"),
    ("0x1.014df8p+4", "0x1.19999ap+0", "0x1.e08158p-22"),
]


@pytest.mark.parametrize("vocab", [300, 40000])
def test_sample_min_p_border_at_a_logit_of_zero(vocab):
    """The differences from the largest logit of hundreds of millions of floats
    around 0 round to the border; it is found in a bounded number of steps."""
    m, T, mp = (np.array([float.fromhex(c[i]) for c in CANCEL]) for i in range(3))
    assert np.array_equal(m, m.astype(np.float32)) and np.all(np.abs(m + T * np.log(mp)) <= 2.0 ** -52 * m)
    g = np.random.default_rng(31)
    rows = len(CANCEL)
    z = (g.standard_normal((rows, vocab)) * 0.5).astype(np.float32)
    z = np.minimum(z, (m[:, None] * 0.9).astype(np.float32))
    # close to the border, but farther than the double's rounding
    z[:, 10:30] = np.geomspace(1e-9, 1e-5, 20) * np.where(np.arange(20) % 2, 1, -1)
    z[:, 7] = m
    check_rows(z, T, None, None, mp)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    B = B_()
    zt, out = torch.from_numpy(z).cuda(), torch.empty(rows, dtype=torch.int32, device="cuda")
    to = lambda x, t: torch.from_numpy(x.astype(t)).cuda()  # noqa: E731
    args = (to(T, np.float32), None, None, to(mp, np.float32), to(np.full(rows, 0.3), np.float64))
    ws = workspace(B.dflash_sample_filtered_bytes(rows, vocab))
    torch.cuda.synchronize()
    start.record()
    B.dflash_sample_filtered(zt, rows, vocab, *args, out, None, None, ws)
    end.record()
    end.synchronize()
    # 6 10^8 steps of an fp64 subtraction would take seconds, a bounded search microseconds
    assert start.elapsed_time(end) < 50.0


# --------------------------------------------------------------- generation
def tiny_model():
    import workload as W
    from block_diffusion_speculative_fuse_gb300.device import DeviceModel
    t = W.get_workload("tiny_e2e").target
    return t, DeviceModel(t, W.target_weights(t, 71, std=0.05), W.shared_weights(t, 71, std=0.05), draft=False)


@pytest.mark.parametrize("where", [[0], [-1], [0, -1]])     # in the prompt's own pass, in the first step, in both
def test_sampled_generation_reports_the_target_forwards_errors(where):
    from block_diffusion_speculative_fuse_gb300.generate import TargetRunner, sample_generate
    t, model = tiny_model()
    good = np.random.default_rng(2).integers(0, t.vocab, (2, 5)).astype(np.int32)
    u = np.random.default_rng(3).random((2, 3))
    runner = TargetRunner(model, 2, 32, 5)
    want = sample_generate(runner, good, 3, u)
    bad = good.copy()
    bad[1, where] = t.vocab                    # no such token: recorded, token 0 in its place
    with pytest.raises(B_().DflashError) as e:
        sample_generate(runner, bad, 3, u)
    assert e.value.code == -1 and "302" in str(e.value)
    assert np.array_equal(sample_generate(runner, good, 3, u), want)


def test_sampled_generation_fills_the_runner_and_no_more():
    from block_diffusion_speculative_fuse_gb300.generate import TargetRunner, sample_generate
    t, model = tiny_model()
    prompts = np.random.default_rng(2).integers(0, t.vocab, (2, 5)).astype(np.int32)
    u = np.random.default_rng(3).random((2, 29))
    want = sample_generate(TargetRunner(model, 2, 64, 5), prompts, 28, u)
    runner = TargetRunner(model, 2, 32, 5)     # positions 0 .. 31: the last token's is not needed
    assert np.array_equal(sample_generate(runner, prompts, 28, u), want)
    with pytest.raises(B_().DflashError) as e:
        sample_generate(runner, prompts, 29, u)
    assert e.value.code == -3


# ------------------------------------------------------------------- append
def test_append_angles_of_far_positions_and_high_frequencies():
    """The angle pos * inv_freq modulo a turn, where pos * inv_freq passes what a
    double holds: frequencies of up to 1e9, positions of up to 2^24."""
    B = B_()
    T, d, cols = 48, 128, 1 << 20
    g = np.random.default_rng(41)
    rope = B.dflash_rope_init(d)
    f = np.concatenate((10.0 ** g.uniform(3, 9, 40), 10.0 ** g.uniform(-6, 3, 20), [0.0, 1e9, 2 * math.pi, 1.0]))
    for p, x in enumerate(f):
        rope.inv_freq[p] = float(x)
    pos = np.concatenate(([0, 1, cols * PAGE - 1], g.integers(1 << 20, cols * PAGE, T - 3)))
    # a pool page for every table column that is used
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    used = sorted({int(p) // PAGE for p in pos})
    table[0, torch.tensor(used).cuda()] = torch.arange(len(used), dtype=torch.int32, device="cuda")
    pool = torch.zeros(1, len(used), 4, 1, PAGE, d, dtype=torch.bfloat16, device="cuda")
    kv = B.DflashKV(pool=pool.data_ptr(), page_table=table.data_ptr(), n_pages=len(used), max_pages=cols, n_rows=1,
                    dtype=0, scales=None)
    k = torch.zeros(T, 1, d, device="cuda")
    k[..., :d // 2] = 1.0                      # (1, 0) turns to (cos, sin)
    ws = workspace()
    B.dflash_kv_rope_append(heads(1, 1, 1, d, 2), rope, 0, None, k, k, i32(np.zeros(T)), i32(pos), T, None, kv, ws)
    assert B.dflash_get_status(ws) == (0, 0)
    got = pool.double().cpu().numpy()
    turn = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    for t, at in enumerate(pos):
        page, slot = used.index(int(at) // PAGE), at % PAGE
        x = got[0, page, 0, 0, slot] + got[0, page, 2, 0, slot]
        part = [Fraction(float(v)) * int(at) / turn for v in f]
        a = np.array([float((q - math.floor(q)) * turn) for q in part])
        # two bf16 terms: 2^-16 of the value; the angle: 2^-22 rad
        assert np.all(np.abs(x[:d // 2] - np.cos(a)) <= 2.0 ** -16 * np.abs(np.cos(a)) + 2.0 ** -21), at
        assert np.all(np.abs(x[d // 2:] - np.sin(a)) <= 2.0 ** -16 * np.abs(np.sin(a)) + 2.0 ** -21), at


@pytest.mark.parametrize("vocab,rows", [(50001, 96), (151936, 200), (300001, 90)])
def test_sample_rows_of_a_wide_batch_are_those_of_single_calls(vocab, rows):
    """Bit for bit, for batches so wide that a row is one CTA's and is read again
    in every pass (more than 85 rows a round of SMs, of more than 40960 tokens),
    against calls in which a cluster holds it: all settings, flat, peaked and tied
    logits, holes."""
    B = B_()
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rnd = np.random.default_rng(vocab)
    z = torch.randn(rows, vocab, generator=g, device="cuda") * torch.linspace(0.2, 5.0, rows, device="cuda")[:, None]
    z[::7] = torch.round(z[::7])
    z[3::9, ::3] = float("-inf")
    z[5] = 0.25
    to = lambda x, t: torch.from_numpy(np.asarray(x).astype(t)).cuda()  # noqa: E731
    pick = lambda xs: np.array(xs)[rnd.integers(0, len(xs), rows)]      # noqa: E731
    T = to(pick([0.0, 0.5, 0.8, 1.0, 1.3]), np.float32)
    k = to(pick([0, 0, 1, 50, 200, 300, 20000, vocab]), np.int32)
    p = to(pick([1.0, 1.0, 0.3, 0.9, 0.95, 0.999]), np.float32)
    m = to(pick([0.0, 0.0, 0.02, 1e-6]), np.float32)
    a = to(rnd.random(rows), np.float64)
    ws = workspace(B.dflash_sample_filtered_bytes(rows, vocab))

    def call(i, n):
        out = [torch.empty(n, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
        s = slice(i, i + n)
        B.dflash_sample_filtered(z[s], n, vocab, T[s], k[s], p[s], m[s], a[s], *out, ws)
        return out
    wide = call(0, rows)
    single = [torch.cat(x) for x in zip(*(call(i, 1) for i in range(rows)))]
    for x, y in zip(wide, single):
        assert torch.equal(x, y)
    assert B.dflash_get_status(ws) == (0, 0)


@pytest.mark.parametrize("d,rot,inter,norm", [(128, 128, False, True), (64, 48, True, True), (128, 64, False, False)])
def test_append_error_of_the_norm_and_the_rotation(d, rot, inter, norm):
    """Two-term store of fp32 rows.  In units of 2^-24 of the pair's magnitude:
    the angle 3.4 (2^-22.2 rad), sine and cosine 2, mscale 1, the rotation 3;
    with a norm the mean square's 8 (up to 20 roundings, halved by the root),
    its inverse root 4 and two products 2: 24 in all, below 2^-19; the store
    2^-16 of the value."""
    B = B_()
    T, hkv = 300, 4
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    k, v = (5 * torch.randn(T, hkv, d, generator=g, device="cuda") for _ in range(2))
    gain = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    pages = (T + PAGE - 1) // PAGE
    pool = torch.zeros(1, pages, 4, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    kv = B.DflashKV(pool=pool.data_ptr(), page_table=table.data_ptr(), n_pages=pages, max_pages=pages, n_rows=1,
                    dtype=0, scales=None)
    rope = B.dflash_rope_init(rot, inter, scaling="yarn", factor=4.0, orig_ctx=256)
    ws = workspace()
    B.dflash_kv_rope_append(heads(1, 4, hkv, d, 2), rope, 0, None, k, v, i32(np.zeros(T)), i32(np.arange(T)), T, None,
                            kv, ws, k_norm=gain if norm else None)
    assert B.dflash_get_status(ws) == (0, 0)
    got = pool.double().cpu().numpy()[0].transpose(1, 0, 3, 2, 4).reshape(4, -1, hkv, d)[:, :T]
    x = k.double().cpu().numpy()
    if norm:
        x = O.rms_norm(x, gain.double().cpu().numpy(), float(np.float32(1e-6)))
    f, mag = O.rope_freqs(rot, 1e6, "yarn", 4.0, 256)
    e = O.rotate(x, np.arange(T), f, mag, inter)
    size = np.abs(x)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    size[..., a] = size[..., b] = mag * np.hypot(x[..., a], x[..., b])
    assert np.all(np.abs(got[0] + got[2] - e) <= 2.0 ** -16 * np.abs(e) + 2.0 ** -19 * size)
    vd = v.double().cpu().numpy()
    assert np.all(np.abs(got[1] + got[3] - vd) <= 2.0 ** -16 * np.abs(vd))
