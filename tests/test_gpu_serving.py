"""Serving operators on the GPU against the 64-bit oracle (oracle/serving.py).

Tolerances (half a step of a rounding: bf16 2^-8, fp32 2^-24, E4M3 2^-4 or
half its smallest subnormal, 2^-10):
* append: the stored value's rounding, and 2^-19 of the pair's (or element's)
  magnitude for the fp32 norm and rotation (the angle is good to 2^-22 rad,
  the rest is a dozen fp32 roundings);
* attention: probabilities rounded to bf16 (2^-8 of sum p |v|), the output
  rounded (2^-8), and the scores' fp32 error: a sum of d products loses at
  most d 2^-24 of sum |q k|, which moves every p (and lse) by that much;
* sampling: tokens and counts are equal; logprob is one fp32 rounding of a
  value good to 1e-9.
"""
import math

import numpy as np
import pytest
import torch

from oracle import fp8, serving as O

pytestmark = pytest.mark.gpu
PAGE = 16


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_diffusion_speculative_fuse_gb300 import _build, binding
    _build.build()
    binding.load()


def B_():
    from block_diffusion_speculative_fuse_gb300 import binding
    return binding


def workspace(size=1 << 16):
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    B_().dflash_workspace_init(ws)
    return ws


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


class Cache:
    """A cache over a shuffled pool; page_ids[r]: the pages of request r."""

    def __init__(self, L, hkv, d, page_ids, n_pages, width, kind="bf16", fill=None, seed=0):
        B = B_()
        planes = 4 if kind == "two" else 2
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (L, n_pages, planes, hkv, PAGE, d)
        self.scales = None
        if kind == "e4m3":
            self.pool = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
            self.scales = torch.rand(shape[:-1], generator=g, device="cuda")
        else:
            self.pool = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
            if fill is not None:
                self.pool.fill_(fill)
        self.table = np.full((len(page_ids), width), -7, np.int32)
        for r, ids in enumerate(page_ids):
            self.table[r, :len(ids)] = ids
        self.table_d = i32(self.table)
        self.kv = B.DflashKV(pool=self.pool.data_ptr(), page_table=self.table_d.data_ptr(), n_pages=n_pages,
                             max_pages=width, n_rows=len(page_ids), dtype=1 if kind == "e4m3" else 0,
                             scales=None if self.scales is None else self.scales.data_ptr())


def heads(L, hq, hkv, d, terms=1):
    return B_().DflashHeads(n_layers=L, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=PAGE, kv_terms=terms)


# ------------------------------------------------------------------- append
APPEND = [  # T, hq, hkv, d, rot, interleaved, scaling, norm, dtype, kind
    (1, 4, 2, 64, 64, False, "none", True, torch.bfloat16, "bf16"),
    (1, 32, 8, 128, 128, True, "yarn", False, torch.bfloat16, "bf16"),
    (17, 8, 2, 128, 64, False, "linear", True, torch.float32, "two"),
    (33, 8, 8, 64, 48, True, "ntk", True, torch.bfloat16, "e4m3"),
    (40, 2, 1, 128, 16, False, "none", False, torch.float32, "e4m3"),
    (5, 16, 1, 64, 0, False, "none", True, torch.float32, "bf16"),
    (700, 48, 24, 128, 128, False, "none", True, torch.bfloat16, "two"),
    (64, 80, 40, 64, 32, True, "none", False, torch.bfloat16, "bf16"),
]


@pytest.mark.parametrize("T,hq,hkv,d,rot,inter,scaling,norm,dt,kind", APPEND)
def test_append(T, hq, hkv, d, rot, inter, scaling, norm, dt, kind):
    B = B_()
    rnd = np.random.default_rng(T * d + hq)
    g = torch.Generator(device="cuda").manual_seed(T)
    reqs, layer, L = min(T, 3), 1, 2
    far = 1 << 20   # page-table columns: positions up to 2^24
    req = rnd.integers(0, reqs, T)
    # distinct positions of each request, most of them far along
    pos = np.array([(far - 64) * PAGE + t if t % 3 else 5 + t for t in range(T)])
    dead = rnd.random(T) < 0.2 if T > 10 else np.zeros(T, bool)
    pos[dead] = -1
    used = sorted({(r, p // PAGE) for r, p in zip(req, pos) if p >= 0})
    n_pages = len(used) + 2
    perm = rnd.permutation(n_pages)
    c = Cache(L, hkv, d, [[] for _ in range(reqs)], n_pages, far, kind, seed=T + 1)
    for i, (r, col) in enumerate(used):
        c.table_d[r, col] = int(perm[i])
    qkv = (3 * torch.randn(T, (hq + 2 * hkv) * d + 8, generator=g, device="cuda")).to(dt)
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    gains = (1 + 0.3 * torch.randn(2, d, generator=g, device="cuda")).to(torch.bfloat16)
    q_out = torch.full((T, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = workspace()
    rope = B.dflash_rope_init(rot, inter, base=1e6, scaling=scaling, factor=4.0, orig_ctx=32768)
    pool0 = c.pool.clone()
    scales0 = None if c.scales is None else c.scales.clone()
    B.dflash_kv_rope_append(heads(L, hq, hkv, d, 2 if kind == "two" else 1), rope, layer, q, k, v, i32(req),
                            i32(pos), T, q_out, c.kv, ws, gains[0] if norm else None,
                            gains[1] if norm else None)
    torch.cuda.synchronize()
    assert B.dflash_get_status(ws) == (0, 0)

    f, mag = O.rope_freqs(rot, 1e6, scaling, 4.0, 32768)

    def exact(x, gain):
        x = x.double().cpu().numpy()
        if gain is None:
            return x, np.abs(x)
        if norm:
            x = O.rms_norm(x, gain.double().cpu().numpy(), 1e-6)
        y = O.rotate(x, pos, f, mag, inter)
        size = np.abs(x)                       # magnitude of the pair behind each element
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        size[..., a] = size[..., b] = mag * np.hypot(x[..., a], x[..., b])
        return y, size
    live = pos >= 0
    qe, qs = exact(q, gains[0])
    got = q_out.double().cpu().numpy()
    assert np.all(np.abs(got - qe)[live] <= (2.0 ** -8 * np.abs(qe) + 2.0 ** -18 * qs)[live])
    assert np.all(got[~live] == 9.0)
    table = c.table_d.cpu().numpy()
    pool = c.pool.cpu()
    for which, (x, gain) in enumerate(((k, gains[1]), (v, None))):
        e, size = exact(x, gain)
        for t in np.flatnonzero(live):
            page, slot = table[req[t], pos[t] // PAGE], pos[t] % PAGE
            err = 2.0 ** -18 * size[t]
            if kind == "e4m3":
                codes = pool[layer, page, which, :, slot].numpy()
                s = c.scales[layer, page, which, :, slot].double().cpu().numpy()[:, None]
                amax = np.abs(e[t]).max(-1, keepdims=True)
                assert np.all(np.abs(s * 448 - amax) <= 2.0 ** -8 * amax + err.max() + 2.0 ** -22 * amax)
                tol = 2.0 ** -4 * np.abs(e[t]) * (1 + 2.0 ** -7) + 2.0 ** -10 * s + 2.0 ** -8 * np.abs(e[t]) + 2 * err
                assert np.all(np.abs(fp8.e4m3_decode(codes) * s - e[t]) <= tol)
                continue
            got = pool[layer, page, which, :, slot].double().numpy()
            assert np.all(np.abs(got - e[t]) <= 2.0 ** -8 * np.abs(e[t]) + err)
            if kind == "two":
                low = pool[layer, page, 2 + which, :, slot].double().numpy()
                assert np.all(np.abs(got + low - e[t]) <= 2.0 ** -16 * np.abs(e[t]) + 2 * err)
    # everything else is as it was
    mask = torch.ones(pool.shape[:-1], dtype=torch.bool)
    for t in np.flatnonzero(live):
        mask[layer, table[req[t], pos[t] // PAGE], :, :, pos[t] % PAGE] = False
    assert torch.equal(pool[mask], pool0.cpu()[mask])
    if scales0 is not None:
        assert torch.equal(c.scales.cpu()[mask], scales0.cpu()[mask])


def test_append_in_place_and_keys_only():
    B = B_()
    T, hq, hkv, d = 21, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    rope = B.dflash_rope_init(128)
    req, pos = i32(np.zeros(T)), i32(np.arange(T))
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    outs = []
    for mode in ("copy", "in place", "keys only"):
        c = Cache(1, hkv, d, [[2, 0]], 3, 2, fill=0.0)
        qq = q.clone()
        q_out = torch.empty_like(q) if mode == "copy" else qq
        ws = workspace()
        none = mode == "keys only"
        B.dflash_kv_rope_append(heads(1, hq, hkv, d), rope, 0, None if none else qq, k, v, req, pos, T,
                                None if none else q_out, c.kv, ws, gain, gain)
        outs.append((q_out.clone(), c.pool.clone()))
        if none:
            assert torch.equal(qq, q)
    assert torch.equal(outs[0][0], outs[1][0])
    assert torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][1], outs[2][1])


def test_append_out_of_range_rows_are_dropped():
    B = B_()
    d, hkv = 64, 2
    c = Cache(1, hkv, d, [[1, 2], [0, 9]], 3, 2, fill=3.0)
    x = torch.randn(6, hkv, d, device="cuda").to(torch.bfloat16)
    # good; request 2 of 2; page column 2 of 2; page id 9 of 3; request -1; skipped
    req, pos = i32([0, 2, 0, 1, -1, 0]), i32([0, 0, 32, 16, 3, -5])
    ws = workspace()
    B.dflash_kv_rope_append(heads(1, hkv, hkv, d), B.dflash_rope_init(64), 0, x, x, x, req, pos, 6,
                            torch.empty_like(x), c.kv, ws)
    torch.cuda.synchronize()
    assert B.dflash_get_status(ws) == (-3, 501)
    expect = torch.full_like(c.pool, 3.0)
    expect[0, 1, :, :, 0] = x[0]     # position 0: no rotation
    assert torch.equal(c.pool, expect)


def test_append_agrees_with_the_quantizing_cache():
    """An E4M3 append stores what a bf16 append followed by the library's
    conversion stores."""
    B = B_()
    T, hkv, d = 30, 4, 128
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.randn(T, hkv, d, generator=g, device="cuda") for _ in range(2))
    req, pos = i32(np.zeros(T)), i32(np.arange(T))
    stores = {}
    for kind in ("bf16", "e4m3"):
        c = Cache(1, hkv, d, [[1, 0]], 2, 2, kind)
        B.dflash_kv_rope_append(heads(1, 4, hkv, d), B.dflash_rope_init(128), 0, None, k, v, req, pos, T,
                                None, c.kv, workspace())
        stores[kind] = c
    for t in range(T):
        page, slot = [1, 0][t // PAGE], t % PAGE
        # on the host: torch's CUDA division by a number multiplies by its reciprocal
        x = stores["bf16"].pool[0, page, :, :, slot].float().cpu()
        s = x.abs().amax(-1) / 448.0
        assert torch.equal(stores["e4m3"].scales[0, page, :, :, slot].cpu(), s)
        want = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(stores["e4m3"].pool[0, page, :, :, slot].cpu(), want)


# ---------------------------------------------------------------- attention
def attention_case(batch, n, group, hq, hkv, d, causal, prefix, ctx, layers=1, layer=0, scale=0.0, seed=0,
                   lse=True, spoil=True, table_width=None, share=None):
    """Runs one call and returns everything a check needs.  prefix per group,
    ctx per request; whole prefix pages are shared (share: pages per group,
    where the table shares fewer than prefix_len says is not allowed)."""
    B = B_()
    rnd = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids, nxt, of_group = [], 0, {}
    for r in range(batch):
        gi = r // group
        whole = prefix[gi] // PAGE
        if gi not in of_group:
            of_group[gi] = list(range(nxt, nxt + whole))
            nxt += whole
        need = max((ctx[r] + PAGE - 1) // PAGE, 0)
        extra = max(0, need - whole)
        ids.append(of_group[gi] + list(range(nxt, nxt + extra)))
        nxt += extra
    n_pages = nxt + 3
    perm = rnd.permutation(n_pages)
    ids = [[int(perm[i]) for i in row] for row in ids]
    width = table_width or max(1, max(len(i) for i in ids))
    c = Cache(layers, hkv, d, ids, n_pages, width, seed=seed + 1)
    # a prefix that ends inside a page: the same tokens in every request's own page
    for gi in range(batch // group):
        part, col = prefix[gi] % PAGE, prefix[gi] // PAGE
        rows = [r for r in range(gi * group, (gi + 1) * group) if ctx[r] > prefix[gi] - part and len(ids[r]) > col]
        for r in rows[1:]:
            c.pool[:, ids[r][col], :, :, :part] = c.pool[:, ids[rows[0]][col], :, :, :part]
    if spoil:
        # nothing at or past a context may matter
        owned = np.zeros((n_pages, PAGE), bool)
        for r in range(batch):
            for p in range(max(0, min(ctx[r], width * PAGE))):
                owned[ids[r][p // PAGE], p % PAGE] = True
        bad = torch.from_numpy(~owned).cuda()
        pool = c.pool.permute(0, 2, 3, 1, 4, 5)    # [L, planes, hkv, pages, 16, d], a view
        pool[:, :, :, bad] = float("nan")
    q = (1.3 * torch.randn(batch, n, hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    L = torch.full((batch, n, hq), 7.0, device="cuda") if lse else None
    hd = heads(layers, hq, hkv, d)
    ws = workspace(B.dflash_attention_prefix_bytes(hd, batch, n, group))
    args = (hd, layer, q, batch, n, group, causal, scale, c.kv, i32(ctx), i32(prefix), out, L, ws)
    B.dflash_attention_prefix(*args)
    torch.cuda.synchronize()
    return dict(c=c, q=q, out=out, lse=L, ws=ws, ids=ids, args=args, width=width)


def keys_of(c, ids, layer, count):
    kv = c.pool[layer, torch.tensor(ids, dtype=torch.long)[:(count + PAGE - 1) // PAGE].cuda()].double().cpu().numpy()
    kv = kv.transpose(1, 0, 3, 2, 4).reshape(2, -1, kv.shape[2], kv.shape[4])
    return kv[0, :count], kv[1, :count]


def check_attention(s, batch, n, hq, d, causal, ctx, layer=0, scale=0.0, requests=None):
    scale = scale or 1.0 / math.sqrt(d)
    for r in requests if requests is not None else range(batch):
        m = max(0, min(ctx[r], s["width"] * PAGE))
        k, v = keys_of(s["c"], s["ids"][r], layer, m)
        q = s["q"][r].double().cpu().numpy()
        limits = [m - n + i + 1 if causal else m for i in range(n)]
        o, lse, size = O.attend(q, k, v, scale, limits)
        G = hq // (k.shape[1] if m else 1)
        worst = scale * max((np.abs(q[i, h]) @ np.abs(k[:, h // G]).T).max() for i in range(n) for h in range(hq)) \
            if m else 0.0
        delta = (d + 16) * 2.0 ** -24 * worst + 2.0 ** -20
        tol = (2.0 ** -8 + 2 * delta) * size + (2.0 ** -8 + 2 * delta) * np.abs(o) + 1e-30
        got = s["out"][r].double().cpu().numpy()
        assert np.all(np.abs(got - o) <= tol), (r, float(np.max(np.abs(got - o) / tol)))
        if s["lse"] is not None:
            gl = s["lse"][r].double().cpu().numpy()
            assert np.array_equal(np.isfinite(gl), np.isfinite(lse))
            f = np.isfinite(lse)
            assert np.all(np.abs(gl[f] - lse[f]) <= delta + 2.0 ** -21 * (1 + np.abs(lse[f])))
            assert np.all(gl[~f] == -np.inf)


ATTEND = [  # batch, n, group, hq, hkv, d, causal, prefix per group, ctx
    (1, 1, 1, 1, 1, 64, False, [0], [1]),
    (1, 1, 1, 4, 1, 128, True, [0], [33]),
    (2, 1, 2, 4, 4, 64, True, [192], [200, 209]),
    (3, 1, 3, 8, 2, 128, True, [47], [48, 64, 80]),               # the prefix ends inside a page
    (4, 1, 2, 8, 1, 64, False, [128, 1000], [130, 128, 1500, 1001]),
    (6, 1, 3, 16, 1, 128, True, [64, 33], [0, 64, 100, 90, 0, 34]),   # empty requests, 16 heads to one
    (4, 1, 4, 4, 2, 64, True, [512], [0, 0, 0, 0]),               # nobody there
    (3, 5, 3, 8, 4, 128, True, [160], [165, 170, 400]),
    (3, 5, 3, 8, 4, 128, True, [160], [160, 170, 3]),             # rows before the start, prefix not all seen
    (2, 16, 2, 32, 8, 128, True, [300], [316, 700]),
    (2, 32, 1, 8, 1, 64, False, [0, 0], [500, 31]),               # 256 rows to one KV head
    (9, 16, 9, 8, 2, 64, True, [640], [656 + 7 * i for i in range(9)]),
    (33, 2, 11, 8, 2, 128, True, [256, 16, 1024], [256 + 3 * i for i in range(11)] +
     [16 + 5 * i for i in range(11)] + [1024 + 2 + i for i in range(11)]),
    (40, 1, 40, 8, 2, 128, False, [2048], [2048 + 13 * i for i in range(40)]),
    (64, 1, 1, 4, 4, 64, True, [0] * 64, [1 + 17 * i % 300 for i in range(64)]),
]


@pytest.mark.parametrize("batch,n,group,hq,hkv,d,causal,prefix,ctx", ATTEND)
def test_attention(batch, n, group, hq, hkv, d, causal, prefix, ctx):
    s = attention_case(batch, n, group, hq, hkv, d, causal, prefix, ctx, seed=batch + n)
    assert B_().dflash_get_status(s["ws"]) == (0, 0)
    check_attention(s, batch, n, hq, d, causal, ctx)


def test_attention_second_layer_scale_and_no_lse():
    ctx = [70, 90]
    s = attention_case(2, 3, 2, 4, 2, 64, True, [64], ctx, layers=3, layer=2, scale=0.37, lse=False)
    check_attention(s, 2, 3, 4, 64, True, ctx, layer=2, scale=0.37)


def test_attention_is_the_same_wherever_the_prefix_is_said_to_end():
    """Up to rounding; and bit for bit between two runs."""
    B = B_()
    ctx = [1000, 1100, 1003]
    s = attention_case(3, 4, 3, 16, 4, 128, True, [960], ctx)
    first = s["out"].clone()
    B.dflash_attention_prefix(*s["args"])
    assert torch.equal(first, s["out"])
    for said in (0, 100, 512, 959):
        args = list(s["args"])
        args[10] = i32([said])
        B.dflash_attention_prefix(*args)
        check_attention(s, 3, 4, 16, 128, True, ctx)


def test_attention_reports_bad_pages_and_lengths():
    B = B_()
    s = attention_case(2, 1, 2, 4, 2, 64, True, [64], [100, 80], spoil=False)
    s["c"].table_d[1, 4] = 10 ** 6           # request 1, positions 64 .. 79
    B.dflash_attention_prefix(*s["args"])
    assert B.dflash_get_status(s["ws"]) == (-3, 521)
    check_attention(s, 2, 1, 4, 64, True, [100, 80], requests=[0])
    # its keys read as zeros: score 0, value 0
    k, v = keys_of(s["c"], s["ids"][1], 0, 80)
    k[64:], v[64:] = 0.0, 0.0
    o, _, size = O.attend(s["q"][1].double().cpu().numpy(), k, v, 0.125, [80])
    assert np.all(np.abs(s["out"][1].double().cpu().numpy() - o) <= 2.0 ** -6 * size)
    s = attention_case(1, 1, 1, 4, 2, 64, False, [0], [48])
    args = list(s["args"])
    args[9] = i32([49])                       # the table holds 48 positions
    B.dflash_attention_prefix(*args)
    assert B.dflash_get_status(s["ws"]) == (-3, 522)
    check_attention(s, 1, 1, 4, 64, False, [48])


def test_attention_far_pages():
    """Pages whose element offsets pass 32 bits."""
    B = B_()
    hq, hkv, d, batch = 8, 8, 128, 2
    n_pages = (1 << 32) // (2 * hkv * PAGE * d) + 40
    pool = torch.empty((1, n_pages, 2, hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    ids = [list(range(n_pages - 30, n_pages - 20)) + [n_pages - 1], list(range(n_pages - 30, n_pages - 20)) + [0]]
    for i in sorted({i for row in ids for i in row}):
        pool[0, i] = torch.randn(pool.shape[2:], device="cuda").to(torch.bfloat16)

    class C:
        pass
    c = C()
    c.pool = pool
    table = i32(ids)
    kv = B.DflashKV(pool=pool.data_ptr(), page_table=table.data_ptr(), n_pages=n_pages, max_pages=11, n_rows=2,
                    dtype=0, scales=None)
    q = torch.randn(batch, 1, hq, d, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(batch, 1, hq, device="cuda")
    hd = heads(1, hq, hkv, d)
    ws = workspace(B.dflash_attention_prefix_bytes(hd, batch, 1, 2))
    ctx = [170, 163]
    B.dflash_attention_prefix(hd, 0, q, batch, 1, 2, True, 0.0, kv, i32(ctx), i32([160]), out, lse, ws)
    assert B.dflash_get_status(ws) == (0, 0)
    check_attention(dict(c=c, q=q, out=out, lse=lse, ids=ids, width=11), batch, 1, hq, d, True, ctx)
    # and an append to the last page
    k, v = (torch.randn(1, hkv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    B.dflash_kv_rope_append(hd, B.dflash_rope_init(0), 0, None, k, v, i32([0]), i32([175]), 1, None, kv, ws)
    assert torch.equal(pool[0, n_pages - 1, :, :, 15], torch.stack((k[0], v[0])))


ATTEND_LONG = [
    (24, 1, 24, 16, 2, 128, True, [6000], [6001 + 40 * i if i % 5 else 0 for i in range(24)]),   # 192 rows, two tiles
    (300, 1, 300, 4, 1, 64, True, [1504], [1505 + 11 * (i % 40) for i in range(300)]),           # five row tiles
    (2, 32, 1, 16, 1, 128, True, [0, 0], [5000, 1]),               # 512 rows of one request; rows before the start
    (2, 7, 2, 12, 1, 128, False, [4090], [4096, 4091]),            # 84 rows, odd and even chunks apart
    (1024, 1, 1024, 2, 1, 64, True, [160], [1 + i for i in range(1024)]),
    (1, 1, 1, 8, 8, 128, True, [0], [70001]),                      # more partials than a warp has lanes
    (1, 32, 1, 16, 16, 64, True, [0], [129]),
    (20, 16, 20, 8, 2, 128, True, [640], [656 + 7 * i for i in range(20)]),   # 1280 rows of 128, requests of 64
    (8, 16, 8, 8, 1, 128, False, [2048], [2048] * 8),              # nothing but the prefix
]


@pytest.mark.parametrize("batch,n,group,hq,hkv,d,causal,prefix,ctx", ATTEND_LONG)
def test_attention_long(batch, n, group, hq, hkv, d, causal, prefix, ctx):
    s = attention_case(batch, n, group, hq, hkv, d, causal, prefix, ctx, layers=2, layer=1, seed=batch + n)
    assert B_().dflash_get_status(s["ws"]) == (0, 0)
    check_attention(s, batch, n, hq, d, causal, ctx, layer=1,
                    requests=range(0, batch, max(1, batch // 40)))


def test_attention_bad_page_in_a_shared_prefix():
    """Its keys read as zeros for every request of the group."""
    B = B_()
    ctx = [700 + i for i in range(12)]
    s = attention_case(12, 1, 12, 16, 2, 128, False, [640], ctx, spoil=False)
    bad = 20                                 # positions 320 .. 335
    s["c"].table_d[:, bad] = -7
    B.dflash_attention_prefix(*s["args"])
    assert B.dflash_get_status(s["ws"]) == (-3, 521)
    s["c"].pool[0, s["ids"][0][bad]] = 0     # the oracle's copy of that page
    check_attention(s, 12, 1, 16, 128, False, ctx)


def test_attention_graphs_that_share_a_workspace():
    """Two captured calls of different shapes, replayed in turn on one stream
    with lengths that changed since the capture."""
    B = B_()
    shapes = [dict(batch=12, n=1, group=12, hq=16, hkv=2, d=128, causal=True, prefix=[640], ctx=[700 + i for i in range(12)]),
              dict(batch=3, n=4, group=1, hq=8, hkv=2, d=64, causal=True, prefix=[0] * 3, ctx=[90, 40, 200])]
    cases = [attention_case(**x) for x in shapes]
    ws = workspace(max(s["args"][-1].nbytes for s in cases))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for s in cases:
        s["args"] = (*s["args"][:-1], ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            B.dflash_attention_prefix(*s["args"])
        graphs.append(graph)
    for cut in (0, 30, 60, 7):
        ctx = [[max(0, c - cut) for c in x["ctx"]] for x in shapes]
        for s, graph, c in zip(cases, graphs, ctx):
            s["out"].fill_(9.0)
            s["args"][9].copy_(i32(c))
            graph.replay()
        torch.cuda.synchronize()
        for s, x, c in zip(cases, shapes, ctx):
            check_attention(s, x["batch"], x["n"], x["hq"], x["d"], True, c)
    assert B.dflash_get_status(ws) == (0, 0)


# ----------------------------------------------------------------- sampling
def draw_rows(z, T, k=None, p=None, m=None, a=None, outputs=True):
    B = B_()
    rows, vocab = z.shape
    to = lambda x, t: None if x is None else torch.as_tensor(np.asarray(x, t)).cuda()  # noqa: E731
    a = np.random.default_rng(rows * vocab).random(rows) if a is None else np.asarray(a)
    zt = z if isinstance(z, torch.Tensor) else torch.from_numpy(z).cuda()
    token = torch.full((rows,), -5, dtype=torch.int32, device="cuda")
    kept = torch.full((rows,), -5, dtype=torch.int32, device="cuda") if outputs else None
    lp = torch.full((rows,), -5.0, device="cuda") if outputs else None
    ws = workspace(B.dflash_sample_filtered_bytes(rows, vocab))
    B.dflash_sample_filtered(zt, rows, vocab, to(T, np.float32), to(k, np.int32), to(p, np.float32),
                             to(m, np.float32), to(a, np.float64), token, kept, lp, ws)
    torch.cuda.synchronize()
    return token.cpu().numpy(), None if kept is None else kept.cpu().numpy(), \
        None if lp is None else lp.cpu().numpy(), B.dflash_get_status(ws), a


def check_rows(z, T, k=None, p=None, m=None, a=None, status=(0, 0)):
    tok, kept, lp, st, a = draw_rows(z, T, k, p, m, a)
    assert st == status
    z = z.cpu().numpy() if isinstance(z, torch.Tensor) else z
    f32 = lambda x, i, off: off if x is None else float(np.float32(x[i]))  # noqa: E731
    for i in range(z.shape[0]):
        want = O.sample(z[i], f32(T, i, 1.0), int(f32(k, i, 0)), f32(p, i, 1.0), f32(m, i, 0.0), a[i])
        assert (tok[i], kept[i]) == want[:2], (i, tok[i], kept[i], want)
        assert abs(lp[i] - want[2]) <= 2.0 ** -23 * abs(want[2]) + 1e-8


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 1000, 4097, 50001, 151936, 300001])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (50, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.05), (40, 0.8, 0.01),
                                   (1, 0.5, 0.5), (0, 0.999, 0.0)])
def test_sample(vocab, k, p, m):
    g = np.random.default_rng(vocab)
    rows = 5 if vocab > 60000 else 9
    z = (g.standard_normal((rows, vocab)) * np.linspace(0.5, 5, rows)[:, None]).astype(np.float32)
    z[:, ::7][:, 1:] = -np.inf
    T = np.linspace(0.4, 1.6, rows)
    check_rows(z, T, [k] * rows, [p] * rows, [m] * rows)


@pytest.mark.parametrize("vocab", [257, 40000, 151936])
def test_sample_ties(vocab):
    """Logits with few distinct values: borders that fall on ties."""
    g = np.random.default_rng(vocab + 1)
    z = np.round(g.standard_normal((6, vocab)) * 2).astype(np.float32)
    z[4] = 0.5                                     # all equal
    z[5] = np.where(g.random(vocab) < 0.5, 0.0, -0.0)
    check_rows(z, [1.0] * 6, [50, vocab // 3, 0, 7, 10, 3], [1.0, 0.7, 0.5, 0.3, 0.9, 1.0])
    check_rows(z, [0.7] * 6, None, [0.99, 0.2, 0.5, 0.0, 0.45, 0.6], [0.0, 0.0, 1.0, 0.1, 1.0, 0.5])


def test_sample_extreme_settings():
    g = np.random.default_rng(7)
    z = (g.standard_normal((10, 3001)) * 3).astype(np.float32)
    z[8] = np.float32(3e38) * np.sign(z[8])
    z[9, :] = -np.inf
    z[9, 1234] = -3e38
    T = [0.0, 1e-3, 1e4, 1e30, 1e-38, 1.0, 1.0, 1.0, 1.0, 1.0]
    a = [0.0, 0.5, 1 - 2.0 ** -53, 0.3, 0.9, 0.0, 1 - 2.0 ** -53, 0.5, 0.75, 0.1]
    k = [5, 0, 0, 100, 0, 4000, 3001, -3, 0, 3]
    p = [0.5, 0.9, 0.5, 0.7, 0.9, 1.5, 0.0, -1.0, 0.9, 0.5]
    m = [0.0, 0.0, 0.0, 0.0, 0.0, 1e-30, 0.0, 7.0, 0.0, 0.0]
    check_rows(z, T, k, p, m, a)
    check_rows(z, T, None, None, None, a)


def test_sample_border_past_the_counted_range():
    """top_k and min_p borders among tokens that carry no mass."""
    z = -np.arange(0, 400, 0.1, dtype=np.float32)[None].repeat(4, 0)
    check_rows(z, [1.0] * 4, [1000, 0, 3999, 2000], None, [0.0, 1e-30, 1e-25, 1e-35])


def test_sample_single_token_has_probability_one():
    """One kept token: its logprob is exactly 0."""
    g = np.random.default_rng(11)
    for vocab in (1, 700, 300001):
        z = g.standard_normal((4, vocab)).astype(np.float32)
        tok, kept, lp, _, _ = draw_rows(z, [0.8, 0.3, 1.0, 0.0], [1, 1, 1, 1])
        assert np.array_equal(tok, z.argmax(1)) and np.all(kept == 1) and np.all(lp == 0.0)


def test_sample_bad_rows():
    g = np.random.default_rng(8)
    z = g.standard_normal((9, 500)).astype(np.float32)
    z[1] = -np.inf
    z[2, 77] = np.nan
    z[3, 0] = np.inf
    T = [1.0] * 4 + [-1.0, np.nan, np.inf, 1.0, 1.0]
    a = [0.4] * 7 + [1.0, 0.6]
    p = [0.9] * 8 + [np.nan]
    tok, kept, lp, st, _ = draw_rows(z, T, None, p, None, a)
    assert st == (-1, 541)
    assert tok[0] == O.sample(z[0], 1.0, 0, float(np.float32(0.9)), 0.0, 0.4)[0]
    assert np.all(tok[1:] == -1) and np.all(kept[1:] == 0) and np.all(lp[1:] == 0.0)


def test_sample_strided_rows_without_outputs():
    g = np.random.default_rng(9)
    wide = torch.from_numpy((g.standard_normal((6, 1501)) * 2).astype(np.float32)).cuda()
    z = wide[:, 3:1400]                    # odd start, odd stride
    check_rows(z, [0.9] * 6, [30] * 6, [0.9] * 6)
    tok = draw_rows(z, [0.9] * 6, [30] * 6, [0.9] * 6, outputs=False)
    assert np.array_equal(tok[0], draw_rows(z, [0.9] * 6, [30] * 6, [0.9] * 6)[0])


@pytest.mark.parametrize("rows", [1, 40, 700])
def test_sample_row_results_do_not_depend_on_the_batch(rows):
    g = torch.Generator(device="cuda").manual_seed(10)
    z = 2 * torch.randn(rows, 20011, generator=g, device="cuda")
    a = np.random.default_rng(1).random(rows)
    tok, kept, lp, _, _ = draw_rows(z, [0.8] * rows, None, [0.9] * rows, None, a)
    for i in (0, rows // 2, rows - 1):
        one = draw_rows(z[i:i + 1], [0.8], None, [0.9], None, a[i:i + 1])
        assert (one[0][0], one[1][0], one[2][0]) == (tok[i], kept[i], lp[i])


def long_rows(vocab, rows, special, T, k, p, m, a):
    """Checks the special rows in a batch that is wide enough to take one CTA
    per row (the others are filler)."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = 3 * torch.randn(rows, vocab, generator=g, device="cuda")
    at = np.arange(len(special)) * (rows // len(special))
    z[torch.from_numpy(at).cuda()] = torch.from_numpy(np.stack(special)).cuda()

    def full(x, off):
        out = np.full(rows, off, np.float64)
        out[at] = x
        return out
    tok, kept, lp, st, _ = draw_rows(z, full(T, 1.0), full(k, 0), full(p, 0.95), full(m, 0.0), full(a, 0.5))
    f32 = lambda x: float(np.float32(x))  # noqa: E731
    for j, i in enumerate(at):
        want = O.sample(special[j], f32(T[j]), int(k[j]), f32(p[j]), f32(m[j]), a[j])
        assert (tok[i], kept[i]) == want[:2], (j, tok[i], kept[i], want)
        assert abs(lp[i] - want[2]) <= 2.0 ** -23 * abs(want[2]) + 1e-8
    return tok, kept, lp, st


@pytest.mark.parametrize("rows", [48, 96])
def test_sample_many_long_rows(rows):
    """Batches of rows too long to lie in shared memory all at once: borders
    among a few, among thousands and among tied logits, odd vocabulary."""
    g = np.random.default_rng(21)
    vocab = 151937
    flat = (g.standard_normal((3, vocab)) * 0.2).astype(np.float32)      # thousands of candidates per step
    peaked = (g.standard_normal((3, vocab)) * 4).astype(np.float32)
    steps = np.round(g.standard_normal((3, vocab)) * 2).astype(np.float32)
    equal = np.full(vocab, -7.25, np.float32)
    holes = peaked[0].copy()
    holes[g.random(vocab) < 0.7] = -np.inf
    special = [*flat, *peaked, *steps, equal, holes, peaked[1] * np.float32(0.01)]
    n = len(special)
    T = [1.0, 0.7, 2.0] * 4
    _, _, _, st = long_rows(vocab, rows, special, T, [0, 5000, 0, 0, 40, 0, 0, 30000, 0, 99, 0, 7],
                            [0.9, 0.5, 0.3, 0.95, 1.0, 0.8, 0.5, 0.7, 1.0, 0.4, 0.9, 0.6],
                            [0.0, 0.0, 0.0, 0.0, 0.0, 0.01, 0.0, 0.0, 0.2, 0.0, 1e-4, 0.0], g.random(n))
    assert st == (0, 0)
    long_rows(vocab, rows - 3, special, T, [0] * n, [1.0] * n, [0.0] * n, g.random(n))
    special[4] = special[4].copy()
    special[4][vocab - 1] = np.nan
    tok, kept, lp, st = long_rows(vocab, rows, special, [0.0] + T[1:], [0] * n, [0.9] * n, [0.0] * n, g.random(n))
    at = 4 * (rows // n)
    assert st == (-1, 541) and tok[at] == -1 and kept[at] == 0


@pytest.mark.parametrize("rows", [42, 100])
def test_sample_many_long_rows_with_plateaus(rows):
    """A top-p border among more than 2^16 logits of the same value, with
    others a few units in the last place away."""
    vocab, special, p = 300001, [], []
    g = np.random.default_rng(22)
    for x in (-0.3, -1.7, -3.1, -4.03, -5.9, -7.77):
        z = np.full(vocab, x, np.float32)
        z[g.random(vocab) < 0.4] = np.nextafter(np.float32(x), np.float32(0))
        z[12345] = 0.0
        special.append(z)
        p.append(0.2 + 0.6 * g.random())
    n = len(special)
    long_rows(vocab, rows, special, [1.0] * n, [0] * n, p, [0.0] * n, g.random(n))


@pytest.mark.parametrize("rows", [40, 100])
def test_sample_many_long_rows_with_a_full_step(rows):
    """More than 2^18 logits within one of the steps that a row's mass is first
    counted by, and a border close to the step's end."""
    vocab, many, special, p = 393216, 300000, [], []
    g = np.random.default_rng(23)
    ln2 = math.log(2.0)
    for over in (-0.003, 0.003, -0.001, 0.001):
        z = np.empty(vocab, np.float32)
        z[0] = 0.0
        z[1:many + 1] = -(100 + 0.49) * 46 / 1023 * ln2
        z[many + 1:] = -(101 + g.integers(1, 9, vocab - many - 1)) * 46 / 1023 * ln2
        w = np.exp(z.astype(np.float64))
        p.append((1 + over) * w[:many + 1].sum() / w.sum())
        special.append(g.permutation(z))
    n = len(special)
    long_rows(vocab, rows, special, [1.0] * n, [0] * n, p, [0.0] * n, g.random(n))


def test_sample_huge_and_tiny_temperatures():
    """A temperature outside [1e-30, 1e30] counts as the bound."""
    g = np.random.default_rng(24)
    z = (g.standard_normal((6, 5000)) * 1e30).astype(np.float32)
    z[3:] = np.float32(3e38) * np.sign(z[3:])
    T = [1e30, 3e38, 1e-38, 1e38, 1e31, 1e-45]
    check_rows(z, T, None, [0.9] * 6, None, g.random(6))
    check_rows(z, T, [100] * 6, None, [0.0, 0.3, 0.0, 0.5, 0.0, 0.5], g.random(6))


# ----------------------------------------------------------------- together
def test_decode_steps_together_eager_and_captured():
    """append -> attend -> logits -> sample, three tokens for requests that
    share a prompt: eager on a side stream, then as a replayed graph with the
    lengths advanced on the device; against the oracle step by step."""
    B = B_()
    from block_diffusion_speculative_fuse_gb300.device import PagedKV
    import workload as W
    batch, hq, hkv, d, vocab, prefix = 4, 8, 2, 64, 512, 80
    shape = W.ModelShape(n_layers=1, hidden=256, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, mlp=256, vocab=vocab)
    per = 3
    table = np.array([[0, 1, 2, 3, 4] + list(range(5 + per * r, 5 + per * (r + 1))) for r in range(batch)], np.int32)
    g = torch.Generator(device="cuda").manual_seed(3)
    rope = B.dflash_rope_init(d, scaling="linear", factor=2.0)
    head = torch.randn(vocab, hq * d, generator=g, device="cuda") * 0.5
    steps = 3
    qkv = torch.randn(steps, batch, (hq + 2 * hkv) * d, generator=g, device="cuda").to(torch.bfloat16)
    u = torch.rand(steps, batch, generator=g, device="cuda", dtype=torch.float64)
    settings = [torch.full((batch,), x, dtype=t, device="cuda") for x, t in
                ((0.9, torch.float32), (40, torch.int32), (0.9, torch.float32), (0.01, torch.float32))]
    f, mag = O.rope_freqs(d, 1e6, "linear", 2.0)

    def build():
        kv = PagedKV(shape, table, int(table.max()) + 1)
        kv.pool.copy_(torch.randn(kv.pool.shape, generator=torch.Generator(device="cuda").manual_seed(4),
                                  device="cuda"))
        ws = kv.attention_workspace(hq, batch, 1, batch)
        st = dict(kv=kv, ws=ws, x=qkv[0].clone(), u=u[0].clone(), pos=i32([prefix] * batch), ctx=i32([prefix + 1] * batch),
                  q=torch.empty(batch, hq, d, dtype=torch.bfloat16, device="cuda"),
                  out=torch.empty(batch, 1, hq, d, dtype=torch.bfloat16, device="cuda"),
                  logits=torch.empty(batch, vocab, device="cuda"),
                  token=torch.empty(batch, dtype=torch.int32, device="cuda"))
        st["req"], st["pre"] = i32(np.arange(batch)), i32([prefix])
        return st

    def step(s):
        x = s["x"]
        q, k, v = (t.unflatten(1, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], 1))
        s["kv"].append_rotated(rope, 0, q, k, v, s["req"], s["pos"], s["ws"], q_out=s["q"])
        s["kv"].attend_prefix(0, s["q"].view(batch, 1, hq, d), s["ctx"], s["pre"], batch, s["out"], s["ws"])
        torch.matmul(s["out"].view(batch, -1).float(), head.T, out=s["logits"])
        B.dflash_sample_filtered(s["logits"], batch, vocab, *settings, s["u"], s["token"], None, None, s["ws"])
        s["pos"] += 1
        s["ctx"] += 1

    def feed(s, i):
        s["x"].copy_(qkv[i])
        s["u"].copy_(u[i])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = build()
    eager = []
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        for i in range(steps):
            feed(a, i)
            step(a)
            eager.append((a["q"].clone(), a["out"].clone(), a["logits"].clone(), a["token"].clone()))
    side.synchronize()
    b = build()
    warm = build()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        step(warm)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(b)
    for i in range(steps):
        feed(b, i)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager[i], (b["q"], b["out"], b["logits"], b["token"])):
            assert torch.equal(x, y)
    assert B.dflash_get_status(a["ws"]) == (0, 0) and B.dflash_get_status(b["ws"]) == (0, 0)

    # the oracle, step by step
    for i in range(steps):
        q, out, logits, token = eager[i]
        x = qkv[i].double().cpu().numpy().reshape(batch, -1, d)[:, :hq]
        qe = O.rotate(x, [prefix + i] * batch, f, mag, False)
        half = np.hypot(x[..., :d // 2], x[..., d // 2:])
        size = np.concatenate((half, half), -1)
        assert np.all(np.abs(q.double().cpu().numpy() - qe) <= 2.0 ** -8 * np.abs(qe) + 2.0 ** -18 * size)
        check_attention(dict(c=a["kv"], q=q.view(batch, 1, hq, d), out=out, lse=None, ids=table.tolist(),
                             width=table.shape[1]), batch, 1, hq, d, True, [prefix + i + 1] * batch)
        for r in range(batch):
            want = O.sample(logits[r].cpu().numpy(), float(np.float32(0.9)), 40, float(np.float32(0.9)),
                            float(np.float32(0.01)), float(u[i, r]))
            assert int(token[r]) == want[0]


def test_sampled_generation_is_the_loop_of_its_parts():
    """sample_generate: temperature 0 reproduces ar_generate; with settings,
    every token is the oracle's draw from the target's own logits."""
    import workload as W
    from block_diffusion_speculative_fuse_gb300.device import DeviceModel
    from block_diffusion_speculative_fuse_gb300.generate import TargetRunner, ar_generate, sample_generate
    t = W.get_workload("tiny_e2e").target
    shared, tw = W.shared_weights(t, 71, std=0.05), W.target_weights(t, 71, std=0.05)
    model = DeviceModel(t, tw, shared, draft=False)
    prompts = np.random.default_rng(2).integers(0, t.vocab, (3, 9)).astype(np.int32)
    n = 6
    u = np.random.default_rng(3).random((3, n))
    greedy = ar_generate(TargetRunner(model, 3, 32, 9), prompts, n)
    assert np.array_equal(sample_generate(TargetRunner(model, 3, 32, 9), prompts, n, u, temperature=0.0), greedy)
    keep = []
    toks = sample_generate(TargetRunner(model, 3, 32, 9), prompts, n, u, temperature=0.8, top_k=20, top_p=0.9,
                           keep_logits=keep)
    for i in range(n):
        for r in range(3):
            want = O.sample(keep[i][r], float(np.float32(0.8)), 20, float(np.float32(0.9)), 0.0, u[r, i])
            assert toks[r, i] == want[0]
