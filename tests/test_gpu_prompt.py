"""Operators of a long prompt on the GPU (chunk attention, attention mass,
eviction, token scores) against the 64-bit oracle (oracle/serving.py).

Tolerances (half a step of a rounding: bf16 2^-8, fp32 2^-24):
* chunk attention: probabilities rounded to bf16 (2^-8 of sum p |v|), the
  output rounded (2^-8), and the scores' fp32 error: a sum of d products loses
  at most d 2^-24 of sum |q k|, which moves every p (and lse) by that much.
"""
import math

import numpy as np
import pytest
import torch

from oracle import serving as O

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


def heads(L, hq, hkv, d, terms=1):
    return B_().DflashHeads(n_layers=L, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, page_size=PAGE, kv_terms=terms)


class Cache:
    """A cache over a shuffled pool for requests of these lengths; every value
    that no request owns is NaN."""

    def __init__(self, L, hkv, d, lens, seed=0, width=None, spoil=True, spare=3):
        B = B_()
        rnd = np.random.default_rng(seed)
        need = [max(0, (n + PAGE - 1) // PAGE) for n in lens]
        self.n_pages = sum(need) + spare
        perm = rnd.permutation(self.n_pages)
        self.width = width or max(1, max(need))
        self.table = np.full((len(lens), self.width), -7, np.int32)
        self.ids, at = [], 0
        for r, k in enumerate(need):
            self.ids.append([int(x) for x in perm[at:at + k]])
            self.table[r, :k] = self.ids[r]
            at += k
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = torch.randn((L, self.n_pages, 2, hkv, PAGE, d), generator=g, device="cuda").to(torch.bfloat16)
        if spoil:
            owned = np.zeros((self.n_pages, PAGE), bool)
            for r, n in enumerate(lens):
                for p in range(n):
                    owned[self.ids[r][p // PAGE], p % PAGE] = True
            self.pool.permute(0, 2, 3, 1, 4, 5)[:, :, :, torch.from_numpy(~owned).cuda()] = float("nan")
        self.table_d = i32(self.table)
        self.kv = B.DflashKV(pool=self.pool.data_ptr(), page_table=self.table_d.data_ptr(), n_pages=self.n_pages,
                             max_pages=self.width, n_rows=len(lens), dtype=0, scales=None)

    def keys(self, r, layer, count):
        """K and V [count][hkv][d] of a request in 64 bits."""
        pages = torch.tensor(self.ids[r], dtype=torch.long)[:(count + PAGE - 1) // PAGE].cuda()
        kv = self.pool[layer, pages].double().cpu().numpy().transpose(1, 0, 3, 2, 4)
        kv = kv.reshape(2, -1, kv.shape[3], kv.shape[4])
        return kv[0, :count], kv[1, :count]


# ---------------------------------------------------------- chunk attention
def rows_of(T, width, hq, d, fill=None, seed=0):
    """[T][hq][d] bf16, columns of a wider array."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (1.3 * torch.randn(T, width, generator=g, device="cuda")).to(torch.bfloat16)
    if fill is not None:
        x.fill_(fill)
    return x[:, :hq * d].unflatten(1, (hq, d))


def chunk_case(ns, ctx, hq, hkv, d, causal=True, layers=1, layer=0, scale=0.0, seed=0, lse=True, lead=0, tail=0,
               wide=0, width=None, spare_ws=0):
    B = B_()
    c = Cache(layers, hkv, d, ctx, seed, width)
    start = np.concatenate([[0], np.cumsum(ns)]) + lead
    T = int(start[-1]) + tail
    q, out = (rows_of(max(T, 1), hq * d + wide, hq, d, f, seed + 1) for f in (None, 7.0))
    T = max(T, 1)
    L = torch.full((T, hq), 7.0, device="cuda") if lse else None
    hd = heads(layers, hq, hkv, d)
    ws = workspace(B.dflash_attention_chunk_bytes(hd, len(ns), T) + spare_ws)
    args = (hd, layer, q, i32(start), len(ns), T, causal, scale, c.kv, i32(ctx), out, L, ws)
    B.dflash_attention_chunk(*args)
    torch.cuda.synchronize()
    return dict(c=c, q=q, out=out, lse=L, ws=ws, args=args, start=start, ns=ns, ctx=ctx, T=T)


def check_chunk(s, hq, d, causal=True, layer=0, scale=0.0, requests=None, status=(0, 0)):
    assert B_().dflash_get_status(s["ws"]) == status
    scale = scale or 1.0 / math.sqrt(d)
    out = s["out"].double().cpu().numpy()
    for r in requests if requests is not None else range(len(s["ns"])):
        n, m, a = s["ns"][r], s["ctx"][r], int(s["start"][r])
        if n == 0:
            continue
        k, v = s["c"].keys(r, layer, m)
        q = s["q"][a:a + n].double().cpu().numpy()
        G = hq // s["c"].pool.shape[3]
        o, lse, size = O.attend(q, k, v, scale, [m - n + i + 1 if causal else m for i in range(n)])
        worst = scale * max(float((np.abs(q[:, h]) @ np.abs(k[:, h // G]).T).max()) for h in range(hq)) if m else 0.0
        delta = (d + 16) * 2.0 ** -24 * worst + 2.0 ** -20
        tol = (2.0 ** -8 + 2 * delta) * (size + np.abs(o)) + 1e-30
        got = out[a:a + n]
        assert np.all(np.abs(got - o) <= tol), (r, float(np.nanmax(np.abs(got - o) / tol)))
        if s["lse"] is not None:
            gl = s["lse"][a:a + n].double().cpu().numpy()
            f = np.isfinite(lse)
            assert np.all(np.abs(gl[f] - lse[f]) <= delta + 2.0 ** -21 * (1 + np.abs(lse[f])))
            assert np.all(gl[~f] == -np.inf)
    # rows of no request are left as they were
    other = np.ones(s["T"], bool)
    other[int(s["start"][0]):int(s["start"][-1])] = False
    assert np.all(out[other] == 7.0)
    if s["lse"] is not None:
        assert np.all(s["lse"].cpu().numpy()[other] == 7.0)


CHUNK = [  # rows per request, cached positions per request, hq, hkv, d, causal
    ([1], [1], 1, 1, 64, True),
    ([1], [1], 4, 1, 128, False),
    ([1], [0], 4, 2, 128, True),                       # a row that sees nothing
    ([1], [4096], 32, 8, 128, True),
    ([3], [130], 16, 1, 64, True),                     # 16 heads to one
    ([0, 5, 0, 7, 0], [0, 5, 40, 29, 0], 8, 4, 64, True),
    ([0, 0], [33, 0], 8, 4, 64, True),                 # nobody there
    ([40, 300], [17, 3], 8, 2, 128, True),             # rows before the start
    ([40, 300], [17, 0], 8, 2, 64, False),
    ([100], [100], 6, 2, 64, True),                    # three heads to one
    ([61, 2], [500, 18], 15, 3, 128, True),            # five
    ([45], [77], 14, 2, 64, False),                    # seven
    ([33], [300], 11, 1, 128, True),                   # eleven
    ([200, 1, 64, 65], [777, 900, 64, 1000], 32, 8, 128, True),
    ([600, 257], [600, 300], 2, 2, 64, True),          # a head to one: 256 rows per unit
    ([129], [1031], 4, 4, 128, True),
    ([70, 33], [1000, 2], 8, 2, 128, False),
    ([33, 17], [9000, 6001], 8, 1, 128, True),         # units cut into many pieces
    ([500], [2500], 16, 4, 64, True),
]


@pytest.mark.parametrize("ns,ctx,hq,hkv,d,causal", CHUNK)
def test_chunk(ns, ctx, hq, hkv, d, causal):
    wide = 8 * (len(ns) % 3)
    s = chunk_case(ns, ctx, hq, hkv, d, causal, seed=sum(ns) + d, lead=sum(ns) % 3, tail=sum(ns) % 5, wide=wide)
    check_chunk(s, hq, d, causal)


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_many_requests(d):
    rnd = np.random.default_rng(d)
    ns = [int(x) for x in rnd.choice([0, 1, 1, 1, 2, 9], 900)]
    ctx = [int(x) for x in rnd.integers(0, 200, 900)]
    s = chunk_case(ns, ctx, 4, 2, d, seed=d)
    check_chunk(s, 4, d, requests=range(0, 900, 7))


def test_chunk_second_layer_scale_and_no_lse():
    s = chunk_case([30, 1], [90, 300], 8, 2, 64, layers=3, layer=1, scale=0.3, lse=False, width=40)
    check_chunk(s, 8, 64, layer=1, scale=0.3)


# ------------------------------------------------------------- token scores
def check_scores(z, T, ids, n, bad=(), wrong_id=(), stride=None):
    """Runs a call on logits z (a tensor) and compares every row."""
    B = B_()
    rows, vocab = z.shape
    ws = workspace(B.dflash_score_tokens_bytes(rows, vocab, n))
    lp, ent = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    rank = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
    ti = torch.full((rows, n), 7, dtype=torch.int32, device="cuda") if n else None
    tl = torch.full((rows, n), 7.0, device="cuda") if n else None
    Td = torch.as_tensor(T, dtype=torch.float32).cuda() if T is not None else None
    B.dflash_score_tokens(z, rows, vocab, Td, i32(ids), lp, rank, ent, n, ti, tl, ws)
    torch.cuda.synchronize()
    status = B.dflash_get_status(ws)
    assert status == ((0, 0) if not bad and not wrong_id else (-1, 571 if bad and not wrong_id else status[1]))
    zh = z.double().cpu().numpy()
    lp, rank, ent = lp.double().cpu().numpy(), rank.cpu().numpy(), ent.double().cpu().numpy()
    for r in range(rows):
        if r in bad:
            assert np.isnan(lp[r]) and np.isnan(ent[r]) and rank[r] == -1
            if n:
                assert (ti[r] == -1).all() and torch.isnan(tl[r]).all()
            continue
        tok = -1 if r in wrong_id else ids[r]
        e = O.score(zh[r], 1.0 if T is None else T[r], tok, n)
        mean = math.log(vocab) + 15
        tol = 2.0 ** -22 * (1 + mean)
        assert abs(ent[r] - e[2]) <= 2 * tol + 2.0 ** -22 * (abs(e[2]) + mean), (r, ent[r], e[2])
        if r in wrong_id:
            assert np.isnan(lp[r]) and rank[r] == -1
        else:
            assert rank[r] == e[1]
            if np.isfinite(e[0]):
                assert abs(lp[r] - e[0]) <= tol + 2.0 ** -22 * (abs(e[0]) + mean), (r, lp[r], e[0])
            else:
                assert lp[r] == e[0]
        if n:
            got, gl = ti[r].cpu().numpy(), tl[r].double().cpu().numpy()
            k = len(e[3])
            assert list(got[:k]) == e[3] and (got[k:] == -1).all() and (gl[k:] == -np.inf).all()
            assert np.all(np.abs(gl[:k] - e[4]) <= tol + 2.0 ** -22 * (np.abs(e[4]) + mean))


def logits(rows, vocab, spread=2.0, dtype=torch.float32, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (spread * torch.randn(rows, vocab + pad, generator=g, device="cuda")).to(dtype)
    return z[:, :vocab]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,n,pad", [
    (1, 1, 1, 0), (3, 2, 5, 1), (5, 7, 0, 0), (2, 64, 64, 3), (7, 1009, 8, 0), (4, 1009, 64, 2), (1, 4097, 20, 0),
    (1, 40000, 20, 0), (3, 40001, 64, 5), (40, 12345, 5, 1), (200, 9000, 3, 0), (330, 501, 1, 0), (2, 151936, 20, 0),
    (1, 393216, 10, 0)])
def test_score(dtype, rows, vocab, n, pad):
    rnd = np.random.default_rng(vocab + n)
    z = logits(rows, vocab, dtype=dtype, seed=vocab, pad=pad)
    if vocab > 20:
        z[:, 3:9] = -math.inf
    ids = rnd.integers(0, vocab, rows)
    ids[rnd.random(rows) < 0.2] = -rnd.integers(1, 200)
    if rows > 2 and vocab > 20:
        ids[1] = 5      # a token whose logit is -inf
    check_scores(z, rnd.choice([0.3, 0.7, 1.0, 3.0], rows).astype(np.float32) if n % 2 else None, ids, n)


@pytest.mark.parametrize("vocab", [33, 3000, 70001])
def test_score_ties(vocab):
    """Plateaus: constant rows, two levels, steps; -0 and +0 are equal."""
    z = torch.zeros(5, vocab, device="cuda")
    z[0, 1::2] = -0.0
    z[1, 7::3] = 1.0
    z[2] = (torch.arange(vocab, device="cuda") // 5 % 40).float()
    z[3] = -math.inf
    z[3, vocab // 2:vocab // 2 + 9] = 2.5
    z[4] = torch.linspace(-3, 3, vocab, device="cuda")     # ascending
    ids = [vocab - 1, 7, vocab // 3, vocab // 2 + 4, 0]
    for n in (1, 20, 64):
        check_scores(z, None, ids, n)
        check_scores(z.to(torch.bfloat16), [0.5] * 5, ids, n)


def test_score_bad_rows_and_ids():
    z = logits(9, 5000)
    z[1, 77] = math.nan
    z[2, 4999] = math.inf
    z[3] = -math.inf
    z[4, :2500] = math.nan
    z[4, 2500:] = -math.inf
    T = [1.0, 1.0, 1.0, 1.0, 1.0, 0.0, math.nan, math.inf, 1.0]
    check_scores(z, T, [4] * 9, 4, bad=(1, 2, 3, 4, 5, 6, 7))
    check_scores(logits(3, 300), None, [1, 300, 2 ** 31 - 1], 4, wrong_id=(1, 2))


def test_score_extreme_temperatures_and_logits():
    z = logits(6, 20000, spread=1.0)
    z[4] *= 1e4
    z[5] = z[5] * 1e30
    check_scores(z, [1e-35, 1e-3, 1e6, 1e38, 1.0, 1e30], [int(z[0].argmax()), 3, 4, 5, int(z[4].argmax()), 9], 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_score_rows_at_odd_addresses(dtype):
    """Rows that start anywhere in a 16-byte vector, and end anywhere."""
    for off in range(1, 9):
        z = logits(5, 3001 + off, dtype=dtype, seed=off, pad=3)[:, off:]
        ids = [0, 1, 3000, 7, -1]
        check_scores(z, None, ids, 7)
        tiny = logits(6, 20, dtype=dtype, seed=off)[:, off:off + 1 + off % 3]
        check_scores(tiny, None, [0] * 6, 2)


def test_score_optional_outputs_and_single_rows():
    """Outputs may be left out, and a row's results do not depend on the others."""
    B = B_()
    z = logits(170, 151936, seed=5)
    ids = i32(np.arange(170) * 7)
    ws = workspace()
    res = []
    for lo, hi in ((0, 170), (0, 1), (3, 40), (169, 170)):
        k = hi - lo
        ent, ti, tl = (torch.zeros(k, device="cuda"), torch.zeros(k, 6, dtype=torch.int32, device="cuda"),
                       torch.zeros(k, 6, device="cuda"))
        B.dflash_score_tokens(z[lo:hi], k, 151936, None, None, None, None, ent, 6, ti, tl, ws)
        lp = torch.zeros(k, device="cuda")
        B.dflash_score_tokens(z[lo:hi], k, 151936, None, ids[lo:hi].contiguous(), lp, None, None, 0, None, None, ws)
        res.append((lo, hi, ent, ti, tl, lp))
    assert B.dflash_get_status(ws) == (0, 0)
    for lo, hi, ent, ti, tl, lp in res[1:]:
        assert torch.equal(ti, res[0][3][lo:hi])
        for a, b in ((ent, res[0][2]), (tl, res[0][4]), (lp, res[0][5])):
            assert torch.allclose(a, b[lo:hi], rtol=0, atol=2.0 ** -22 * (1 + math.log(151936) + 30))


# ----------------------------------------------------------- attention mass
def mass_case(ns, ctx, hq, hkv, d, last=0, causal=True, add=False, seed=0, lead=1, tail=2, wide=8, room=5, layers=1,
              layer=0, scale=0.0):
    """A chunk attention call for the lse, then the mass call over the same rows."""
    B = B_()
    s = chunk_case(ns, ctx, hq, hkv, d, causal, seed=seed, lead=lead, tail=tail, wide=wide, layers=layers, layer=layer,
                   scale=scale)
    hd, kv, start, T = s["args"][0], s["c"].kv, s["args"][3], s["T"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    mass0 = torch.rand(len(ns), hkv, max(1, max(ctx)) + room, generator=g, device="cuda")
    s["mass0"], s["mass"] = mass0.clone(), mass0
    ws = workspace(B.dflash_attention_mass_bytes(hd, len(ns), T))
    s["mass_args"] = (hd, layer, s["q"], start, len(ns), T, last, causal, scale, kv, i32(ctx), s["lse"], mass0, add, ws)
    B.dflash_attention_mass(*s["mass_args"])
    torch.cuda.synchronize()
    assert B.dflash_get_status(ws) == (0, 0)
    return s


def check_mass(s, hq, d, last=0, causal=True, add=False, layer=0, scale=0.0):
    scale = scale or 1.0 / math.sqrt(d)
    got, before = s["mass"].double().cpu().numpy(), s["mass0"].double().cpu().numpy()
    lse = s["lse"].double().cpu().numpy()
    for r, (n, m) in enumerate(zip(s["ns"], s["ctx"])):
        w = min(n, last) if last else n
        a = int(s["start"][r]) + n - w
        k, _ = s["c"].keys(r, layer, m)
        q = s["q"][a:a + w].double().cpu().numpy()
        assert np.array_equal(got[r, :, m:], before[r, :, m:])
        if m == 0:
            continue
        want = O.attention_mass(q, k, lse[a:a + w], scale, [m - w + i + 1 if causal else m for i in range(w)])
        G = hq // k.shape[1]
        worst = scale * max([float((np.abs(q[:, h]) @ np.abs(k[:, h // G]).T).max()) for h in range(hq)] + [0.0]) \
            if w else 0.0
        f = lse[a:a + w][np.isfinite(lse[a:a + w])]
        size = worst + (float(np.abs(f).max()) if f.size else 0.0)
        rel = (d + 16) * 2.0 ** -24 * worst + 2.0 ** -23 * size + 2.0 ** -21 + w * G * 2.0 ** -24
        old = before[r, :, :m] if add else 0.0
        err = np.abs(got[r, :, :m] - want - old)
        tol = rel * want + 2.0 ** -23 * (want + old) + 1e-30
        assert np.all(err <= tol), (r, float((err / tol).max()))


MASS = [  # rows per request, cached positions, hq, hkv, d, last, causal, add
    ([1], [1], 1, 1, 64, 0, True, False),
    ([1], [0], 4, 2, 128, 0, True, False),
    ([1], [4096], 32, 8, 128, 32, True, True),
    ([0, 5, 0, 7, 0], [0, 5, 40, 29, 300], 8, 4, 64, 0, True, False),
    ([0, 5, 2], [300, 5, 40], 8, 4, 64, 3, True, True),
    ([40], [17], 8, 2, 128, 0, True, False),           # rows before the start
    ([100, 3], [700, 129], 6, 2, 64, 33, True, False), # three heads to one
    ([61], [500], 15, 3, 128, 0, False, True),
    ([33], [300], 11, 1, 128, 0, True, False),
    ([200, 64], [777, 64], 32, 8, 128, 0, True, False),    # many tiles
    ([300], [300], 2, 2, 64, 0, True, True),           # a whole prompt, a head to one
    ([70, 33], [1000, 2], 8, 2, 128, 16, False, False),
    ([32, 32, 9], [9000, 6001, 8191], 8, 2, 128, 32, True, False),
]


@pytest.mark.parametrize("ns,ctx,hq,hkv,d,last,causal,add", MASS)
def test_mass(ns, ctx, hq, hkv, d, last, causal, add):
    s = mass_case(ns, ctx, hq, hkv, d, last, causal, add, seed=sum(ctx) + d)
    check_mass(s, hq, d, last, causal, add)


def test_mass_many_requests_layers_and_scale():
    rnd = np.random.default_rng(4)
    ns = [int(x) for x in rnd.choice([0, 1, 1, 2, 9], 700)]
    ctx = [int(x) + n for x, n in zip(rnd.integers(0, 600, 700), ns)]
    s = mass_case(ns, ctx, 4, 2, 64, 1, seed=3, layers=2, layer=1, scale=0.2)
    check_mass(s, 4, 64, 1, layer=1, scale=0.2)


def test_mass_of_all_rows_adds_up_to_the_rows():
    s = mass_case([150, 20], [600, 20], 8, 2, 128, seed=9)
    got = s["mass"].double().cpu().numpy()
    for r, m in enumerate(s["ctx"]):
        assert np.allclose(got[r, :, :m].sum(1), s["ns"][r] * 4, rtol=1e-4)


# ------------------------------------------------------------------ eviction
def evict_case(ctx, keep, hkv, d, sink=0, recent=0, kind="bf16", same_pool=False, seed=0, mass=None, layers=2, layer=1,
               room=3, spread=3.0):
    B = B_()
    rnd = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    planes = 4 if kind == "two" else 2
    new = [min(max(k, 0), c) for k, c in zip(keep, ctx)]
    need = [(c + 15) // 16 for c in ctx], [(n + 15) // 16 for n in new]
    total = [sum(x) + 2 for x in need]
    if same_pool:
        total = [sum(total)] * 2
    perm = [rnd.permutation(total[0]), None]
    perm[1] = perm[0][::-1] if same_pool else rnd.permutation(total[1])
    tables = []
    for side in (0, 1):
        t = np.full((len(ctx), max(1, max(need[side])) + 1), -3, np.int32)
        at = 0
        for r, k in enumerate(need[side]):
            t[r, :k] = perm[side][at:at + k]
            at += k
        tables.append(t)

    def pool(pages):
        if kind == "e4m3":
            return (torch.randint(0, 256, (layers, pages, planes, hkv, PAGE, d), generator=g, device="cuda",
                                  dtype=torch.uint8), torch.rand(layers, pages, planes, hkv, PAGE, generator=g,
                                                                 device="cuda"))
        return torch.randint(-2 ** 15, 2 ** 15, (layers, pages, planes, hkv, PAGE, d), generator=g, device="cuda",
                             dtype=torch.int16), None
    src = pool(total[0])
    dst = src if same_pool else pool(total[1])
    td = [i32(t) for t in tables]
    kvs = [B.DflashKV(pool=x[0].data_ptr(), page_table=t.data_ptr(), n_pages=n, max_pages=t.shape[1], n_rows=len(ctx),
                      dtype=1 if kind == "e4m3" else 0, scales=None if x[1] is None else x[1].data_ptr())
           for x, t, n in zip((src, dst), td, total)]
    if mass is None:
        mass = torch.exp(spread * torch.randn(len(ctx), hkv, max(1, max(ctx)) + room, generator=g, device="cuda"))
        mass = torch.where(mass < 0.3, 0.0, mass)
    kept = torch.full((len(ctx), hkv, max(1, max(new)) + 1), -9, dtype=torch.int32, device="cuda")
    new_len = torch.full((len(ctx),), -9, dtype=torch.int32, device="cuda")
    mass_out = torch.full_like(mass, -9.0)
    hd = heads(layers, hkv, hkv, d, planes // 2)
    before = [None if x is None else x.clone() for x in src + dst]
    ws = workspace(B.dflash_kv_evict_bytes(hd, len(ctx), total[1]))
    args = (hd, layer, kvs[0], kvs[1], len(ctx), i32(ctx), i32(keep), sink, recent, mass, kept, new_len, mass_out, ws)
    B.dflash_kv_evict(*args)
    torch.cuda.synchronize()
    return dict(src=src, dst=dst, before=before, tables=tables, td=td, mass=mass, kept=kept, new_len=new_len,
                mass_out=mass_out, ws=ws, new=new, args=args, kvs=kvs)


def check_evict(s, ctx, keep, hkv, sink, recent, layer=1):
    assert B_().dflash_get_status(s["ws"]) == (0, 0)
    assert list(s["new_len"].cpu().numpy()) == s["new"]
    mass, kept, mass_out = (s[k].cpu().numpy() for k in ("mass", "kept", "mass_out"))
    want = s["before"][2].clone()
    scales = None if s["before"][3] is None else s["before"][3].clone()
    for r, c in enumerate(ctx):
        n = s["new"][r]
        assert (kept[r, :, n:] == -9).all() and (mass_out[r, :, n:] == -9.0).all()
        for h in range(hkv):
            k = np.array(O.evict(mass[r, h], c, keep[r], sink, recent), np.int64)
            assert np.array_equal(kept[r, h, :n], k), (r, h)
            assert np.array_equal(mass_out[r, h, :n], mass[r, h, k], equal_nan=True)
            if n == 0:
                continue
            at = np.arange(n)
            to, ts = torch.from_numpy(s["tables"][1][r, at // 16].astype(np.int64)), torch.from_numpy(at % 16)
            fr, fs = torch.from_numpy(s["tables"][0][r, k // 16].astype(np.int64)), torch.from_numpy(k % 16)
            want[layer, to, :, h, ts] = s["before"][0][layer, fr, :, h, fs]
            if scales is not None:
                scales[layer, to, :, h, ts] = s["before"][1][layer, fr, :, h, fs]
    assert torch.equal(s["dst"][0], want)
    if scales is not None:
        assert torch.equal(s["dst"][1], scales)


EVICT = [  # ctx, keep, hkv, d, sink, recent, kind, same pool
    ([1], [1], 1, 64, 0, 0, "bf16", False),
    ([40], [17], 2, 128, 0, 0, "bf16", False),
    ([0, 33, 5, 100], [4, 0, 9, 31], 4, 64, 4, 8, "bf16", True),
    ([700, 1025, 16], [100, 1024, 3], 3, 128, 2, 5, "two", False),
    ([3000], [1], 8, 64, 0, 0, "e4m3", False),
    ([300, 299], [64, 250], 2, 128, 300, 10, "e4m3", True),   # more protected than kept
    ([20001], [5000], 2, 128, 4, 64, "bf16", False),          # over a cluster
    ([70000, 9], [12345, 9], 1, 64, 1, 1, "bf16", False),
    ([64, 2500], [-3, 10 ** 6], 2, 64, 0, 0, "bf16", False),
]


@pytest.mark.parametrize("ctx,keep,hkv,d,sink,recent,kind,same", EVICT)
def test_evict(ctx, keep, hkv, d, sink, recent, kind, same):
    s = evict_case(ctx, keep, hkv, d, sink, recent, kind, same, seed=sum(ctx) + d)
    check_evict(s, ctx, keep, hkv, sink, recent)


@pytest.mark.parametrize("ctx", [900, 30000])
def test_evict_ties_and_special_masses(ctx):
    """Equal masses go to the lower position; NaN last, -0 and 0 alike."""
    m = torch.zeros(5, 1, ctx, device="cuda")
    m[0, 0, ::2] = -0.0
    m[1, 0, ctx // 2:] = 1.0
    m[2] = torch.arange(ctx, device="cuda") % 7
    m[3, 0, ::3] = math.nan
    m[3, 0, 1::3] = -math.inf
    m[4, 0, 10:50] = math.inf
    m[4, 0, 60:] = -1.0
    keep = [ctx // 3, ctx // 2 + 5, ctx // 4, ctx // 3 * 2 + 9, 45]
    for sink, recent in ((0, 0), (3, 20)):
        s = evict_case([ctx] * 5, keep, 1, 64, sink, recent, mass=m, seed=ctx)
        check_evict(s, [ctx] * 5, keep, 1, sink, recent)


def test_evict_refuses_pages_in_use():
    """A target page that the call reads, or writes twice: nothing is copied."""
    B = B_()
    for clash in ("read", "twice"):
        s = evict_case([100, 90], [40, 40], 2, 64, same_pool=True, seed=1)
        pool = s["dst"][0].clone()
        s["td"][1][1, 2] = s["td"][0][0, 1] if clash == "read" else s["td"][1][0, 0]
        s["dst"][0].random_(-100, 100)
        before = s["dst"][0].clone()
        B.dflash_kv_evict(*s["args"])
        torch.cuda.synchronize()
        assert B.dflash_get_status(s["ws"]) == (-1, 584)
        assert torch.equal(s["dst"][0], before) and not torch.equal(pool, before)


def test_evict_reports_bad_pages_and_lengths():
    B = B_()
    base = dict(ctx=[60, 50], keep=[30, 30], hkv=1, d=64)
    s = evict_case(**base)
    s["td"][1][0, 1] = 999                     # a target page: its positions are dropped
    s["dst"][0].zero_()
    B.dflash_kv_evict(*s["args"])
    assert B.dflash_get_status(s["ws"]) == (-3, 583)
    assert torch.count_nonzero(s["dst"][0][1, int(s["tables"][1][0, 1])]) == 0
    assert torch.count_nonzero(s["dst"][0][1, int(s["tables"][1][1, 1])]) > 0
    s = evict_case(**base)
    s["td"][0][1, :] = -1                      # source pages: zeros
    B.dflash_workspace_init(s["ws"])
    B.dflash_kv_evict(*s["args"])
    assert B.dflash_get_status(s["ws"]) == (-3, 585)
    assert torch.count_nonzero(s["dst"][0][1, int(s["tables"][1][1, 0])]) == 0
    for at, value, site in ((5, [10 ** 6, 50], 581), (6, [32, 10 ** 6], 582), (6, [30, 49], 582)):
        s = evict_case(**base)
        args = list(s["args"])
        args[at] = i32(value)
        B.dflash_kv_evict(*args)
        torch.cuda.synchronize()
        assert B.dflash_get_status(s["ws"]) == (-3, site)
