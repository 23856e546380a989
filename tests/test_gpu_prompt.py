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
