"""Operators of a long prompt on the GPU: bad input, values that a row must not
see, captured calls that share a workspace, far pages, and a run of the operators
together as they are used."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as O
from test_gpu_prompt import (PAGE, B_, Cache, built, check_chunk, check_mass, chunk_case, heads, i32,  # noqa: F401
                             logits, mass_case, workspace)

pytestmark = pytest.mark.gpu


def test_chunk_reports_bad_rows_lengths_and_pages():
    """The requests that are at fault are skipped or cut, the others as always."""
    B = B_()
    for start in ([0, 5, 31, 30], [0, 5, 40, 30], [-2, 5, 25, 30]):   # (ranges must not overlap)
        s = chunk_case([5, 20, 5], [50, 60, 70], 8, 2, 64, seed=1)
        s["out"].fill_(7.0)
        s["lse"].fill_(7.0)
        args = list(s["args"])
        args[3] = i32(start)
        B.dflash_attention_chunk(*args)
        torch.cuda.synchronize()
        assert B.dflash_get_status(s["ws"]) == (-3, 551)
        # request 0 is right where its range is, request 2 where it still has its own rows
        good = [r for r in range(3) if 0 <= start[r] <= start[r + 1] <= 30 and [start[r], start[r + 1]] ==
                [int(s["start"][r]), int(s["start"][r + 1])]]
        for r in good:
            a, n, m = int(s["start"][r]), s["ns"][r], s["ctx"][r]
            k, v = s["c"].keys(r, 0, m)
            o, _, size = O.attend(s["q"][a:a + n].double().cpu().numpy(), k, v, 0.125, [m - n + i + 1 for i in range(n)])
            assert np.all(np.abs(s["out"][a:a + n].double().cpu().numpy() - o) <= 2.0 ** -7 * (size + np.abs(o)))
        B.dflash_workspace_init(s["ws"])
        B.dflash_attention_chunk(*s["args"])     # and the workspace is ready again
        check_chunk(s, 8, 64)
    s = chunk_case([9, 4], [48, 33], 8, 2, 64, seed=2)
    args = list(s["args"])
    args[9] = i32([49, 33])                      # the table holds 48 positions
    B.dflash_attention_chunk(*args)
    check_chunk(s, 8, 64, status=(-3, 552))
    for d, bad in ((64, 1 << 30), (128, -1)):
        s = chunk_case([40, 3], [300, 100], 8, 2, d, seed=3)
        s["c"].table_d[0, 3] = bad               # positions 48 .. 63 of request 0 read as zeros
        B.dflash_attention_chunk(*s["args"])
        s["c"].pool[0, s["c"].ids[0][3]] = 0
        check_chunk(s, 8, d, status=(-3, 553))


def test_mass_reports_bad_rows_lengths_and_pages():
    B = B_()
    s = mass_case([5, 20], [50, 60], 8, 2, 64, seed=1)
    ws = s["mass_args"][-1]
    for at, value, site in ((3, [1, 6, 3], 561), (10, [50, 10 ** 6], 562)):
        args = list(s["mass_args"])
        args[at] = i32(value)
        B.dflash_attention_mass(*args)
        torch.cuda.synchronize()
        assert B.dflash_get_status(ws) == (-3, site)
        B.dflash_workspace_init(ws)
    short = torch.full((2, 2, 55), 3.0, device="cuda")      # room for 55 positions of 60
    args = list(s["mass_args"])
    args[12] = short
    B.dflash_attention_mass(*args)
    assert B.dflash_get_status(ws) == (-3, 564)
    B.dflash_attention_mass(*s["mass_args"])
    assert torch.equal(short[1], s["mass"][1, :, :55]) and torch.equal(short[0, :, :50], s["mass"][0, :, :50])
    assert torch.all(short[0, :, 50:] == 3.0)
    B.dflash_workspace_init(ws)
    s["mass"].copy_(s["mass0"])                 # (a length of 10^6 counted as the table's 64)
    s["c"].table_d[1, 1] = 10 ** 7
    B.dflash_attention_mass(*s["mass_args"])
    assert B.dflash_get_status(ws) == (-3, 563)
    s["c"].pool[0, s["c"].ids[1][1]] = 0
    check_mass(s, 8, 64)


NOT_FINITE = [  # rows, ctx, hq, hkv, d
    ([5, 1], [165, 40], 8, 4, 64),
    ([130, 7], [400, 7], 8, 2, 128),            # several units, keys of later units
    ([33], [4000], 4, 1, 128),                  # cut into pieces
    ([300], [300], 2, 2, 64),                   # 256 rows per unit
    ([40], [17], 8, 2, 128),                    # rows before the start
]


@pytest.mark.parametrize("ns,ctx,hq,hkv,d", NOT_FINITE)
def test_chunk_keys_that_only_later_rows_see_may_hold_anything(ns, ctx, hq, hkv, d):
    """An infinity or NaN in K or V of a row's own position changes no bit of the rows
    before it, nor of other heads and requests; the rows that see it in V are not
    finite.  The same K spoils its own mass alone."""
    B = B_()
    s = mass_case(ns, ctx, hq, hkv, d, seed=ns[0])
    out, lse, pool, mass = \
        (s["out"].clone(), s["lse"].clone(), s["c"].pool.clone(), s["mass"].clone())
    G, bad, tries = hq // hkv, [float("nan"), float("inf"), float("-inf")], 0
    for r, (n, m) in enumerate(zip(ns, ctx)):
        for back in sorted({1, 2, n // 3, n // 2, n - 1, n}):       # the position of row n - back
            pos = m - back
            if back < 1 or pos < 0 or back > n:
                continue
            for plane in (0, 1):
                h, col = (r + back) % hkv, (7 * back + 3 * r) % d
                s["c"].pool.copy_(pool)
                s["c"].pool[0, s["c"].ids[r][pos // PAGE], plane, h, pos % PAGE, col] = bad[tries % 3]
                tries += 1
                B.dflash_attention_chunk(*s["args"])
                sees = torch.zeros(s["T"], hq, dtype=torch.bool, device="cuda")
                a = int(s["start"][r])
                sees[a + n - back:a + n, h * G:(h + 1) * G] = True
                assert torch.equal(s["out"][~sees], out[~sees]), (r, back, plane)
                assert torch.equal(s["lse"][~sees], lse[~sees]), (r, back, plane)
                if plane == 1:
                    assert not torch.isfinite(s["out"][sees]).all(-1).any(), (r, back)
                else:
                    args = list(s["mass_args"])
                    args[11], args[13] = lse, False
                    B.dflash_attention_mass(*args)
                    other = torch.ones_like(mass, dtype=torch.bool)
                    other[r, h, pos] = False
                    assert torch.equal(s["mass"][other], mass[other]), (r, back)
    assert tries > 0 and B.dflash_get_status(s["ws"]) == (0, 0)


def test_chunk_far_pages():
    """Pages whose element offsets pass 32 bits, and rows far apart."""
    B = B_()
    hq, hkv, d = 8, 8, 128
    n_pages = (1 << 32) // (2 * hkv * PAGE * d) + 40
    pool = torch.empty((1, n_pages, 2, hkv, PAGE, d), dtype=torch.bfloat16, device="cuda")
    ids = [[*range(n_pages - 30, n_pages - 20), n_pages - 1], [n_pages - 3, 0]]
    for i in sorted({i for row in ids for i in row}):
        pool[0, i] = torch.randn(pool.shape[2:], device="cuda").to(torch.bfloat16)
    c = Cache(1, hkv, d, [1])
    c.pool, c.ids = pool, ids
    table = i32([ids[0], ids[1] + [0] * 9])
    c.kv = B.DflashKV(pool=pool.data_ptr(), page_table=table.data_ptr(), n_pages=n_pages, max_pages=11, n_rows=2,
                      dtype=0, scales=None)
    width = 1 << 27                              # elements between rows: 40 of them pass 32 bits
    buf = torch.empty(40 * width, dtype=torch.bfloat16, device="cuda")
    q = buf.view(40, width)[:, :hq * d].unflatten(1, (hq, d))
    out = buf.view(40, width)[:, hq * d:2 * hq * d].unflatten(1, (hq, d))
    q.copy_(torch.randn(40, hq, d, device="cuda"))
    out.fill_(7.0)
    lse = torch.full((40, hq), 7.0, device="cuda")
    hd = heads(1, hq, hkv, d)
    ws = workspace(B.dflash_attention_chunk_bytes(hd, 2, 40))
    ns, ctx, start = [20, 19], [170, 21], [0, 20, 39]
    B.dflash_attention_chunk(hd, 0, q, i32(start), 2, 40, True, 0.0, c.kv, i32(ctx), out, lse, ws)
    torch.cuda.synchronize()
    s = dict(c=c, q=q, out=out, lse=lse, ws=ws, start=np.array(start), ns=ns, ctx=ctx, T=40)
    check_chunk(s, hq, d)
    mass = torch.zeros(2, hkv, 170, device="cuda")
    s["mass0"], s["mass"] = mass.clone(), mass
    B.dflash_attention_mass(hd, 0, q, i32(start), 2, 40, 0, True, 0.0, c.kv, i32(ctx), lse, mass, False, ws)
    check_mass(s, hq, d)
    # eviction from and to such pages of one pool
    to = i32([[n_pages - 10, n_pages - 11], [n_pages - 12, 5]])
    dst = B.DflashKV(pool=pool.data_ptr(), page_table=to.data_ptr(), n_pages=n_pages, max_pages=2, n_rows=2, dtype=0,
                     scales=None)
    kept = torch.zeros(2, hkv, 32, dtype=torch.int32, device="cuda")
    wse = workspace(B.dflash_kv_evict_bytes(hd, 2, n_pages))
    B.dflash_kv_evict(hd, 0, c.kv, dst, 2, i32(ctx), i32([32, 17]), 1, 2, mass, kept, None, None, wse)
    assert B.dflash_get_status(wse) == (0, 0)
    for r, n in enumerate((32, 17)):
        for h in range(hkv):
            k = O.evict(mass[r, h].cpu().numpy(), ctx[r], n, 1, 2)
            assert kept[r, h, :n].tolist() == k
            for i in (0, n // 2, n - 1):
                assert torch.equal(pool[0, int(to[r, i // 16]), :, h, i % 16], pool[0, ids[r][k[i] // 16], :, h, k[i] % 16])


def test_graphs_that_share_a_workspace():
    """Captured calls of different shapes (with and without a second kernel, and a mass)
    over one workspace, replayed in turn with lengths that changed since the capture."""
    B = B_()
    shapes = [dict(ns=[1] * 6, ctx=[700 + 300 * i for i in range(6)], hq=16, hkv=2, d=128),
              dict(ns=[90, 40, 2], ctx=[90, 400, 200], hq=8, hkv=2, d=64),
              dict(ns=[4], ctx=[3000], hq=8, hkv=1, d=128)]
    cases = [mass_case(seed=i, **x) for i, x in enumerate(shapes)]
    ws = workspace(max(s["ws"].nbytes for s in cases))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for s in cases:
        lens = i32(s["ctx"])
        s["lens"] = lens
        a, m = list(s["args"]), list(s["mass_args"])
        a[9], a[12], m[10], m[14] = lens, ws, lens, ws
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            B.dflash_attention_chunk(*a)
            B.dflash_attention_mass(*m)
        graphs.append(graph)
    full = [list(s["ctx"]) for s in cases]
    for cut in (0, 30, 89, 7):
        for s, graph, lens in zip(cases, graphs, full):
            s["ctx"] = [c - cut for c in lens]
            s["out"].fill_(7.0)
            s["lse"].fill_(7.0)
            s["mass"].copy_(s["mass0"])
            s["lens"].copy_(i32(s["ctx"]))
            graph.replay()
        torch.cuda.synchronize()
        for s, x in zip(cases, shapes):
            s["ws"] = ws
            check_chunk(s, x["hq"], x["d"])
            check_mass(s, x["hq"], x["d"])


def test_calls_repeat_bit_for_bit_and_on_another_stream():
    B = B_()
    side = torch.cuda.Stream()
    for ns, ctx in (([300, 1, 45], [4000, 900, 45]), ([1, 1], [9000, 30])):
        s = mass_case(ns, ctx, 16, 4, 128, seed=ns[0])
        first = s["out"].clone(), s["lse"].clone(), s["mass"].clone()
        for k in ("out", "lse", "mass"):
            s[k].fill_(7.0)
        s["mass"].copy_(s["mass0"])
        side.wait_stream(torch.cuda.current_stream())
        B.dflash_attention_chunk(*s["args"], stream=side)
        B.dflash_attention_mass(*s["mass_args"], stream=side)
        side.synchronize()
        rows = slice(int(s["start"][0]), int(s["start"][-1]))
        assert torch.equal(s["out"][rows], first[0][rows]) and torch.equal(s["lse"][rows], first[1][rows])
        assert torch.equal(s["mass"], first[2])


def test_prompt_in_chunks_together_with_eviction_and_decode():
    """A prompt appended and attended in chunks, its last rows' weights summed, the cache cut
    to the heaviest positions, and tokens decoded from what is left; through the
    cache's own methods, against the oracle."""
    B = B_()
    import workload as W
    from block_diffusion_speculative_fuse_gb300.device import PagedKV
    hq, hkv, d, vocab = 8, 2, 64, 512
    G = hq // hkv
    shape = W.ModelShape(n_layers=2, hidden=256, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, mlp=256, vocab=vocab)
    lens, keep, layer = [150, 61], [48, 61], 1
    batch, per = 2, 12
    big = PagedKV(shape, np.random.default_rng(0).permutation(2 * per).reshape(2, per), 2 * per)
    small = PagedKV(shape, np.arange(10).reshape(2, 5), 10)
    g = torch.Generator(device="cuda").manual_seed(6)
    rope = B.dflash_rope_init(d, base=1e4)
    f, mag = O.rope_freqs(d, 1e4)
    ws = big.chunk_workspace(hq, batch, 256)
    mass = torch.zeros(batch, hkv, per * PAGE, device="cuda")
    seq = [torch.randn(n + 3, (hq + 2 * hkv) * d, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    parts = lambda x: (t.unflatten(1, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], 1))  # noqa: E731

    def rows(cache, x, req, pos):
        q, k, v = parts(x)
        qo = torch.empty(x.shape[0], hq, d, dtype=torch.bfloat16, device="cuda")
        cache.append_rotated(rope, layer, q, k, v, i32(req), i32(pos), ws, q_out=qo)
        return qo

    def oracle(q, k, v, limits):
        o, lse, size = O.attend(q.double().cpu().numpy(), k, v, 0.125, limits)
        return o, lse, 2.0 ** -7 * (size + np.abs(o)) + 1e-6

    # chunks of 64: what a request has of them
    queries = [[], []]
    for at in (0, 64, 128):
        ns = [max(0, min(64, n - at)) for n in lens]
        x = torch.cat([s[at:at + n] for s, n in zip(seq, ns)])
        req = np.repeat([0, 1], ns)
        pos = np.concatenate([at + np.arange(n) for n in ns])
        q = rows(big, x, req, pos)
        start, ctx = i32([0, ns[0], sum(ns)]), i32([min(n, at + 64) for n in lens])
        out, lse = torch.zeros_like(q), torch.zeros(sum(ns), hq, device="cuda")
        big.attend_chunk(layer, q, start, ctx, out, ws, lse=lse)
        big.attention_mass(layer, q, start, ctx, lse, mass, ws, last=16)
        for r in range(batch):
            mine = slice(0, ns[0]) if r == 0 else slice(ns[0], sum(ns))
            if ns[r] == 0:
                continue
            k, v = (t.double().cpu().numpy() for t in big.read_logical(layer, r, min(lens[r], at + 64)))
            o, le, tol = oracle(q[mine], k, v, [at + i + 1 for i in range(ns[r])])
            assert np.all(np.abs(out[mine].double().cpu().numpy() - o) <= tol)
            queries[r].append((q[mine], le, at, ns[r]))
    total = np.zeros((batch, hkv, per * PAGE))
    for r in range(batch):
        for q, le, at, n in queries[r]:
            w, m = min(n, 16), min(lens[r], at + 64)
            k, _ = (t.double().cpu().numpy() for t in big.read_logical(layer, r, m))
            total[r, :, :m] += O.attention_mass(q[n - w:].double().cpu().numpy(), k, le[n - w:], 0.125,
                                                [m - w + i + 1 for i in range(w)])
    assert np.allclose(mass.cpu().numpy(), total, rtol=2e-5, atol=1e-9)
    # cut, and three tokens on from it: keys keep their angles, new rows go on from the old length
    kept, new_len = torch.zeros(batch, hkv, 61, dtype=torch.int32, device="cuda"), i32([0, 0])
    left = torch.zeros_like(mass)
    wse = small.evict_workspace(batch)
    big.evict_to(small, layer, i32(lens), i32(keep), mass, kept, wse, sink=2, recent=8, new_len=new_len, mass_out=left)
    assert new_len.tolist() == [48, 61] and B.dflash_get_status(wse) == (0, 0)
    mine = [[O.evict(mass[r, h].cpu().numpy(), lens[r], keep[r], 2, 8) for h in range(hkv)] for r in range(batch)]
    full = [[t.double().cpu().numpy() for t in big.read_logical(layer, r, lens[r])] for r in range(batch)]
    for r in range(batch):
        k, v = (t.double().cpu().numpy() for t in small.read_logical(layer, r, keep[r]))
        for h in range(hkv):
            assert kept[r, h, :keep[r]].tolist() == mine[r][h]
            assert np.array_equal(k[:, h], full[r][0][mine[r][h], h]) and np.array_equal(v[:, h], full[r][1][mine[r][h], h])
            assert torch.equal(left[r, h, :keep[r]], mass[r, h, torch.tensor(mine[r][h]).cuda()])
    for i in range(3):
        x = torch.stack([seq[r][lens[r] + i] for r in range(batch)])
        q, k, v = parts(x)
        turned = O.rotate(k.double().cpu().numpy(), [lens[r] + i for r in range(batch)], f, mag, False)
        # (the append stores at the position it rotates by: rotated rows go in unrotated)
        kr = torch.from_numpy(turned).cuda().to(torch.bfloat16)
        qr = torch.from_numpy(O.rotate(q.double().cpu().numpy(), [lens[r] + i for r in range(batch)], f, mag, False))
        qr = qr.cuda().to(torch.bfloat16)
        small.append_rotated(B.dflash_rope_init(0), layer, None, kr, v.contiguous(), i32([0, 1]),
                             i32([keep[r] + i for r in range(batch)]), ws)
        out = torch.zeros(batch, hq, d, dtype=torch.bfloat16, device="cuda")
        small.attend_chunk(layer, qr, i32([0, 1, 2]), i32([keep[r] + i + 1 for r in range(batch)]), out, ws)
        for r in range(batch):
            kk, vv = (t.double().cpu().numpy() for t in small.read_logical(layer, r, keep[r] + i + 1))
            assert np.array_equal(kk[-1], kr[r].double().cpu().numpy())
            o, _, tol = oracle(qr[r:r + 1], kk, vv, [keep[r] + i + 1])
            assert np.all(np.abs(out[r:r + 1].double().cpu().numpy() - o) <= tol)
    assert B.dflash_get_status(ws) == (0, 0)


def test_evict_captured_and_replayed():
    """With lengths, budgets and masses that changed since the capture."""
    B = B_()
    from test_gpu_prompt import check_evict, evict_case
    ctx, keep = [5000, 77, 900], [700, 60, 899]
    s = evict_case(ctx, keep, 2, 128, 2, 9, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.dflash_kv_evict(*s["args"])
    for i in range(3):
        ctx2, keep2 = [c - 13 * i for c in ctx], [max(0, k - 40 * i) for k in keep]
        s["args"][5].copy_(i32(ctx2))
        s["args"][6].copy_(i32(keep2))
        s["mass"].copy_(torch.rand_like(s["mass"]))
        for k in ("kept", "new_len", "mass_out"):
            s[k].fill_(-9)
        s["before"][2] = s["dst"][0].clone()
        s["new"] = [min(k, c) for k, c in zip(keep2, ctx2)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_evict(s, ctx2, keep2, 2, 2, 9)


def test_score_captured_and_replayed():
    B = B_()
    z = logits(5, 30000, seed=2)
    ids, top = i32([3, -1, 29999, 8, 100]), 6
    outs = (torch.zeros(5, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(5, device="cuda"))
    ti, tl = torch.zeros(5, top, dtype=torch.int32, device="cuda"), torch.zeros(5, top, device="cuda")
    ws = workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.dflash_score_tokens(z, 5, 30000, None, ids, *outs, top, ti, tl, ws)
    for seed in (3, 4):
        z.copy_(logits(5, 30000, seed=seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for r in range(5):
            e = O.score(z[r].double().cpu().numpy(), 1.0, int(ids[r]), top)
            assert abs(float(outs[0][r]) - e[0]) < 2e-5 and int(outs[1][r]) == e[1] and ti[r].tolist() == e[3]
            assert abs(float(outs[2][r]) - e[2]) < 2e-5
    assert B.dflash_get_status(ws) == (0, 0)


def test_scored_sequences_are_the_targets_own_logits():
    """score_sequences against the logits of one forward over the whole sequences; the same
    for every chunk size, since a row does not depend on the call's other rows."""
    import workload as W
    from block_diffusion_speculative_fuse_gb300.device import DeviceModel
    from block_diffusion_speculative_fuse_gb300.generate import TargetRunner, score_sequences
    t = W.get_workload("tiny_e2e").target
    shared, tw = W.shared_weights(t, 71, std=0.05), W.target_weights(t, 71, std=0.05)
    model = DeviceModel(t, tw, shared, draft=False)
    tokens = np.random.default_rng(2).integers(0, t.vocab, (3, 14)).astype(np.int32)
    z = torch.empty((3 * 13, t.vocab), dtype=torch.float32, device="cuda")
    TargetRunner(model, 3, 32, 13).forward(i32(tokens[:, :-1]), i32([0, 0, 0]), 13, logits=z)
    z = z.view(3, 13, -1).double().cpu().numpy()
    T = [1.0, 0.7, 1.3]
    first = None
    for chunk in (64, 5, 1):
        res = score_sequences(TargetRunner(model, 3, 32, 13), tokens, n_top=4, temperature=T, chunk=chunk)
        assert res["logprob"].shape == (3, 13) and res["top_id"].shape == (3, 13, 4)
        for r in range(3):
            for i in range(13):
                e = O.score(z[r, i], float(np.float32(T[r])), int(tokens[r, i + 1]), 4)
                tol = 2.0 ** -22 * (16 + math.log(t.vocab)) * 4
                assert abs(res["logprob"][r, i] - e[0]) <= tol and abs(res["entropy"][r, i] - e[2]) <= tol
                assert res["rank"][r, i] == e[1] and list(res["top_id"][r, i]) == e[3]
                assert np.all(np.abs(res["top_logprob"][r, i] - e[4]) <= tol)
        if first is None:
            first = res
        assert all(np.array_equal(res[k], first[k]) for k in res)
    plain = score_sequences(TargetRunner(model, 3, 32, 13), tokens)
    assert sorted(plain) == ["entropy", "logprob", "rank"] and np.array_equal(plain["rank"], first["rank"])
