"""Cases for the operators of a long prompt over the paged K/V cache.

Four operators that a program with projections of its own uses one after the
other:

* chunk: attention of a ragged batch of new tokens to the paged cache
  (dflash_attention_chunk);
* mass: the attention weight that each cached key receives from the last rows
  (dflash_attention_mass);
* evict: the heaviest positions of each request and KV head, moved together
  into other pages (dflash_kv_evict);
* score: log probability, rank, entropy and the best alternatives of given
  tokens (dflash_score_tokens).

``run`` computes them with elementary torch operations, or through the
framework's entry points where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one request: a call's latency
        dict(name="chunk_token", op="chunk", reqs=1, n=1, single=0, hq=32, hkv=8, d=128, past=4095,
             ragged=False, causal=True, pad=0, strided=False),
        # two short chunks of small heads in odd number, rows to spare: a small odd call
        dict(name="chunk_small_odd", op="chunk", reqs=2, n=37, single=1, hq=15, hkv=5, d=64, past=211,
             ragged=True, causal=True, pad=5, strided=True),
        # 8 prompts of 1024 tokens from an empty cache
        dict(name="chunk_prompts_8x1024", op="chunk", reqs=8, n=1024, single=0, hq=32, hkv=8, d=128,
             past=0, ragged=False, causal=True, pad=0, strided=False),
        # a server's mixed step: 32 requests decode one token, one brings 2000 of its prompt
        dict(name="chunk_mixed_b33", op="chunk", reqs=1, n=2000, single=32, hq=32, hkv=8, d=128,
             past=6192, ragged=False, causal=True, pad=0, strided=True),
        # 4096 tokens of a long prompt behind 28672 cached ones
        dict(name="chunk_4096_at_32k", op="chunk", reqs=1, n=4096, single=0, hq=32, hkv=8, d=128,
             past=28672, ragged=False, causal=True, pad=0, strided=False),
        # what the last 32 tokens of 8 prompts attended to
        dict(name="mass_window_8x16k", op="mass", reqs=8, n=48, last=32, hq=32, hkv=8, d=128,
             past=16336, ragged=False, causal=True, add=False),
        # three requests of odd length, every row of a small chunk, added up
        dict(name="mass_small_odd", op="mass", reqs=3, n=21, last=0, hq=12, hkv=4, d=64, past=300,
             ragged=True, causal=True, add=True),
        # 32 requests of 8192 positions cut to a quarter
        dict(name="evict_32x8k", op="evict", reqs=32, ctx=8192, keep=2048, sink=4, recent=64, hkv=8,
             d=128, ragged=False),
        # one long request cut to an eighth
        dict(name="evict_one_96k", op="evict", reqs=1, ctx=98304, keep=12288, sink=4, recent=256,
             hkv=8, d=128, ragged=False),
        # one token at the drafter's vocabulary with 20 alternatives: a call's latency
        dict(name="score_one", op="score", rows=1, vocab=151936, top=20, half=False, temp=False,
             spread=2.2),
        # the rows of a 2048-token prompt at the drafter's vocabulary
        dict(name="score_prompt_2048", op="score", rows=2048, vocab=151936, top=5, half=False,
             temp=False, spread=2.2),
        # bf16 logits of an odd vocabulary, own temperatures
        dict(name="score_bf16_odd", op="score", rows=301, vocab=32003, top=8, half=True, temp=True,
             spread=3.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "mass", "evict", "score"])
    if op in ("chunk", "mass"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 5, 8])
        hq = hkv * rng.choice([1, 2, 3, 4])
        reqs = _log(rng, 1, 8)
        if op == "mass":
            n = _log(rng, 1, 64)
            return dict(op=op, reqs=reqs, n=n, last=rng.choice([0, 1, 16, 32]), hq=hq, hkv=hkv, d=d,
                        past=_log(rng, 1, 16384), ragged=rng.random() < 0.5,
                        causal=rng.random() < 0.8, add=rng.random() < 0.5)
        n = _log(rng, 1, 4096 // reqs)
        return dict(op=op, reqs=reqs, n=n, single=rng.choice([0, 0, 1, 7, 32]), hq=hq, hkv=hkv, d=d,
                    past=_log(rng, 1, 25000 // reqs) - 1, ragged=rng.random() < 0.5,
                    causal=rng.random() < 0.8, pad=rng.choice([0, 0, 3]),
                    strided=rng.random() < 0.5)
    if op == "evict":
        reqs = _log(rng, 1, 32)
        ctx = _log(rng, 20, min(98304, 262144 // reqs))
        return dict(op=op, reqs=reqs, ctx=ctx, keep=_log(rng, 1, max(2, ctx // 2)),
                    sink=rng.choice([0, 1, 4]), recent=rng.choice([0, 1, 16, 64]),
                    hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                    ragged=rng.random() < 0.5)
    return dict(op=op, rows=_log(rng, 1, 1024), vocab=_log(rng, 2, 151936),
                top=rng.choice([0, 1, 5, 20]), half=rng.random() < 0.4, temp=rng.random() < 0.5,
                spread=rng.uniform(0.5, 4.0))


def _lengths(case):
    """Rows and cached positions (its rows' own among them) of each request."""
    rnd = np.random.default_rng([case["reqs"], case["n"], case["past"]])
    n = np.full(case["reqs"], case["n"])
    past = np.full(case["reqs"], case["past"])
    if case["ragged"]:
        n = rnd.integers(1, case["n"] + 1, case["reqs"])
        past = rnd.integers(0, case["past"] + 1, case["reqs"])
    single = case.get("single", 0)   # requests that bring one token, anywhere in the batch
    at = np.sort(rnd.integers(0, case["reqs"] + 1, single))
    n = np.insert(n, at, 1)
    past = np.insert(past, at, rnd.integers(case["past"] // 2, case["past"] + 1, single))
    return n, past + n


def work(case):
    if case["op"] in ("chunk", "mass"):
        n, ctx = _lengths(case)
        G, d, hkv = case["hq"] // case["hkv"], case["d"], case["hkv"]
        pairs = rows = 0
        for a, c in zip(n.tolist(), ctx.tolist()):
            w = min(a, case["last"]) if case.get("last") else a
            rows += w
            pairs += w * c - (w * (w - 1) // 2 if case["causal"] else 0)
        keys = int(ctx.sum())
        if case["op"] == "chunk":
            return {"bytes": rows * hkv * G * (4 * d + 4) + 4 * d * hkv * keys,
                    "flops": 4 * d * hkv * G * pairs}
        return {"bytes": rows * hkv * G * (2 * d + 4) + hkv * keys * (2 * d + (8 if case["add"] else 4)),
                "flops": 2 * d * hkv * G * pairs}
    if case["op"] == "evict":
        ctx, keep = _evict_lengths(case)
        new = int(np.minimum(ctx, keep).sum())
        # the masses, the kept vectors in and out, their positions and masses
        return {"bytes": case["hkv"] * (4 * int(ctx.sum()) + new * (8 * case["d"] + 8)),
                "flops": case["hkv"] * int(ctx.sum())}
    size = 2 if case["half"] else 4
    return {"bytes": case["rows"] * (size * case["vocab"] + 20 + 8 * case["top"]),
            "flops": 6 * case["rows"] * case["vocab"]}


# --------------------------------------------------------------------- inputs
def _generators(seed):
    gpu = torch.Generator(device="cuda")
    gpu.manual_seed(seed)
    return gpu, np.random.default_rng(seed)


def _paged_rows(lengths, rnd, spare=3):
    """A page table over a shuffled pool for requests of these lengths."""
    need = [(int(n) + PAGE - 1) // PAGE for n in lengths]
    pages = rnd.permutation(sum(need) + spare).astype(np.int32)
    table = np.zeros((len(need), max(1, max(need))), np.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = pages[at:at + k]
        at += k
    return table, sum(need) + spare


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).cuda()


def _chunk_state(case, seed):
    gpu, rnd = _generators(seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n, ctx = _lengths(case)
    start = np.concatenate([[0], np.cumsum(n)])
    T = int(start[-1]) + case.get("pad", 0)
    table, n_pages = _paged_rows(ctx, rnd)
    pool = torch.randn(1, n_pages, 2, hkv, PAGE, d, generator=gpu, device="cuda").to(torch.bfloat16)
    # strided: q as the columns of a fused projection, whose width is out's too
    wide = (hq + 2 * hkv) * d if case.get("strided") else hq * d
    q = (1.5 * torch.randn(T, wide, generator=gpu, device="cuda")).to(torch.bfloat16)
    s = dict(case=case, pool=pool, table=_i32(table), n_pages=n_pages, T=T, batch=len(n),
             start=_i32(start), ctx=_i32(ctx), rows=n.tolist(), lens=ctx.tolist(),
             q=q[:, :hq * d].unflatten(1, (hq, d)))
    if case["op"] == "chunk":
        s["out"] = torch.zeros(T, wide, dtype=torch.bfloat16, device="cuda")[:, :hq * d].unflatten(1, (hq, d))
        s["lse"] = torch.zeros(T, hq, dtype=torch.float32, device="cuda")
        return s
    # what an attention call over the same rows leaves
    s["lse"] = _attend(s, torch.float32)["lse"].contiguous()
    s["mass0"] = torch.rand(len(n), hkv, int(ctx.max()), generator=gpu, device="cuda")
    s["mass"] = s["mass0"].clone()
    return s


def _evict_lengths(case):
    rnd = np.random.default_rng([case["reqs"], case["ctx"], case["keep"]])
    ctx, keep = np.full(case["reqs"], case["ctx"]), np.full(case["reqs"], case["keep"])
    if case["ragged"]:
        ctx = rnd.integers(0, case["ctx"] + 1, case["reqs"])
        keep = rnd.integers(1, case["keep"] + 1, case["reqs"])
    return ctx, keep


def _evict_state(case, seed):
    gpu, rnd = _generators(seed)
    hkv, d = case["hkv"], case["d"]
    ctx, keep = _evict_lengths(case)
    table, n_pages = _paged_rows(ctx, rnd)
    to_table, to_pages = _paged_rows(np.minimum(ctx, keep), rnd)
    # a pool of the cache's values; masses as attention leaves them: few heavy keys, many of
    # about none, some exactly none
    pool = torch.randn(1, n_pages, 2, hkv, PAGE, d, generator=gpu, device="cuda").to(torch.bfloat16)
    width = max(1, int(ctx.max()))
    mass = torch.exp(3.0 * torch.randn(case["reqs"], hkv, width, generator=gpu, device="cuda") - 6.0)
    mass = torch.where(mass < 2e-5, 0.0, mass)
    return dict(case=case, pool=pool, table=_i32(table), n_pages=n_pages, mass=mass,
                ctx=_i32(ctx), keep=_i32(keep), lens=ctx.tolist(), keeps=keep.tolist(),
                to_pool=torch.zeros(1, to_pages, 2, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda"),
                to_table=_i32(to_table), to_pages=to_pages,
                kept=torch.zeros(case["reqs"], hkv, int(keep.max()), dtype=torch.int32, device="cuda"),
                new_len=torch.zeros(case["reqs"], dtype=torch.int32, device="cuda"),
                mass_out=torch.zeros_like(mass))


def _score_state(case, seed):
    gpu, rnd = _generators(seed)
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    z = case["spread"] * torch.randn(rows, vocab, generator=gpu, device="cuda")
    # a few likely tokens above the bulk, as a trained model's rows have
    many = min(24, vocab)
    likely = (rnd.integers(0, vocab, (rows, 1)) + np.arange(many) * (vocab // many)) % vocab
    z.scatter_add_(1, torch.from_numpy(likely).cuda(),
                   torch.from_numpy(rnd.exponential(3.0, (rows, many)).astype(np.float32)).cuda())
    # a grammar's masked tokens
    z[:, vocab // 3:vocab // 3 + vocab // 50] = float("-inf")
    # given tokens: most of them likely ones, a few rows without one
    ids = np.where(rnd.random(rows) < 0.7, likely[:, 0], rnd.integers(0, vocab, rows))
    ids = np.where(rnd.random(rows) < 0.05, -1, ids)
    return dict(case=case, z=z.to(torch.bfloat16) if case["half"] else z, ids=_i32(ids),
                T=torch.from_numpy(rnd.choice([0.6, 0.8, 1.0, 1.5], rows).astype(np.float32)).cuda()
                if case["temp"] else None,
                logprob=torch.zeros(rows, dtype=torch.float32, device="cuda"),
                rank=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                entropy=torch.zeros(rows, dtype=torch.float32, device="cuda"),
                top_id=torch.zeros(rows, top, dtype=torch.int32, device="cuda") if top else None,
                top_lp=torch.zeros(rows, top, dtype=torch.float32, device="cuda") if top else None)


def prepare(case, seed):
    return {"chunk": _chunk_state, "mass": _chunk_state, "evict": _evict_state,
            "score": _score_state}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _request(s, r, dt):
    """q [hkv][rows * G][d], K and V [hkv][keys][d] of request r and the number
    of keys that each of its rows sees."""
    case = s["case"]
    hkv, G, d = case["hkv"], case["hq"] // case["hkv"], case["d"]
    a, c = s["rows"][r], s["lens"][r]
    first = sum(s["rows"][:r])
    q = s["q"][first:first + a].to(dt).reshape(a, hkv, G, d).transpose(0, 1).reshape(hkv, a * G, d)
    pages = s["table"][r, :(c + PAGE - 1) // PAGE].long()
    k, v = (s["pool"][0, pages, i].to(dt).transpose(0, 1).reshape(hkv, -1, d)[:, :c] for i in (0, 1))
    row = torch.arange(a, device="cuda")
    seen = c - a + 1 + row if case["causal"] else torch.full_like(row, c)
    return first, q, k, v, seen


def _attend(s, dt):
    """out and lse of every row, one request and KV head at a time, at most
    2^29 scores at once."""
    case = s["case"]
    hkv, G, d = case["hkv"], case["hq"] // case["hkv"], case["d"]
    out = torch.zeros(s["T"], case["hq"], d, dtype=dt, device="cuda")
    lse = torch.zeros(s["T"], case["hq"], dtype=dt, device="cuda")
    for r, a in enumerate(s["rows"]):
        first, q, k, v, seen = _request(s, r, dt)
        keys = k.shape[1]
        if a * G * keys * hkv <= 1 << 29:
            groups = [slice(0, hkv)]
        else:
            groups = [slice(h, h + 1) for h in range(hkv)]
        hidden = torch.arange(keys, device="cuda") >= seen.repeat_interleave(G)[:, None]
        for h in groups:
            x = (q[h] @ k[h].transpose(1, 2)) * (1.0 / math.sqrt(d))
            x.masked_fill_(hidden, float("-inf"))
            m = x.amax(-1, keepdim=True)
            x = torch.exp(x - m)
            total = x.sum(-1, keepdim=True)
            o = (x @ v[h]) / total
            nh = o.shape[0]
            at = slice(h.start * G, h.stop * G)
            out[first:first + a, at] = o.view(nh, a, G, d).transpose(0, 1).reshape(a, nh * G, d)
            lse[first:first + a, at] = (m + torch.log(total)).view(nh, a, G).transpose(0, 1).reshape(a, nh * G)
    return {"out": out, "lse": lse}


def _chunk_plain(s):
    res = _attend(s, torch.float32)
    live = sum(s["rows"])
    s["out"][:live] = res["out"][:live].to(torch.bfloat16)
    s["lse"][:live] = res["lse"][:live]
    return {"out": s["out"], "lse": s["lse"]}


def _masses(s, dt):
    case = s["case"]
    hkv, G, d = case["hkv"], case["hq"] // case["hkv"], case["d"]
    mass = s["mass0"].to(dt).clone()
    for r, a in enumerate(s["rows"]):
        first, q, k, _, seen = _request(s, r, dt)
        w = min(a, case["last"]) if case["last"] else a
        x = (q[:, (a - w) * G:] @ k.transpose(1, 2)) * (1.0 / math.sqrt(d))
        lse = s["lse"][first + a - w:first + a].to(dt).view(w, hkv, G).transpose(0, 1).reshape(hkv, w * G, 1)
        hidden = torch.arange(k.shape[1], device="cuda") >= seen[a - w:].repeat_interleave(G)[:, None]
        x = torch.exp(x - lse).masked_fill_(hidden, 0.0).sum(1)
        c = s["lens"][r]
        mass[r, :, :c] = mass[r, :, :c] + x if case["add"] else x
    return mass


def _mass_plain(s):
    s["mass"].copy_(_masses(s, torch.float32))
    return {"mass": s["mass"]}


def _evict_plain(s):
    case = s["case"]
    hkv, d = case["hkv"], case["d"]
    for r, c in enumerate(s["lens"]):
        new = min(c, s["keeps"][r])
        if new == 0:
            continue
        weight = s["mass"][r, :, :c].clone()
        weight[:, :min(case["sink"], c)] = float("inf")
        weight[:, max(0, c - case["recent"]):] = float("inf")
        order = torch.sort(weight, dim=1, descending=True, stable=True)[1][:, :new]
        kept = torch.sort(order, dim=1)[0]                                    # [hkv, new]
        s["kept"][r, :, :new] = kept
        s["mass_out"][r, :, :new] = s["mass"][r].gather(1, kept)
        head = torch.arange(hkv, device="cuda")[:, None]
        page = s["table"][r].long()[kept // PAGE]
        at = torch.arange(new, device="cuda")
        to = s["to_table"][r].long()[at // PAGE]
        for i in (0, 1):
            s["to_pool"][0, to[None], i, head, (at % PAGE)[None]] = s["pool"][0, page, i, head, kept % PAGE]
    s["new_len"].copy_(torch.minimum(s["ctx"], s["keep"]))
    return {"pool": s["to_pool"], "kept": s["kept"], "new_len": s["new_len"], "mass": s["mass_out"]}


def _score_plain(s):
    case = s["case"]
    z = s["z"].float()
    rows, vocab = z.shape
    T = 1.0 if s["T"] is None else s["T"][:, None]
    top = z.amax(1, keepdim=True)
    t = (z - top) / T
    w = torch.exp(t)
    total = w.sum(1, keepdim=True)
    log_total = torch.log(total)
    s["entropy"].copy_((log_total - (w * torch.where(w > 0, t, 0.0)).sum(1, keepdim=True) / total)[:, 0])
    given = s["ids"] >= 0
    at = s["ids"].long().clamp(min=0)[:, None]
    zi = z.gather(1, at)
    s["logprob"].copy_(torch.where(given, (t.gather(1, at) - log_total)[:, 0], 0.0))
    better = (z > zi) | ((z == zi) & (torch.arange(vocab, device="cuda") < at))
    s["rank"].copy_(torch.where(given, better.sum(1), -1))
    res = {"logprob": s["logprob"], "rank": s["rank"], "entropy": s["entropy"]}
    if case["top"]:
        k = min(case["top"], vocab)
        order, index = torch.sort(z, dim=1, descending=True, stable=True)
        lp = (order[:, :k] - top) / T - log_total
        s["top_id"].fill_(-1)
        s["top_lp"].fill_(float("-inf"))
        s["top_id"][:, :k] = torch.where(lp > float("-inf"), index[:, :k], -1)
        s["top_lp"][:, :k] = lp
        res.update(top_id=s["top_id"], top_lp=s["top_lp"])
    return res


# --------------------------------------------------------- the framework's own
def _workspace(s, size):
    """The caller's workspace, allocated once and kept with its other buffers."""
    if "ws" not in s:
        from block_diffusion_speculative_fuse_gb300 import binding as B
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
        B.dflash_workspace_init(s["ws"])
    return s["ws"]


def _cache(s, pool, table, n_pages):
    """The library's descriptors of a cache, built once per cache."""
    if pool not in s.setdefault("caches", {}):
        from block_diffusion_speculative_fuse_gb300 import binding as B
        case = s["case"]
        heads = B.DflashHeads(n_layers=1, n_q_heads=case.get("hq", case["hkv"]), n_kv_heads=case["hkv"],
                              head_dim=case["d"], page_size=PAGE, kv_terms=1)
        kv = B.DflashKV(pool=s[pool].data_ptr(), page_table=s[table].data_ptr(), n_pages=s[n_pages],
                        max_pages=s[table].shape[1], n_rows=s[table].shape[0], dtype=0, scales=None)
        s["caches"][pool] = (heads, kv)
    return s["caches"][pool]


def _chunk_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    heads, kv = _cache(s, "pool", "table", "n_pages")
    ws = _workspace(s, lambda: B.dflash_attention_chunk_bytes(heads, s["batch"], s["T"]))
    B.dflash_attention_chunk(heads, 0, s["q"], s["start"], s["batch"], s["T"], s["case"]["causal"], 0.0,
                             kv, s["ctx"], s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _mass_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    heads, kv = _cache(s, "pool", "table", "n_pages")
    ws = _workspace(s, lambda: B.dflash_attention_mass_bytes(heads, s["batch"], s["T"]))
    if s["case"]["add"]:
        s["mass"].copy_(s["mass0"])   # the running sums, which the call adds to
    B.dflash_attention_mass(heads, 0, s["q"], s["start"], s["batch"], s["T"], s["case"]["last"],
                            s["case"]["causal"], 0.0, kv, s["ctx"], s["lse"], s["mass"],
                            s["case"]["add"], ws)
    return {"mass": s["mass"]}


def _evict_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    case = s["case"]
    heads, src = _cache(s, "pool", "table", "n_pages")
    _, dst = _cache(s, "to_pool", "to_table", "to_pages")
    ws = _workspace(s, lambda: B.dflash_kv_evict_bytes(heads, case["reqs"], s["to_pages"]))
    B.dflash_kv_evict(heads, 0, src, dst, case["reqs"], s["ctx"], s["keep"], case["sink"],
                      case["recent"], s["mass"], s["kept"], s["new_len"], s["mass_out"], ws)
    return {"pool": s["to_pool"], "kept": s["kept"], "new_len": s["new_len"], "mass": s["mass_out"]}


def _score_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    rows, vocab = s["z"].shape
    top = s["case"]["top"]
    ws = _workspace(s, lambda: B.dflash_score_tokens_bytes(rows, vocab, top))
    B.dflash_score_tokens(s["z"], rows, vocab, s["T"], s["ids"], s["logprob"], s["rank"], s["entropy"],
                          top, s["top_id"], s["top_lp"], ws)
    res = {"logprob": s["logprob"], "rank": s["rank"], "entropy": s["entropy"]}
    if top:
        res.update(top_id=s["top_id"], top_lp=s["top_lp"])
    return res


def run(state):
    op = state["case"]["op"]
    if own:
        return {"chunk": _chunk_own, "mass": _mass_own, "evict": _evict_own, "score": _score_own}[op](state)
    return {"chunk": _chunk_plain, "mass": _mass_plain, "evict": _evict_plain,
            "score": _score_plain}[op](state)


# ------------------------------------------------------------ exact, in 64 bits
def _keys_exact(s, r, plane):
    c = s["lens"][r]
    pages = s["table"][r, :(c + PAGE - 1) // PAGE].long()
    return s["pool"][0, pages, plane].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :c]


def _scores_exact(s, r, row0, row1, h):
    """Scores [rows][G][keys] of rows [row0, row1) of request r at KV head h."""
    case = s["case"]
    G, d, c, a = case["hq"] // case["hkv"], case["d"], s["lens"][r], s["rows"][r]
    first = int(s["start"][r])
    q = s["q"][first + row0:first + row1, h * G:(h + 1) * G].double()
    x = torch.einsum("tgd,kd->tgk", q, _keys_exact(s, r, 0)[h]) / math.sqrt(d)
    if case["causal"]:
        last = c - a + torch.arange(row0, row1, device="cuda")
        x[(torch.arange(c, device="cuda")[None] > last[:, None])[:, None].expand_as(x)] = float("-inf")
    return x


def _chunk_exact(s):
    case = s["case"]
    G = case["hq"] // case["hkv"]
    out = torch.zeros(s["T"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], case["hq"], dtype=torch.float64, device="cuda")
    for r, a in enumerate(s["rows"]):
        first, v = int(s["start"][r]), _keys_exact(s, r, 1)
        for h in range(case["hkv"]):
            for row0 in range(0, a, 1024):
                row1 = min(a, row0 + 1024)
                x = _scores_exact(s, r, row0, row1, h)
                total = torch.logsumexp(x, -1)
                p = torch.exp_(x - total[..., None])
                out[first + row0:first + row1, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", p, v[h])
                lse[first + row0:first + row1, h * G:(h + 1) * G] = total
    return {"out": out, "lse": lse}


def _mass_exact(s):
    case = s["case"]
    G = case["hq"] // case["hkv"]
    mass = s["mass0"].double()
    for r, a in enumerate(s["rows"]):
        first, c = int(s["start"][r]), s["lens"][r]
        w = a if case["last"] == 0 else min(a, case["last"])
        for h in range(case["hkv"]):
            x = _scores_exact(s, r, a - w, a, h)
            lse = s["lse"][first + a - w:first + a, h * G:(h + 1) * G].double()
            got = torch.exp(x - lse[..., None]).sum((0, 1))
            mass[r, h, :c] = got + (mass[r, h, :c] if case["add"] else 0.0)
    return {"mass": mass}


def _evict_exact(s):
    case = s["case"]
    hkv, d = case["hkv"], case["d"]
    mass = s["mass"].double().cpu().numpy()
    table, to_table = s["table"].cpu().numpy(), s["to_table"].cpu().numpy()
    src = s["pool"][0].double()
    pool = torch.zeros(s["to_pool"].shape, dtype=torch.float64, device="cuda")
    kept = np.zeros(s["kept"].shape, np.int32)
    mass_out = np.zeros(mass.shape)
    new_len = np.zeros(case["reqs"], np.int32)
    for r, c in enumerate(s["lens"]):
        new = new_len[r] = min(c, s["keeps"][r])
        at = np.arange(new)
        safe = (np.arange(c) < case["sink"]) | (np.arange(c) >= c - case["recent"])
        for h in range(hkv):
            order = np.lexsort((np.arange(c), np.where(safe, -np.inf, -mass[r, h, :c])))
            k = np.sort(order[:new])
            kept[r, h, :new], mass_out[r, h, :new] = k, mass[r, h, k]
            page = torch.from_numpy(table[r, k // PAGE].astype(np.int64)).cuda()
            slot = torch.from_numpy(k % PAGE).cuda()
            to = torch.from_numpy(to_table[r, at // PAGE].astype(np.int64)).cuda()
            pool[0, to, :, h, torch.from_numpy(at % PAGE).cuda()] = src[page, :, h, slot]
    return {"pool": pool, "kept": torch.from_numpy(kept), "new_len": torch.from_numpy(new_len),
            "mass": torch.from_numpy(mass_out)}


def _score_exact(s):
    case = s["case"]
    rows, vocab = s["z"].shape
    ids, top = s["ids"].cpu().numpy(), case["top"]
    res = {"logprob": np.zeros(rows), "rank": np.full(rows, -1, np.int32), "entropy": np.zeros(rows)}
    if top:
        res["top_id"] = np.full((rows, top), -1, np.int32)
        res["top_lp"] = np.full((rows, top), -np.inf)
    for i in range(rows):
        z = s["z"][i].double()
        T = 1.0 if s["T"] is None else float(s["T"][i].double())
        lp = z / T - torch.logsumexp(z / T, 0)
        res["entropy"][i] = -float(torch.nansum(torch.exp(lp) * lp))   # 0 * -inf counts as none
        if ids[i] >= 0:
            j = int(ids[i])
            res["logprob"][i] = float(lp[j])
            res["rank"][i] = int(torch.count_nonzero(z > z[j]) + torch.count_nonzero(z[:j] == z[j]))
        if top:
            zi = z.cpu().numpy()
            border = np.partition(zi, -min(vocab, top))[-min(vocab, top)]
            best = np.flatnonzero(zi >= max(border, np.finfo(np.float64).min))
            best = best[np.argsort(-zi[best], kind="stable")][:top]
            res["top_id"][i, :len(best)] = best
            res["top_lp"][i, :len(best)] = lp.cpu().numpy()[best]
    return {k: torch.from_numpy(v) for k, v in res.items()}


def exact(case, seed):
    state = prepare(case, seed)
    return {"chunk": _chunk_exact, "mass": _mass_exact, "evict": _evict_exact,
            "score": _score_exact}[case["op"]](state)
