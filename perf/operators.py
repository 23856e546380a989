"""Cases for the serving operators around the paged K/V cache.

Three operators of a decode step over a batch of requests:

* append: rotate q and k by their positions and store k, v in the paged cache
  (dflash_kv_rope_append);
* attend: attention of a batch whose requests share a long prefix, the prefix
  read once for all (dflash_attention_prefix);
* sample: a token per row under temperature, top-k, top-p and min-p, from
  given uniforms (dflash_sample_filtered).

``run`` computes them with elementary torch operations, or through the
framework's entry points where ``own`` is true.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
LN2 = math.log(2.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one request, the drafter's heads: a call's latency
        dict(name="append_token", op="append", T=1, reqs=1, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, scaling="none", norm=True, fp32=False, terms=1, pad=0, far=4096),
        # block verify of 32 requests x 16 rows, interleaved pairs over half of
        # the head, frequencies stretched for a long context
        dict(name="append_verify_b32", op="append", T=512, reqs=32, hq=32, hkv=8, d=128, rot=64,
             interleaved=True, scaling="yarn", norm=False, fp32=False, terms=1, pad=0, far=100000),
        # prefill of 8 prompts of 1024 tokens
        dict(name="append_prefill_8x1024", op="append", T=8192, reqs=8, hq=32, hkv=8, d=128,
             rot=128, interleaved=False, scaling="linear", norm=True, fp32=False, terms=1, pad=0,
             far=2048),
        # ragged rows with padding into a two-term target cache, from fp32
        dict(name="append_ragged_two_term", op="append", T=333, reqs=5, hq=4, hkv=4, d=64, rot=32,
             interleaved=False, scaling="none", norm=True, fp32=True, terms=2, pad=21, far=1000000),
        # two short requests, small heads: a call's latency
        dict(name="attend_small", op="attend", groups=1, group=2, n=1, hq=4, hkv=4, d=64,
             prefix=192, suffix=40, causal=True),
        # one token for each of 32 samples of one 16384-token prompt
        dict(name="attend_decode_b32", op="attend", groups=1, group=32, n=1, hq=32, hkv=8, d=128,
             prefix=16384, suffix=1024, causal=True),
        # 8 prompts of odd length with 8 samples each, small heads
        dict(name="attend_decode_8x8", op="attend", groups=8, group=8, n=1, hq=16, hkv=4, d=64,
             prefix=2077, suffix=600, causal=True),
        # block verify (16 rows) of 32 samples of one 16384-token prompt
        dict(name="attend_verify_b32", op="attend", groups=1, group=32, n=16, hq=32, hkv=8, d=128,
             prefix=16384, suffix=512, causal=True),
        # one row at the drafter's vocabulary, the usual chat settings
        dict(name="sample_one", op="sample", rows=1, vocab=151936, k="50", p="0.95", m="off",
             spread=2.2),
        # a batch whose requests each bring their own settings
        dict(name="sample_mixed_b32", op="sample", rows=32, vocab=151936, k="mixed", p="mixed",
             m="mixed", spread=2.2),
        # every row of a 32 x 16 block, nucleus only, flat logits
        dict(name="sample_block_b32", op="sample", rows=512, vocab=151936, k="off", p="0.95",
             m="off", spread=1.3),
        # small odd vocabulary, min-p only
        dict(name="sample_small_odd", op="sample", rows=7, vocab=1009, k="off", p="off", m="0.05",
             spread=3.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "sample"])
    if op == "append":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, 8192)
        reqs = min(T, _log(rng, 1, 64))
        return dict(op=op, T=T, reqs=reqs, hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, 16, 48]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    norm=rng.random() < 0.5, fp32=rng.random() < 0.3, terms=rng.choice([1, 1, 2]),
                    pad=rng.randrange(T) // 4, far=_log(rng, 1, 1000000))
    if op == "attend":
        hkv = rng.choice([1, 2, 4, 8])
        groups, group = rng.choice([1, 1, 1, 2, 3, 8]), _log(rng, 1, 32)
        G = rng.choice([1, 2, 4, 8]) if hkv < 8 else rng.choice([1, 2, 4])
        n = rng.choice([1, 1, 1, 2, 5, 8, 16])
        if groups * group * n > 512:
            n = 1
        return dict(op=op, groups=groups, group=group, n=n, hq=hkv * G, hkv=hkv,
                    d=rng.choice([64, 128]), prefix=_log(rng, 1, 16384 // groups),
                    suffix=_log(rng, n, 1024), causal=rng.random() < 0.7)
    vocab = _log(rng, 2, 151936)
    return dict(op=op, rows=_log(rng, 1, 512), vocab=vocab,
                k=rng.choice(["off", "1", "50", "mixed"]),
                p=rng.choice(["off", "0.3", "0.95", "0.999", "mixed"]),
                m=rng.choice(["off", "0.05", "mixed"]), spread=rng.uniform(0.5, 4.0))


def work(case):
    if case["op"] == "append":
        T, e = case["T"] - case["pad"], 4 if case["fp32"] else 2
        q, kv, d = case["hq"], case["hkv"], case["d"]
        return {"bytes": T * d * (q * (e + 2) + 2 * kv * (e + 2 * case["terms"])) + 8 * T,
                "flops": 6 * T * d * (q + kv)}
    if case["op"] == "attend":
        b = case["groups"] * case["group"]
        rows = b * case["n"] * case["hq"]
        suffix = (case["suffix"] + case["n"]) // 2   # suffix lengths spread over [n, suffix]
        keys = case["groups"] * case["prefix"] + b * suffix
        return {"bytes": rows * (4 * case["d"] + 4) + 4 * case["d"] * case["hkv"] * keys,
                "flops": 4 * case["d"] * rows * (case["prefix"] + suffix)}
    return {"bytes": case["rows"] * (4 * case["vocab"] + 36),
            "flops": 8 * case["rows"] * case["vocab"]}


# --------------------------------------------------------------------- inputs
def _generators(seed):
    gpu = torch.Generator(device="cuda")
    gpu.manual_seed(seed)
    return gpu, np.random.default_rng(seed)


def _paged_rows(lengths, rnd, spare=3):
    """A page table over a shuffled pool for requests of these lengths."""
    need = [(n + PAGE - 1) // PAGE for n in lengths]
    pages = rnd.permutation(sum(need) + spare).astype(np.int32)
    table = np.zeros((len(lengths), max(1, max(need))), np.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = pages[at:at + k]
        at += k
    return table, sum(need) + spare


def _inv_freq(rot, scaling):
    """Frequencies (64 bits) and the magnitude of the rotation."""
    p = np.arange(rot // 2, dtype=np.float64)
    base, factor, orig = 1e6, 4.0, 32768
    f = base ** (-2.0 * p / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        return (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * p / rot), 1.0
    if scaling == "yarn":
        def dim(beta):
            return rot * math.log(orig / (beta * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        keep = 1.0 - np.clip((p - low) / max(high - low, 1e-3), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _append_state(case, seed):
    gpu, rnd = _generators(seed)
    T, reqs, hq, hkv, d = (case[k] for k in ("T", "reqs", "hq", "hkv", "d"))
    dt = torch.float32 if case["fp32"] else torch.bfloat16
    # q, k and v as a fused projection leaves them: columns of one array
    qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=gpu, device="cuda").to(dt)
    counts = np.full(reqs, T // reqs)
    counts[:T % reqs] += 1
    start = 37 * np.arange(reqs) % 200   # rows already cached
    req = np.repeat(np.arange(reqs), counts)
    local = np.concatenate([s + np.arange(c) for s, c in zip(start, counts)])
    slot = local.astype(np.int32)
    table, n_pages = _paged_rows(list(start + counts), rnd)
    pos = slot.copy()
    pos[rnd.choice(T, case["pad"], replace=False)] = -1
    # far positions: the request's cache is entered far along by repeating its
    # last page row (a table as wide as the positions need)
    shift = min(case["far"], 1 << 20) // PAGE
    wide = np.zeros((reqs, table.shape[1] + shift), np.int32)
    wide[:, shift:] = table
    pos = np.where(pos < 0, -1, pos + shift * PAGE).astype(np.int32)
    freq, mscale = _inv_freq(case["rot"], case["scaling"])
    pool = torch.randn(1, n_pages, 2 * case["terms"], hkv, PAGE, d, generator=gpu,
                       device="cuda").to(torch.bfloat16)
    gains = 1 + 0.25 * torch.randn(2, d, generator=gpu, device="cuda")
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dict(case=case, q=qkv[:, :hq * d].unflatten(1, (hq, d)),
                k=qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                v=qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)),
                gains=gains.to(torch.bfloat16), req=to(req.astype(np.int32)), pos=to(pos),
                table=to(wide), n_pages=n_pages, pool=pool, freq=freq, mscale=mscale,
                freq_dev=to(freq), q_out=torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda"))


def _attend_state(case, seed):
    gpu, rnd = _generators(seed)
    ng, g, n, hq, hkv, d = (case[k] for k in ("groups", "group", "n", "hq", "hkv", "d"))
    b = ng * g
    prefix = np.array([max(1, case["prefix"] - 5 * i) for i in range(ng)])
    suffix = rnd.integers(n, max(n, case["suffix"]) + 1, b)
    ctx = np.repeat(prefix, g) + suffix
    # whole pages of the prefix are shared; the page it ends in is each request's own
    shared = prefix // PAGE
    need = [(int(c) + PAGE - 1) // PAGE for c in ctx]
    total = int(shared.sum()) + sum(k - int(shared[r // g]) for r, k in enumerate(need))
    pages = rnd.permutation(total + 2).astype(np.int32)
    table = np.zeros((b, max(need)), np.int32)
    at = 0
    for i in range(ng):
        table[i * g:(i + 1) * g, :shared[i]] = pages[at:at + shared[i]]
        at += int(shared[i])
    for r, k in enumerate(need):
        s = int(shared[r // g])
        table[r, s:k] = pages[at:at + k - s]
        at += k - s
    pool = torch.randn(1, total + 2, 2, hkv, PAGE, d, generator=gpu, device="cuda").to(torch.bfloat16)
    # the page a prefix ends in holds the same prefix tokens for every request
    for i in range(ng):
        r = int(prefix[i]) % PAGE
        if r:
            own_pages = torch.from_numpy(table[i * g:(i + 1) * g, shared[i]].astype(np.int64)).cuda()
            pool[0, own_pages, :, :, :r] = pool[0, own_pages[:1], :, :, :r]
    q = (1.5 * torch.randn(b, n, hq, d, generator=gpu, device="cuda")).to(torch.bfloat16)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).cuda()  # noqa: E731
    return dict(case=case, q=q, pool=pool, table=to(table), n_pages=total + 2, ctx_len=to(ctx),
                prefix_len=to(prefix), prefix_max=int(prefix.max()),
                suffix_max=int(max(suffix.max(), 1)), out=torch.empty_like(q),
                lse=torch.empty(b, n, hq, dtype=torch.float32, device="cuda"))


def _setting(text, rows, mixed, off, rnd):
    if text == "off":
        return None if off is None else np.full(rows, off)
    if text == "mixed":
        return np.array([mixed[i] for i in rnd.integers(0, len(mixed), rows)])
    return np.full(rows, float(text))


def _sample_state(case, seed):
    gpu, rnd = _generators(seed)
    rows, vocab = case["rows"], case["vocab"]
    z = case["spread"] * torch.randn(rows, vocab, generator=gpu, device="cuda")
    # a few likely tokens above the bulk, as a trained model's rows have
    likely = torch.from_numpy(rnd.integers(0, vocab, (rows, 24))).cuda()
    z.scatter_add_(1, likely, torch.from_numpy(rnd.exponential(3.0, (rows, 24)).astype(np.float32)).cuda())
    # a grammar's masked tokens
    z[:, vocab // 3:vocab // 3 + vocab // 50] = float("-inf")
    T = _setting("mixed" if "mixed" in (case["k"], case["p"], case["m"]) else "0.8", rows,
                 [0.0, 0.6, 0.8, 1.0, 1.5], None, rnd)
    k = _setting(case["k"], rows, [0, 1, 20, 50, 1000], None, rnd)
    p = _setting(case["p"], rows, [1.0, 0.5, 0.9, 0.95, 0.99], None, rnd)
    m = _setting(case["m"], rows, [0.0, 0.02, 0.1], None, rnd)
    to = lambda a, t: None if a is None else torch.from_numpy(a.astype(t)).cuda()  # noqa: E731
    return dict(case=case, z=z, T=to(T, np.float32), k=to(k, np.int32), p=to(p, np.float32),
                m=to(m, np.float32), a=to(rnd.random(rows), np.float64),
                token=torch.empty(rows, dtype=torch.int32, device="cuda"),
                kept=torch.empty(rows, dtype=torch.int32, device="cuda"),
                logprob=torch.empty(rows, dtype=torch.float32, device="cuda"))


def prepare(case, seed):
    return {"append": _append_state, "attend": _attend_state,
            "sample": _sample_state}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _rms(x, gain):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain.float()


def _rotate(x, cos, sin, rot, interleaved):
    lead = x[..., :rot]
    if interleaved:
        a, b = lead[..., 0::2], lead[..., 1::2]
        lead = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = lead[..., :rot // 2], lead[..., rot // 2:]
        lead = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((lead, x[..., rot:]), -1)


def _append_plain(s):
    case = s["case"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["norm"]:
        q, k = _rms(q, s["gains"][0]), _rms(k, s["gains"][1])
    angle = s["pos"].double()[:, None] * s["freq_dev"]
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]
    q = _rotate(q, cos, sin, case["rot"], case["interleaved"])
    k = _rotate(k, cos, sin, case["rot"], case["interleaved"])
    pos, req = s["pos"].long(), s["req"].long()
    if case["pad"]:
        live = pos >= 0
        s["q_out"][live] = q[live].to(torch.bfloat16)
        pos, req, k, v = pos[live], req[live], k[live], v[live]
    else:
        s["q_out"].copy_(q)
    page, slot = s["table"][req, pos // PAGE].long(), pos % PAGE
    kh, vh = k.to(torch.bfloat16), v.to(torch.bfloat16)
    planes = [kh, vh]
    if case["terms"] == 2:
        planes += [(k - kh.float()).to(torch.bfloat16), (v - vh.float()).to(torch.bfloat16)]
    s["pool"][0, page, :, :, slot] = torch.stack(planes, 1)
    return {"q": s["q_out"], "pool": s["pool"]}


def _attend_plain(s):
    case = s["case"]
    ng, g, n, hq, hkv, d = (case[k] for k in ("groups", "group", "n", "hq", "hkv", "d"))
    b, G = ng * g, hq // hkv
    scale = 1.0 / math.sqrt(d)
    row = torch.arange(n, device="cuda")
    limit = s["ctx_len"].long()[:, None] + (row - n + 1 if case["causal"] else 0 * row)   # [b, n]
    q = s["q"].float().view(b, n, hkv, G, d) * scale
    # the prefix, once for each group
    P = s["prefix_max"]
    at = torch.arange(P, device="cuda")
    page = s["table"][::g][:, at // PAGE].long()                                       # [ng, P]
    kp = s["pool"][0, page, 0, :, at % PAGE].float().permute(0, 2, 1, 3)               # [ng, hkv, P, d]
    vp = s["pool"][0, page, 1, :, at % PAGE].float().permute(0, 2, 1, 3)
    qp = q.view(ng, g * n, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(ng, hkv, g * n * G, d)
    sp = (qp @ kp.transpose(2, 3)).view(ng, hkv, g, n, G, P)
    seen = torch.minimum(limit.view(ng, g, n), s["prefix_len"].long()[:, None, None])
    sp = torch.where(at < seen[:, None, :, :, None, None], sp, float("-inf"))
    # what follows it, request by request
    S = s["suffix_max"]
    step = torch.arange(S, device="cuda")
    pos = s["prefix_len"].long().repeat_interleave(g)[:, None] + step                  # [b, S]
    last = s["table"].shape[1] - 1
    page = s["table"].gather(1, (pos // PAGE).clamp(max=last)).long()
    ks = s["pool"][0, page, 0, :, pos % PAGE].float().permute(0, 2, 1, 3)              # [b, hkv, S, d]
    vs = s["pool"][0, page, 1, :, pos % PAGE].float().permute(0, 2, 1, 3)
    qs = q.permute(0, 2, 1, 3, 4).reshape(b, hkv, n * G, d)
    ss = (qs @ ks.transpose(2, 3)).view(b, hkv, n, G, S)
    ss = torch.where(pos[:, None, None, None, :] < limit[:, None, :, None, None], ss, float("-inf"))
    # one softmax over both
    mp = sp.amax(-1).permute(0, 2, 1, 3, 4).reshape(b, hkv, n, G)
    m = torch.maximum(mp, ss.amax(-1))
    m = torch.where(m == float("-inf"), 0.0, m)
    ep = torch.exp(sp - m.view(ng, g, hkv, n, G).permute(0, 2, 1, 3, 4)[..., None])
    es = torch.exp(ss - m[..., None])
    total = ep.sum(-1).permute(0, 2, 1, 3, 4).reshape(b, hkv, n, G) + es.sum(-1)
    op = (ep.view(ng, hkv, g * n * G, P) @ vp).view(ng, hkv, g, n, G, d)
    o = op.permute(0, 2, 1, 3, 4, 5).reshape(b, hkv, n, G, d)
    o = o + (es.view(b, hkv, n * G, S) @ vs).view(b, hkv, n, G, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(b, n, hq, d))
    s["lse"].copy_((m + torch.log(total)).permute(0, 2, 1, 3).reshape(b, n, hq))
    return {"out": s["out"], "lse": s["lse"]}


def _sample_plain(s):
    z = s["z"]
    rows, vocab = z.shape
    T = s["T"].double()[:, None]
    order, index = torch.sort(z, dim=1, descending=True, stable=True)
    top = order[:, :1].double()
    # temperature 0 is the largest logit alone
    t = (order.double() - top) / torch.where(T > 0, T, 1.0)
    t = torch.where((T == 0) & (torch.arange(vocab, device="cuda") > 0), float("-inf"), t)
    w = torch.exp(t)
    rank = torch.arange(vocab, device="cuda")[None]
    keep = t > float("-inf")
    if s["k"] is not None:
        k = s["k"].long()[:, None]
        keep = keep & ((rank < k) | (k <= 0))
    w = torch.where(keep, w, 0.0)
    if s["p"] is not None:
        p = s["p"].double()[:, None]
        run = torch.cumsum(w, 1)
        keep = keep & ((run - w < p * run[:, -1:]) | (p >= 1) | (rank == 0))
    if s["m"] is not None:
        m = s["m"].double()[:, None]
        keep = keep & ((t >= torch.log(m)) | (m <= 0) | (rank == 0))
    w = torch.where(keep, w, 0.0)
    by_index = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda").scatter_(1, index, w)
    run = torch.cumsum(by_index, 1)
    S = run[:, -1:]
    token = (run <= s["a"][:, None] * S).sum(1).clamp(max=vocab - 1)
    s["token"].copy_(token)
    s["kept"].copy_(keep.sum(1))
    s["logprob"].copy_(torch.log(by_index.gather(1, token[:, None]) / S)[:, 0])
    return {"token": s["token"], "kept": s["kept"], "logprob": s["logprob"]}


# --------------------------------------------------------- the framework's own
def _workspace(s, size):
    """The caller's workspace, allocated once and kept with its other buffers."""
    if "ws" not in s:
        from block_diffusion_speculative_fuse_gb300 import binding as B
        s["ws"] = torch.empty(size(), dtype=torch.uint8, device="cuda")
        B.dflash_workspace_init(s["ws"])
    return s["ws"]


def _cache(s):
    """The library's descriptors of the cache, built once per cache."""
    if "kv" not in s:
        from block_diffusion_speculative_fuse_gb300 import binding as B
        case = s["case"]
        s["heads"] = B.DflashHeads(n_layers=1, n_q_heads=case["hq"], n_kv_heads=case["hkv"],
                                   head_dim=case["d"], page_size=PAGE, kv_terms=case.get("terms", 1))
        s["kv"] = B.DflashKV(pool=s["pool"].data_ptr(), page_table=s["table"].data_ptr(),
                             n_pages=s["n_pages"], max_pages=s["table"].shape[1],
                             n_rows=s["table"].shape[0], dtype=0, scales=None)
    return s["heads"], s["kv"]


def _append_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    case = s["case"]
    heads, kv = _cache(s)
    if "rope" not in s:
        s["rope"] = B.dflash_rope_init(case["rot"], case["interleaved"], base=1e6,
                                       scaling=case["scaling"], factor=4.0, orig_ctx=32768)
    ws = _workspace(s, lambda: 1 << 16)
    gq, gk = (s["gains"][0], s["gains"][1]) if case["norm"] else (None, None)
    B.dflash_kv_rope_append(heads, s["rope"], 0, s["q"], s["k"], s["v"], s["req"], s["pos"],
                            case["T"], s["q_out"], kv, ws, q_norm=gq, k_norm=gk, eps=1e-6)
    return {"q": s["q_out"], "pool": s["pool"]}


def _attend_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    case = s["case"]
    heads, kv = _cache(s)
    b = case["groups"] * case["group"]
    ws = _workspace(s, lambda: B.dflash_attention_prefix_bytes(heads, b, case["n"], case["group"]))
    B.dflash_attention_prefix(heads, 0, s["q"], b, case["n"], case["group"], case["causal"], 0.0,
                              kv, s["ctx_len"], s["prefix_len"], s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _sample_own(s):
    from block_diffusion_speculative_fuse_gb300 import binding as B
    rows, vocab = s["z"].shape
    ws = _workspace(s, lambda: B.dflash_sample_filtered_bytes(rows, vocab))
    B.dflash_sample_filtered(s["z"], rows, vocab, s["T"], s["k"], s["p"], s["m"], s["a"],
                             s["token"], s["kept"], s["logprob"], ws)
    return {"token": s["token"], "kept": s["kept"], "logprob": s["logprob"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "attend": _attend_own, "sample": _sample_own}[op](state)
    return {"append": _append_plain, "attend": _attend_plain, "sample": _sample_plain}[op](state)


# ------------------------------------------------------------ exact, in 64 bits
def _append_exact(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    pair = np.arange(half)
    first, second = (2 * pair, 2 * pair + 1) if case["interleaved"] else (pair, pair + half)
    pos = s["pos"].cpu().numpy().astype(np.int64)
    turn = np.exp(1j * pos[:, None].astype(np.float64) * s["freq"][None]) * s["mscale"]

    def one(x, gain):
        x = x.double().cpu().numpy()
        if case["norm"] and gain is not None:
            x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6) * gain.double().cpu().numpy()
        if gain is not None:
            z = (x[..., first] + 1j * x[..., second]) * turn[:, None]
            x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = one(s["q"], s["gains"][0]), one(s["k"], s["gains"][1]), one(s["v"], None)
    q[pos < 0] = 0.0
    pool = s["pool"].double().cpu().numpy()
    table, req = s["table"].cpu().numpy(), s["req"].cpu().numpy()
    low = lambda x: x - torch.from_numpy(x).to(torch.bfloat16).double().numpy()  # noqa: E731
    for t in np.flatnonzero(pos >= 0):
        page, slot = table[req[t], pos[t] // PAGE], pos[t] % PAGE
        pool[0, page, 0, :, slot], pool[0, page, 1, :, slot] = k[t], v[t]
        if case["terms"] == 2:
            pool[0, page, 2, :, slot], pool[0, page, 3, :, slot] = low(k[t]), low(v[t])
            pool[0, page, :2, :, slot] -= pool[0, page, 2:, :, slot]
    return {"q": torch.from_numpy(q), "pool": torch.from_numpy(pool)}


def _attend_exact(s):
    case = s["case"]
    n, hq, hkv, d = (case[k] for k in ("n", "hq", "hkv", "d"))
    G = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device="cuda")
    for r, c in enumerate(s["ctx_len"].tolist()):
        pages = s["table"][r, :(c + PAGE - 1) // PAGE].long()
        kv = s["pool"][0, pages].double().permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :c]
        q = s["q"][r].double().reshape(n, hkv, G, d).permute(1, 0, 2, 3).reshape(hkv, n * G, d)
        logits = torch.einsum("hrd,hkd->hrk", q, kv[0]) / math.sqrt(d)
        if case["causal"]:
            late = torch.arange(c, device="cuda") > c - n + torch.arange(n, device="cuda")[:, None]
            logits.view(hkv, n, G, c).masked_fill_(late[None, :, None], float("-inf"))
        total = torch.logsumexp(logits, -1)
        o = torch.einsum("hrk,hkd->hrd", torch.exp(logits - total[..., None]), kv[1])
        out[r] = o.view(hkv, n, G, d).permute(1, 0, 2, 3).reshape(n, hq, d)
        lse[r] = total.view(hkv, n, G).permute(1, 0, 2).reshape(n, hq)
    return {"out": out, "lse": lse}


def _sample_exact(s):
    z = s["z"].double().cpu().numpy()
    rows, vocab = z.shape
    get = lambda key, i, off: off if s[key] is None else float(s[key][i])  # noqa: E731
    T = s["T"].double().cpu().numpy()
    a = s["a"].cpu().numpy()
    token, kept, logprob = np.zeros(rows, np.int32), np.zeros(rows, np.int32), np.zeros(rows)
    for i in range(rows):
        best = int(np.argmax(z[i]))
        if T[i] == 0:
            token[i], kept[i] = best, 1
            continue
        t = (z[i] - z[i, best]) / T[i]
        order = np.argsort(-z[i], kind="stable")
        order = order[:np.count_nonzero(t > -np.inf)]
        k = int(get("k", i, 0))
        order = order[:k] if k > 0 else order
        w = np.exp(t[order])
        count = len(order)
        p, m = get("p", i, 1.0), get("m", i, 0.0)
        if p < 1:
            count = min(count, int(np.searchsorted(np.cumsum(w), p * w.sum())) + 1)
        if m > 0:
            count = min(count, int(np.count_nonzero(t[order] >= math.log(m))))
        chosen = np.sort(order[:max(1, count)])
        c = np.cumsum(np.exp(t[chosen]))
        j = min(int(np.searchsorted(c, a[i] * c[-1], side="right")), len(chosen) - 1)
        token[i], kept[i] = chosen[j], len(chosen)
        logprob[i] = t[chosen[j]] - math.log(c[-1])
    return {"token": torch.from_numpy(token), "kept": torch.from_numpy(kept),
            "logprob": torch.from_numpy(logprob)}


def exact(case, seed):
    if case["op"] == "sample" and case["rows"] * case["vocab"] > 5e7:
        return None   # sorting this many logits on the host takes too long
    state = prepare(case, seed)
    return {"append": _append_exact, "attend": _attend_exact, "sample": _sample_exact}[case["op"]](state)
