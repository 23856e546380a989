"""Launch cases of the serving operators for profiling kernels with ncu.

    python profile_serving.py append | decode | verify | sample | chunk | mass | evict | score

append: 8192 rows of 32 + 8 + 8 heads of 128, with norms (0.2 GB).  decode,
verify: 32 requests of 1 or 16 rows over 16384 shared positions and 1024 or
512 of their own, 32 query and 8 KV heads of 128 (0.3 GB at most).  sample:
512 rows of 151936 logits under top-p (0.3 GB).  chunk: 2048 rows of a prompt
behind 6144 positions.  mass: the weights of the last 32 rows of 8 requests of
16384 positions (0.6 GB).  evict: 8 requests cut from 8192 to 2048 positions (0.4
GB).  score: 608 rows of 151936 logits (0.4 GB).  Each call is made twice.
"""
import argparse
import types

import numpy as np
import torch

from block_diffusion_speculative_fuse_gb300 import _build, binding as B
from block_diffusion_speculative_fuse_gb300.device import PagedKV, i32

HQ, HKV, D = 32, 8, 128


def cache(table, n_pages):
    shape = types.SimpleNamespace(n_layers=1, n_kv_heads=HKV, head_dim=D, kv_terms=1)
    kv = PagedKV(shape, table, n_pages)
    kv.pool.normal_()
    return kv


def append(rows=8192, requests=8):
    per = rows // requests // 16
    kv = cache(np.arange(requests * per).reshape(requests, per), requests * per)
    x = torch.randn(rows, (HQ + 2 * HKV) * D, device="cuda").to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([HQ * D, HKV * D, HKV * D], 1))
    gain = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    req, pos = np.divmod(np.arange(rows), rows // requests)
    ws = kv.attention_workspace(HQ, 1, 1, 1)
    out, req, pos, rope = torch.empty_like(q), i32(req), i32(pos), B.dflash_rope_init(D)
    for _ in range(2):
        kv.append_rotated(rope, 0, q, k, v, req, pos, ws, q_out=out, q_norm=gain, k_norm=gain)
    return ws


def attend(n, own, batch=32, shared=16384):
    s, o = shared // 16, own // 16
    table = np.concatenate((np.tile(np.arange(s), (batch, 1)), s + np.arange(batch * o).reshape(batch, o)), 1)
    kv = cache(table, s + batch * o)
    q = torch.randn(batch, n, HQ, D, device="cuda").to(torch.bfloat16)
    ws = kv.attention_workspace(HQ, batch, n, batch)
    out, ctx, pre = torch.empty_like(q), i32([shared + own] * batch), i32([shared])
    for _ in range(2):
        kv.attend_prefix(0, q, ctx, pre, batch, out, ws)
    return ws


def sample(rows=512, vocab=151936):
    z = 1.3 * torch.randn(rows, vocab, device="cuda")
    T, p = (torch.full((rows,), x, device="cuda") for x in (0.8, 0.95))
    a = torch.rand(rows, dtype=torch.float64, device="cuda")
    token = torch.empty(rows, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.dflash_sample_filtered_bytes(rows, vocab), dtype=torch.uint8, device="cuda")
    B.dflash_workspace_init(ws)
    for _ in range(2):
        B.dflash_sample_filtered(z, rows, vocab, T, None, p, None, a, token, None, None, ws)
    return ws


def rows_of(requests, rows, positions):
    per = positions // 16
    kv = cache(np.arange(requests * per).reshape(requests, per), requests * per)
    q = torch.randn(requests * rows, HQ, D, device="cuda").to(torch.bfloat16)
    start, ctx = i32(rows * np.arange(requests + 1)), i32([positions] * requests)
    ws = kv.chunk_workspace(HQ, requests, requests * rows)
    out, lse = torch.empty_like(q), torch.empty(requests * rows, HQ, device="cuda")
    return kv, q, start, ctx, ws, out, lse


def chunk():
    kv, q, start, ctx, ws, out, lse = rows_of(1, 2048, 8192)
    for _ in range(2):
        kv.attend_chunk(0, q, start, ctx, out, ws, lse=lse)
    return ws


def mass():
    kv, q, start, ctx, ws, out, lse = rows_of(8, 32, 16384)
    kv.attend_chunk(0, q, start, ctx, out, ws, lse=lse)
    sums = torch.zeros(8, HKV, 16384, device="cuda")
    for _ in range(2):
        kv.attention_mass(0, q, start, ctx, lse, sums, ws)
    return ws


def evict(requests=8, positions=8192, keep=2048):
    src, dst = (cache(np.arange(requests * n // 16).reshape(requests, -1), requests * n // 16) for n in (positions, keep))
    sums = torch.rand(requests, HKV, positions, device="cuda")
    kept = torch.empty(requests, HKV, keep, dtype=torch.int32, device="cuda")
    ws = dst.evict_workspace(requests)
    ctx, keep = i32([positions] * requests), i32([keep] * requests)
    for _ in range(2):
        src.evict_to(dst, 0, ctx, keep, sums, kept, ws, sink=4, recent=64)
    return ws


def score(rows=608, vocab=151936, n=5):
    z = 2.2 * torch.randn(rows, vocab, device="cuda")
    ids = torch.randint(vocab, (rows,), dtype=torch.int32, device="cuda")
    f = [torch.empty(rows, device="cuda") for _ in range(2)]
    rank = torch.empty(rows, dtype=torch.int32, device="cuda")
    top = torch.empty(rows, n, dtype=torch.int32, device="cuda"), torch.empty(rows, n, device="cuda")
    ws = torch.empty(B.dflash_score_tokens_bytes(rows, vocab, n), dtype=torch.uint8, device="cuda")
    B.dflash_workspace_init(ws)
    for _ in range(2):
        B.dflash_score_tokens(z, rows, vocab, None, ids, f[0], rank, f[1], n, *top, ws)
    return ws


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["append", "decode", "verify", "sample", "chunk", "mass", "evict",
                                     "score"])
    case = ap.parse_args().case
    _build.build()
    B.load()
    ws = {"append": append, "decode": lambda: attend(1, 1024), "verify": lambda: attend(16, 512),
          "sample": sample, "chunk": chunk, "mass": mass, "evict": evict, "score": score}[case]()
    status = B.dflash_get_status(ws)
    assert status == (0, 0), status
    print(case, "ok")


if __name__ == "__main__":
    main()
