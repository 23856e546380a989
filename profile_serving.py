"""Launch cases of the serving operators for profiling kernels with ncu.

    python profile_serving.py append | decode | verify | sample

append: 8192 rows of 32 + 8 + 8 heads of 128, with norms (0.2 GB).  decode,
verify: 32 requests of 1 or 16 rows over 16384 shared positions and 1024 or
512 of their own, 32 query and 8 KV heads of 128 (0.3 GB at most).  sample:
512 rows of 151936 logits under top-p (0.3 GB).  Each call is made twice.
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


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["append", "decode", "verify", "sample"])
    case = ap.parse_args().case
    _build.build()
    B.load()
    ws = {"append": append, "decode": lambda: attend(1, 1024), "verify": lambda: attend(16, 512),
          "sample": sample}[case]()
    status = B.dflash_get_status(ws)
    assert status == (0, 0), status
    print(case, "ok")


if __name__ == "__main__":
    main()
