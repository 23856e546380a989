"""Serving operators in plain NumPy, 64 bits: rotation of q and k, attention
of query rows to a request's keys, and filtered sampling.  Test
infrastructure: written from the definitions, sharing no code with the CUDA
path."""
import math

import numpy as np


def rope_freqs(rot, base, scaling="none", factor=1.0, orig=0, fast=32.0, slow=1.0):
    """Frequencies of the rot/2 pairs and the magnitude of the rotation."""
    f, mag = [], 1.0
    for p in range(rot // 2):
        plain = math.exp(-2.0 * p / rot * math.log(base))
        if scaling == "none":
            f.append(plain)
        elif scaling == "linear":
            f.append(plain / factor)
        elif scaling == "ntk":
            f.append(math.exp(-2.0 * p / rot * (math.log(base) + rot / (rot - 2.0) * math.log(factor))))
        elif scaling == "yarn":
            # the pair whose wavelength fits `beta` times into the original context
            at = [rot * math.log(orig / (2 * math.pi * beta)) / (2 * math.log(base)) for beta in (fast, slow)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            ramp = min(1.0, max(0.0, (p - lo) / max(hi - lo, 1e-3)))
            f.append(plain * (1.0 - ramp) + plain / factor * ramp)
            mag = 1.0 + 0.1 * math.log(factor)
        else:
            raise ValueError(scaling)
    return np.array(f), mag


def rotate(x, pos, freqs, mag, interleaved):
    """x [T][heads][d] rotated at positions pos [T] (as complex numbers)."""
    x = np.array(x, dtype=np.float64)
    half = len(freqs)
    if half == 0:
        return x
    i = np.arange(half)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z = (x[..., re] + 1j * x[..., im]) * (mag * np.exp(1j * np.outer(pos, freqs)))[:, None, :]
    x[..., re], x[..., im] = z.real, z.imag
    return x


def rms_norm(x, gain, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gain


def attend(q, k, v, scale, limits):
    """q [n][hq][d], k, v [keys][hkv][d]; row i sees the first limits[i] keys.
    Returns out [n][hq][d], lse [n][hq], and sum_j p_j |v_j| (for bounds)."""
    n, hq, d = q.shape
    G = hq // k.shape[1]
    out, lse, mag = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((n, hq, d))
    for i in range(n):
        m = max(0, min(int(limits[i]), k.shape[0]))
        if m == 0:
            continue
        for h in range(hq):
            s = scale * (k[:m, h // G] @ q[i, h])
            top = s.max()
            w = np.exp(s - top)
            lse[i, h] = top + math.log(w.sum())
            out[i, h] = (w / w.sum()) @ v[:m, h // G]
            mag[i, h] = (w / w.sum()) @ np.abs(v[:m, h // G])
    return out, lse, mag


def sample(z, temperature, top_k, top_p, min_p, a):
    """(token, kept, logprob, margin) of one row of logits: margin is the
    smallest relative distance of a decision to its border."""
    z = np.asarray(z, dtype=np.float64)
    if np.isnan(z).any() or not np.isfinite(z.max()):
        return -1, 0, 0.0, 1.0
    if temperature == 0:
        return int(np.argmax(z)), 1, 0.0, 1.0
    t = (z - z.max()) / min(max(float(temperature), 1e-30), float(np.float32(1e30)))
    order = [int(i) for i in np.lexsort((np.arange(len(z)), -z)) if z[i] > -np.inf]
    if top_k > 0:
        order = order[:top_k]
    w = np.exp(t[order])
    margin, count = 1.0, len(order)
    if top_p < 1:
        c = np.cumsum(w)
        want = max(top_p, 0.0) * c[-1]
        count = min(count, 1 + int(np.count_nonzero(c < want)))
        margin = min(margin, float(np.abs(c - want).min() / c[-1]))
    if min_p > 0:
        lim = math.log(min(min_p, 1.0))
        count = min(count, int(np.count_nonzero(t[order] >= lim)))
    kept = sorted(order[:max(count, 1)])
    c = np.cumsum(np.exp(t[kept]))
    j = min(int(np.count_nonzero(c <= a * c[-1])), len(kept) - 1)
    margin = min(margin, float(np.abs(c[:-1] - a * c[-1]).min() / c[-1]) if len(kept) > 1 else 1.0)
    return kept[j], len(kept), float(t[kept[j]] - math.log(c[-1])), margin


def score(z, temperature, token, n):
    """(logprob, rank, entropy, ids, logprobs) of a token and the n best ones
    of a row of logits; None for a row without a finite maximum."""
    z = np.asarray(z, dtype=np.float64)
    if np.isnan(z).any() or not np.isfinite(z.max()):
        return None
    t = z / min(max(float(temperature), 1e-30), float(np.float32(1e30)))
    t = t - t.max()
    lp = t - math.log(np.exp(t).sum())
    p = np.exp(lp)
    entropy = -float((p[p > 0] * lp[p > 0]).sum())
    order = [int(i) for i in np.lexsort((np.arange(len(z)), -z)) if z[i] > -np.inf][:n]
    if token < 0:
        return 0.0, -1, entropy, order, [float(lp[i]) for i in order]
    rank = int(np.count_nonzero(z > z[token]) + np.count_nonzero(z[:token] == z[token]))
    return float(lp[token]), rank, entropy, order, [float(lp[i]) for i in order]


def attention_mass(q, k, lse, scale, limits):
    """q [w][hq][d] with lse [w][hq], k [keys][hkv][d]; row i sees the first
    limits[i] keys.  Weight that each key receives, [hkv][keys]."""
    hkv = k.shape[1]
    G = q.shape[1] // hkv
    mass = np.zeros((hkv, k.shape[0]))
    for i in range(q.shape[0]):
        m = max(0, min(int(limits[i]), k.shape[0]))
        for h in range(q.shape[1]):
            if m:
                mass[h // G, :m] += np.exp(scale * (k[:m, h // G] @ q[i, h]) - lse[i, h])
    return mass


def evict(mass, ctx, keep, sink, recent):
    """Kept positions, ascending, of one request and KV head."""
    def weight(j):
        if j < sink or j >= ctx - recent:
            return (0, 0.0)
        return (2, 0.0) if math.isnan(mass[j]) else (1, -float(mass[j]))
    return sorted(sorted(range(ctx), key=lambda j: (weight(j), j))[:max(0, min(keep, ctx))])
