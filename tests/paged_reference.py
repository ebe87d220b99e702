"""Plain 64-bit implementation of the paged-cache operators, for the tests: the rows of an entry gathered
one by one through the page table, the attention by its definition, the eviction by sorting.  Also the
tolerances: how far bf16 outputs and fp32 statistics of a kernel that multiplies bf16 values exactly and
adds in fp32 can be from it."""
from __future__ import annotations

import numpy as np
import torch

from block_discrete_diffusion_tcgen05_b200 import synth


def bf16(shape, seed, sigma=1.0):
    """Seeded normals as a CPU torch.bfloat16 tensor."""
    return synth.to_torch(synth.normal_bf16(shape, seed, sigma))


def f64(t):
    return t.float().numpy().astype(np.float64)


class Cache:
    """A pool and its table on the CPU.  page = 0: contiguous caches.  Rows of no entry are NaN, table
    entries past an entry's rows `junk`."""

    def __init__(self, B, Hkv, d, page, P, capacity, seed, sigma_k=1.0, sigma_v=1.0, junk=-7, spare=3):
        self.B, self.Hkv, self.d, self.page, self.P = B, Hkv, d, page, list(P)
        rng = np.random.default_rng(seed)
        if page:
            each = max(1, -(-capacity // page))
            self.capacity = each * page
            n = B * each + spare
            order = rng.permutation(n)[:B * each].reshape(B, each).astype(np.int32)
            for b in range(B):
                order[b, -(-self.P[b] // page):] = junk
            self.all_pages = rng.permutation(n)
            self.table = torch.from_numpy(order)
            rows = page
        else:
            self.capacity, n, rows, self.table = capacity, B, capacity, None
        self.k = bf16((n, Hkv, rows, d), seed + 1, sigma_k)
        self.v = bf16((n, Hkv, rows, d), seed + 2, sigma_v)
        live = torch.zeros((n, rows), dtype=torch.bool)
        for b in range(B):
            for r in range(self.P[b]):
                pg, i = self.where(b, r)
                live[pg, i] = True
        for t in (self.k, self.v):
            t.masked_fill_(~live[:, None, :, None], float("nan"))

    def where(self, b, r):
        if self.table is None:
            return b, r
        return int(self.table[b, r // self.page]), r % self.page

    def rows(self, t, b, h, n):
        """The first n rows of entry b, head h of a pool tensor."""
        if n == 0:
            return t[0, h, :0]
        return torch.stack([t[pg, h, i] for pg, i in (self.where(b, r) for r in range(n))])

    def cuda(self):
        """(k, v, table, P) on the GPU."""
        return (self.k.cuda(), self.v.cuda(), None if self.table is None else self.table.cuda(),
                torch.tensor(self.P, dtype=torch.int32, device="cuda"))


def score_slack(q, k, scale, d):
    """Bound on the relative error of exp(x - lse) from the scores: the sum of d products in fp32 (at most
    one unit, 2^-23, of the terms' absolute sum per addition), the scaling and exponent arguments (2^-23 of
    the score's size each), the hardware exponential (2^-22) and the sums' own units."""
    big = np.abs(q) @ np.abs(k).T * scale if k.shape[0] else np.zeros((q.shape[0], 1))
    return ((d + 8) * 2.0 ** -23 * big.max(axis=1) + 2.0 ** -20)[:, None]


def sample(cache, q, k_blk, v_blk, scale=None, skip=()):
    """(out, lse, tolerance of out, tolerance of lse), all [B][Hq][S]...; skip: (entry, row) pairs that
    take no part."""
    B, Hq, S, d = q.shape
    G = Hq // cache.Hkv
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros((B, Hq, S, d)), np.full((B, Hq, S), -np.inf)
    tol_o, tol_l = np.zeros_like(out), np.zeros((B, Hq, S))
    for b in range(B):
        use = [r for r in range(cache.P[b]) if (b, r) not in skip]
        for h in range(cache.Hkv):
            k, v = ([cache.where(b, r) for r in use],) * 2
            k = np.array([f64(cache.k[pg, h, i]) for pg, i in k]).reshape(-1, d)
            v = np.array([f64(cache.v[pg, h, i]) for pg, i in v]).reshape(-1, d)
            if k_blk is not None:
                k, v = np.concatenate([k, f64(k_blk[b, h])]), np.concatenate([v, f64(v_blk[b, h])])
            if not len(k):
                continue
            for g in range(G):
                hq = h * G + g
                qq = f64(q[b, hq])
                x = qq @ k.T * scale
                m = x.max(axis=1, keepdims=True)
                e = np.exp(x - m)
                l = e.sum(axis=1, keepdims=True)
                p = e / l
                out[b, hq] = p @ v
                lse[b, hq] = (m + np.log(l))[:, 0]
                rel = score_slack(qq, k, scale, d)
                # one rounding to bf16 (half a step), and numerator and denominator off by rel each; the
                # probabilities are held to 16 bits and more (2^-16)
                tol_o[b, hq] = 2.0 ** -8 * np.abs(out[b, hq]) + (2 * rel + 2.0 ** -16) * (p @ np.abs(v))
                tol_l[b, hq] = (rel + 2.0 ** -22 * np.abs(lse[b, hq])[:, None])[:, 0]
    return out, lse, tol_o, tol_l


def check_sample(got, ref, what=""):
    out, lse, tol_o, tol_l = ref
    o, l = f64(got[0].cpu()), got[1].cpu().numpy().astype(np.float64)
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(l), none), what
    assert np.isfinite(o).all() and np.isfinite(l[~none]).all(), f"{what}: not finite"
    worst_o = (np.abs(o - out) - tol_o).max()
    worst_l = (np.abs(l[~none] - lse[~none]) - tol_l[~none]).max() if (~none).any() else 0.0
    assert worst_o <= 0, f"{what}: out off by {np.abs(o - out).max():.3e}, over its tolerance by {worst_o:.3e}"
    assert worst_l <= 0, f"{what}: lse off by {np.abs(l - lse)[~none].max():.3e}, over by {worst_l:.3e}"


def weigh(cache, q, lse, weight, scale=None, skip=()):
    """(weight_out, tolerance) for the rows below each length; lse, weight: fp32 CPU tensors."""
    B, Hq, S, d = q.shape
    G = Hq // cache.Hkv
    scale = d ** -0.5 if scale is None else scale
    out = weight.numpy().astype(np.float64)
    tol = np.zeros_like(out)
    L = lse.numpy().astype(np.float64)
    for b in range(B):
        P = cache.P[b]
        for h in range(cache.Hkv):
            k = f64(cache.rows(cache.k, b, h, P)).reshape(-1, d)
            add = np.zeros(P)
            err = np.zeros(P)
            for g in range(G):
                hq = h * G + g
                qq = f64(q[b, hq])
                x = qq @ k.T * scale
                for s in range(S):
                    if np.isneginf(L[b, hq, s]):
                        continue
                    p = np.exp(x[s] - L[b, hq, s])
                    # the exponent's argument is a difference of fp32 values of lse's and the score's size
                    slack = score_slack(qq[s:s + 1], k, scale, d)[0, 0] + 2.0 ** -22 * abs(L[b, hq, s])
                    add += p
                    err += p * slack
            for r in range(P):
                if (b, r) in skip:
                    add[r] = err[r] = 0.0
            out[b, h, :P] += add
            tol[b, h, :P] = err + (G * S + 2) * 2.0 ** -23 * np.abs(out[b, h, :P])
    return out, tol


def rank_key(w, pos, protect):
    """Sort key of a row, larger stays: protected rows, then the weights, NaN below all."""
    if pos >= protect:
        return (2, 0.0)
    if np.isnan(w):
        return (0, 0.0)
    return (1, float(w) + 0.0)


def evict(P, weight, pos, tokens, keep, recent):
    """Per head lists of (source row, target row) and the new weight and pos rows: weight, pos numpy [rows]."""
    if P <= keep:
        return [], weight[:P].copy(), pos[:P].copy()
    order = sorted(range(P), key=lambda j: tuple(-x for x in rank_key(weight[j], int(pos[j]), int(tokens) - recent)) + (j,))
    kept = set(order[:keep])
    holes = [j for j in range(keep) if j not in kept]
    movers = [j for j in range(keep, P) if j in kept]
    assert len(holes) == len(movers)
    w, ps = weight[:keep].copy(), pos[:keep].copy()
    for s, t in zip(movers, holes):
        w[t], ps[t] = weight[s], pos[s]
    return list(zip(movers, holes)), w, ps


def bits(t):
    """bf16 tensor -> uint16 bit patterns (NaN compares by its bits)."""
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)
