"""Inputs and 64-bit references of the serving operators' tests (rotated append,
4-bit cache, capped and masked softmax decode), on the host in numpy and written
apart from the kernels.

Tolerances are derived from the operations, not from results:
* one rounding to a type is off by eps/2 of the value (HALF below);
* a rotation in fp32 (two products, one sum, fused or not) is off by at most
  2·2⁻²⁴·(|x1| + |x2|) before that rounding;
* a score is a sum of d products that are exact in fp32, added in fp32 in some
  order with truncation: off by at most d·2⁻²³·Σ|q_i k_i|·scale, and the cap,
  bias and exp2 argument add a few 2⁻²³ of their own sizes.  A softmax whose
  scores are off by e has weights off by a factor e^(±2e), so its output is off
  by at most (e^(2e) − 1 + n·2⁻²⁴ for the sums)·max|v|; sums over n tokens are
  taken as pairwise by warp and tile, n/16·2⁻²³ at most.
"""
from __future__ import annotations

import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rope_table(positions, rot, device="cuda", base=10000.0):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(positions)[:, None] * inv
    return torch.tensor(np.concatenate([np.cos(ang), np.sin(ang)], 1), dtype=torch.float32, device=device)


def rotate64(x, table, pos, interleaved):
    """x [rows, heads, d] float64, table np [positions, rot], pos [rows]."""
    y, rot = x.copy(), table.shape[1]
    half = rot // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = table[pos, j][:, None], table[pos, half + j][:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotation_slack(x, table, interleaved):
    """What a rotation in fp32 may be off by, per coordinate."""
    y, rot = np.zeros_like(x), table.shape[1]
    half = rot // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        y[..., a] = y[..., b] = 2 * 2.0 ** -24 * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y


def to_bf16(x):
    return torch.tensor(np.asarray(x), dtype=torch.float64).float().bfloat16()


def quantise64(row):
    """Codes, step, zero of one row of d numbers, decided in 64 bits."""
    lo, hi = float(row.min()), float(row.max())
    step, zero = float(to_bf16((hi - lo) / 15)), float(to_bf16(lo))
    if step < 1e-30:
        return np.zeros(row.size, np.int64), 0.0, zero
    return np.clip(np.rint((row - zero) / step), 0, 15).astype(np.int64), step, zero


def unpack(pool, d):
    """uint8 [.., R] records (torch) -> codes [.., 2, 16, d], step, zero [.., 2, 16] in numpy."""
    rec = pool.cpu()
    c = rec[..., : 16 * d].reshape(*rec.shape[:-1], 2, 16, d // 2).numpy().astype(np.int64)
    codes = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], d)
    sz = rec[..., 16 * d:].contiguous().view(torch.bfloat16).double().numpy().reshape(*rec.shape[:-1], 2, 16, 2)
    return codes, sz[..., 0], sz[..., 1]


def q4_values(pool, d):
    """K, V [num_phys, Hkv, S, d] in float64: zero + step·n, not rounded."""
    codes, step, zero = unpack(pool, d)
    x = zero[..., None] + step[..., None] * codes                   # [phys, Hkv, tiles, 2, 16, d]
    k, v = x[..., 0, :, :], x[..., 1, :, :]
    return tuple(y.reshape(*y.shape[:2], -1, d) for y in (k, v))


class Paged:
    """A scattered paged cache for given lengths; physical pages are shuffled, some stay unused."""

    def __init__(self, lens, hkv, d, S, seed, spare=3, max_pages=None):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hkv, self.d, self.S = list(lens), hkv, d, S
        pages = [-(-L // S) for L in lens]
        self.max_pages = max_pages or max(max(pages), 1)
        self.n_phys = sum(pages) + spare
        perm = torch.randperm(self.n_phys, generator=self.g, device="cuda").cpu()
        t, at = torch.full((len(lens), self.max_pages), int(perm[-1]), dtype=torch.int32), 0  # the last page is a spare one
        for b, n in enumerate(pages):
            t[b, :n] = perm[at: at + n]
            at += n
        self.table_h, self.pages = t.numpy(), pages
        self.table = t.cuda()
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def randn(self, *shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=self.g, device="cuda").to(dtype)

    def pools(self, dtype=torch.bfloat16):
        return (self.randn(self.n_phys, self.hkv, self.S, self.d, dtype=dtype),
                self.randn(self.n_phys, self.hkv, self.S, self.d, dtype=dtype))

    def pool_q4(self):
        R = 16 * self.d + 128
        shape = (self.n_phys, self.hkv, self.S // 16)
        pool = torch.randint(0, 256, (*shape, R), generator=self.g, device="cuda", dtype=torch.uint8)
        sz = torch.empty(*shape, 32, 2, device="cuda")
        sz[..., 0] = 0.2 + 0.3 * torch.rand(*shape, 32, generator=self.g, device="cuda")
        sz[..., 1] = -7.0 * sz[..., 0] + torch.randn(*shape, 32, generator=self.g, device="cuda")
        pool[..., 16 * self.d:] = sz.bfloat16().view(*shape, 64).view(torch.uint8)
        return pool


def sees(i, j, L, start, prefix, window):
    j = np.asarray(j)
    j = j.astype(np.int64)
    ok = (j < prefix) | ((j <= i) & ((window == 0) | (i - j < window)))
    return ok & (j >= start) & (j < L) & (i >= 0)


def decode64(pg, K, V, q, scale, *, cap=0.0, slopes=None, window=0, prefix=None, start=None, sel=None, n_sel=None):
    """(out, lse, tolerance of out per row, tolerance of lse) in float64.  K, V: float64 [n_phys, Hkv, S, d]; q: torch."""
    q = np64(q)
    B, T, Hq, d = q.shape
    G, S = Hq // pg.hkv, pg.S
    out, lse = np.zeros((B, T, Hq, d)), np.full((B, T, Hq), -np.inf)
    tol, ltol = np.zeros((B, T, Hq)), np.zeros((B, T, Hq))
    for b, L in enumerate(pg.lens):
        st = 0 if start is None else max(0, start[b])
        pf = 0 if prefix is None else prefix[b]
        for hq in range(Hq):
            h = hq // G
            pages = np.arange(pg.pages[b]) if sel is None else np.asarray(sel[b][h][: n_sel[b][h]], dtype=np.int64)
            ids = pg.table_h[b, pages].astype(np.int64)
            j = (pages[:, None] * S + np.arange(S)).reshape(-1)
            Kb, Vb = K[ids, h].reshape(-1, d), V[ids, h].reshape(-1, d)
            for t in range(T):
                i = L - T + t
                m = sees(i, j, L, st, pf, window)
                if not m.any():
                    continue
                z = Kb[m] @ q[b, t, hq] * scale
                size = (np.abs(Kb[m]) @ np.abs(q[b, t, hq]) * scale).max()
                s = cap * np.tanh(z / cap) if cap else z
                top_cap = min(cap, np.abs(z).max())  # a score is no larger than either
                dist = np.abs(i - j[m])
                e = d * 2.0 ** -23 * size + 4 * 2.0 ** -23 * (top_cap + np.abs(z).max() + 8)
                if slopes is not None:
                    s = s - slopes[hq] * dist
                    e += 4 * 2.0 ** -23 * 150 * abs(slopes[hq])  # what lies further off in score weighs nothing
                top = s.max()
                w = np.exp(s - top)
                den = w.sum()
                out[b, t, hq] = w @ Vb[m] / den
                lse[b, t, hq] = top + math.log(den)
                rel = math.expm1(2 * e) + (m.sum() / 16 + 16) * 2.0 ** -23
                tol[b, t, hq] = rel * (w @ np.abs(Vb[m])).max() / den
                ltol[b, t, hq] = rel + 4 * 2.0 ** -23 * abs(lse[b, t, hq])
                if slopes is not None:
                    ltol[b, t, hq] += 2.0 ** -22 * abs(slopes[hq]) * dist.max()
    return out, lse, tol, ltol


def check_decode(got, got_lse, want):
    out, lse, tol, ltol = want
    o = np64(got)
    assert np.isfinite(o).all()
    off = np.abs(o - out).max(-1)
    assert (off <= tol + 1e-30).all(), f"out off by {off.max():.3e}, allowed {tol.flat[int((off - tol).argmax())]:.3e}"
    e = np64(got_lse)
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(e), none)
    assert (np.abs(e[~none] - lse[~none]) <= ltol[~none]).all(), np.abs(e[~none] - lse[~none]).max()
    assert (o[none] == 0).all()
