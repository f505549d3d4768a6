"""Paged-cache batches for the tests, and the operators by their definition in 64 bits."""

from __future__ import annotations

import math

import numpy as np
import torch

ANY_ENTRY = 0x7FFFFFF0  # table entry of a page that no call may look up


class Batch:
    """A packed batch over a paged cache.

    Positions of sequence b before starts[b] + lens[b] have keys and values (host, float64,
    exactly bf16); pages that a window W with `sinks` still sees are in the cache, everything
    else in the cache is NaN and every other table entry is ANY_ENTRY.
    """

    def __init__(self, lens, starts, H, Hkv, d, page, W, sinks=0, layout="hnd", seed=0, lead=0,
                 trail=0, spare=2, written_only=False):
        rng = np.random.default_rng(seed)
        self.lens, self.starts, self.H, self.Hkv, self.d, self.page = lens, starts, H, Hkv, d, page
        self.W, self.sinks, self.lead = W, sinks, lead
        n = len(lens)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64) + lead
        self.total = int(self.cu[-1]) + trail
        self.end = [s + m for s, m in zip(starts, lens)]

        def normal(shape):
            x = torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16)
            return x

        self.q = normal((self.total, H, d))
        self.max_pages = max(1, max((e + page - 1) // page for e in self.end)) + 1
        visible = [self.visible(b) for b in range(n)]
        self.keys = [normal((len(v), Hkv, d)) for v in visible]
        self.vals = [normal((len(v), Hkv, d)) for v in visible]
        pages = [sorted({int(p) // page for p in v}) for v in visible]
        self.n_pages = sum(map(len, pages)) + spare
        ids = rng.permutation(self.n_pages)
        self.table = np.full((n, self.max_pages), ANY_ENTRY, dtype=np.int32)
        flat = 0
        kc = torch.full((self.n_pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16)
        vc = torch.full_like(kc, float("nan"))
        for b in range(n):
            for p in pages[b]:
                self.table[b, p] = ids[flat]
                flat += 1
            if len(visible[b]):
                at = torch.from_numpy(self.table[b, visible[b] // page].astype(np.int64))
                slot = torch.from_numpy(visible[b] % page)
                kc[at, :, slot] = self.keys[b]
                vc[at, :, slot] = self.vals[b]
        self.pos_of = visible
        self.kc_host, self.vc_host = kc, vc
        self.k_cache, self.v_cache = self._device(kc, layout), self._device(vc, layout)
        self.scale = 1.0 / math.sqrt(d)
        self.t_table = torch.from_numpy(self.table).cuda()
        self.t_cu = torch.from_numpy(self.cu).cuda()
        self.t_first = torch.tensor(starts, dtype=torch.int64).cuda()

    @staticmethod
    def _device(c, layout):
        if layout == "hnd":
            return c.cuda()
        return c.transpose(1, 2).contiguous().cuda().transpose(1, 2)

    def visible(self, b):
        """Positions that some query of the batch sees."""
        if self.lens[b] == 0:
            return np.zeros(0, dtype=np.int64)
        low = max(0, self.starts[b] - self.W + 1)
        return np.concatenate([np.arange(min(self.sinks, low)), np.arange(low, self.end[b])])

    def expect(self, drop=None):
        """out, lse [total, H] and the tolerances of both, in 64 bits; NaN outside sequences.

        The kernels round the weights to bf16 (2^-8 of each), the output to bf16 (2^-8), and form
        scores and sums in 32 bits: a score is off by at most d roundings of 2^-23 of the sum of
        its products' magnitudes, its exponential by 2^-22 and that score error twice (numerator
        and sum), and adding n weights or weighted values in 32 bits by n 2^-23 at most.
        drop: table entries (b, page) that the call finds out of range: keys, values are zero.
        """
        out = np.full((self.total, self.H, self.d), np.nan)
        lse = np.full((self.total, self.H), np.nan)
        tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
        G = self.H // self.Hkv
        for b, (n, s) in enumerate(zip(self.lens, self.starts)):
            if n == 0:
                continue
            rows = slice(int(self.cu[b]), int(self.cu[b + 1]))
            q = self.q[rows].double().numpy().reshape(n, self.Hkv, G, self.d)
            k = self.keys[b].double().numpy().copy()
            v = self.vals[b].double().numpy().copy()
            kp, qp = self.pos_of[b], np.arange(s, s + n)
            if drop:
                gone = np.array([(b, int(p) // self.page) in drop for p in kp])
                k[gone] = 0
                v[gone] = 0
            seen = (kp[None] <= qp[:, None]) & ((kp[None] > qp[:, None] - self.W) |
                                                (kp[None] < self.sinks))
            x = np.einsum("thgd,khd->thgk", q, k, optimize=True) * self.scale
            ax = np.einsum("thgd,khd->thgk", np.abs(q), np.abs(k), optimize=True) * self.scale
            x = np.where(seen[:, None, None], x, -np.inf)
            ds = np.where(seen[:, None, None], ax, 0).max(-1) * self.d * 2.0 ** -23
            m = x.max(-1, keepdims=True)
            p = np.exp(x - m)
            z = p.sum(-1, keepdims=True)
            o = np.einsum("thgk,khd->thgd", p / z, v, optimize=True)
            a = np.einsum("thgk,khd->thgd", p / z, np.abs(v), optimize=True)
            off = 2 * ds + 2.0 ** -22 + len(kp) * 2.0 ** -23
            out[rows] = o.reshape(n, self.H, self.d)
            lse[rows] = (m + np.log(z))[..., 0].reshape(n, self.H)
            t = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + off)[..., None] * a * (1 + 2.0 ** -8)
            tol[rows] = t.reshape(n, self.H, self.d)
            tol_lse[rows] = (off + 2.0 ** -22 * (1 + np.abs(m[..., 0]))).reshape(n, self.H) + 1e-6
        return out, lse, tol, tol_lse


def rotate(x, pos, inv_freq, interleaved):
    """x [tokens, heads, d] float64 turned by pos [tokens, pairs] * inv_freq [pairs]."""
    half = len(inv_freq)
    if half == 0:
        return x.copy()
    angle = pos.astype(np.float64) * inv_freq.astype(np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y = x.copy()
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotation_tolerance(x, pos, inv_freq, interleaved):
    """Half a step of bf16 of the result, plus 2^-21 of the pair's magnitude: four roundings of
    products and sum, and cosine and sine to 2^-22."""
    y = np.abs(rotate(x, pos, inv_freq, interleaved))
    half = len(inv_freq)
    mag = np.zeros_like(x)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    mag[..., a] = mag[..., b] = np.hypot(x[..., a], x[..., b])
    return 2.0 ** -8 * y + 2.0 ** -21 * mag * (1 + 2.0 ** -8)
