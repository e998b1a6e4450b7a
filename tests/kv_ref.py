"""Plain implementations of the KV-cache operators on the host (numpy, 64 bits).

Shares no code with the library.  A cache is held as the values it stands for
(binary64) plus, for 8-bit storage, its codes and scales.
"""

import math

import numpy as np

F32 = np.float32


def quantise(x):
    """Codes (int8) and scales (binary32) of rows x [..., D] (binary32 values)."""
    x = np.asarray(x, F32)
    fine = np.isfinite(x).all(-1)
    amax = np.abs(np.where(fine[..., None], x, 0)).max(-1).astype(F32)
    s = np.maximum(amax / F32(127), F32(2.0 ** -126)).astype(F32)
    q = np.rint(np.where(fine[..., None], x, 0) / s[..., None]).astype(np.int8)
    return np.where(fine[..., None], q, 0).astype(np.int8), np.where(fine, s, F32(np.nan))


class RefCache:
    def __init__(self, B, Hkv, cap, D, dtype, block=0, rng=None):
        self.B, self.Hkv, self.cap, self.D, self.dtype, self.block = B, Hkv, cap, D, dtype, block
        shape = (B, Hkv, cap, D)
        self.raw = {}
        self.scale = {}
        for t in ("k", "v"):
            x = rng.standard_normal(shape).astype(F32) if rng is not None else np.zeros(shape, F32)
            if dtype == "i8":
                self.raw[t], self.scale[t] = quantise(x)
            else:
                self.raw[t] = x.astype(F32 if dtype == "f32" else np.float16)
        nb = cap // block if block else 0
        self.mean = np.zeros((B, Hkv, nb, D), np.int8)
        self.mean_scale = np.zeros((B, Hkv, nb), F32)
        if block:
            for b in range(B):
                for h in range(Hkv):
                    for j in range(nb):
                        self.set_mean(b, h, j)

    def values(self, t):
        """The cached values as binary32 numbers (in binary64)."""
        with np.errstate(invalid="ignore"):
            x = self.raw[t].astype(F32)
            if self.dtype == "i8":
                x = x * self.scale[t][..., None]
        return x.astype(np.float64)

    def set_mean(self, b, h, j):
        n = self.block
        x = self.raw["k"][b, h, j * n:(j + 1) * n].astype(F32)
        if self.dtype == "i8":
            x = x * self.scale["k"][b, h, j * n:(j + 1) * n, None]
        if not np.isfinite(x).all():
            self.mean[b, h, j], self.mean_scale[b, h, j] = 0, np.inf
            return
        e = max(int(np.frexp(np.abs(x).max())[1]), -100)
        g = math.ldexp(n, e - 24)
        total = np.rint(x.astype(np.float64) / g).sum(0)
        assert np.abs(total).max() < 2 ** 24
        self.mean[b, h, j], self.mean_scale[b, h, j] = quantise((total * math.ldexp(1, e - 24))
                                                                .astype(F32))

    def _finish(self, b, lo, hi):
        if self.block:
            for j in range(self.cap // self.block):
                if lo <= (j + 1) * self.block - 1 < hi:
                    for h in range(self.Hkv):
                        self.set_mean(b, h, j)

    def append(self, k, v, lens, n_tok):
        for b in range(self.B):
            lo, n = int(lens[b]), int(n_tok[b])
            for t, x in (("k", k), ("v", v)):
                new = np.asarray(x, F32)[b, :n].transpose(1, 0, 2)
                if self.dtype == "i8":
                    self.raw[t][b, :, lo:lo + n], self.scale[t][b, :, lo:lo + n] = quantise(new)
                else:
                    with np.errstate(over="ignore"):
                        self.raw[t][b, :, lo:lo + n] = new.astype(self.raw[t].dtype)
            self._finish(b, lo, lo + n)

    def keep(self, lens, path, n_keep):
        for b in range(self.B):
            lo, n = int(lens[b]), int(n_keep[b])
            src = lo + np.asarray(path[b][:n], np.int64)
            for d in (self.raw, self.scale):
                for t in d:
                    d[t][b, :, lo:lo + n] = d[t][b, :, src].swapaxes(0, 1) if n else \
                        d[t][b, :, lo:lo + n]
            self._finish(b, lo, lo + n)


def attend(q, K, V, scale):
    """softmax(scale q K^T) V for q [D], K, V [n, D]; zeros for n = 0; and a bound on the error
    of a binary32 evaluation.

    The bound: a score's error is at most eps_s = (D + 16) 2^-23 sum_d |q_d k_d| scale (D
    rounded products and sums, the query's split into two binary16 parts with a remainder below
    2^-22 of its largest element, the scale and the scaling by log2 e), which moves a weight by
    a factor e^(+-2 eps_s) (numerator and denominator); weights, their split and the n-term sums
    add (n + 32) 2^-23 of sum p |v|."""
    D = q.shape[0]
    if K.shape[0] == 0:
        return np.zeros(D), 0.0
    s = K @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    eps = (D + 16) * 2.0 ** -23 * float((np.abs(K) @ np.abs(q)
                                         + np.abs(K).sum(1) * np.abs(q).max() / D).max()) * abs(scale)
    mag = float((p @ np.abs(V)).max())
    return p @ V, mag * (2 * eps + (K.shape[0] + 32) * 2.0 ** -23) + 1e-37


def tree(cache, q, lens, n_tok, mask, scale, heads=None, out=None):
    """(out, tolerance) [B, T, H, D] / [B, T, H]; mask [B][T] ints (None: causal)."""
    B, T, H, D = q.shape
    G = H // cache.Hkv
    out = np.zeros(q.shape) if out is None else out.astype(np.float64).copy()
    tol = np.zeros((B, T, H))
    K, V = cache.values("k"), cache.values("v")
    for b in range(B):
        L = int(lens[b])
        for t in range(int(n_tok[b])):
            bits = (2 << t) - 1 if mask is None else int(mask[b][t])
            pos = list(range(L)) + [L + j for j in range(int(n_tok[b])) if bits >> j & 1]
            for h in (range(cache.Hkv) if heads is None else heads):
                for a in range(h * G, h * G + G):
                    out[b, t, a], tol[b, t, a] = attend(q[b, t, a].astype(np.float64),
                                                        K[b, h, pos], V[b, h, pos], scale)
    return out, tol


def topk(cache, q, lens, k, n_first=1, n_last=1):
    B, H, D = q.shape
    G, n = H // cache.Hkv, cache.block
    idx = np.full((B, H, k), -1, np.int32)
    qc, _ = quantise(q)
    for b in range(B):
        nb = -(-int(lens[b]) // n)
        for h in range(H):
            if nb <= k:
                idx[b, h, :nb] = np.arange(nb)
                continue
            must = set(range(n_first)) | set(range(nb - n_last, nb))
            rest = [j for j in range(nb) if j not in must]
            ms = cache.mean_scale[b, h // G]
            dots = cache.mean[b, h // G].astype(np.int64) @ qc[b, h].astype(np.int64)
            with np.errstate(invalid="ignore"):
                score = [np.inf if np.isinf(ms[j]) else F32(dots[j]) * ms[j] for j in rest]
            order = sorted(range(len(rest)), key=lambda i: (-score[i], rest[i]))
            idx[b, h] = sorted(must | {rest[i] for i in order[:k - len(must)]})
    return idx


def block_attend(cache, q, lens, idx, scale):
    B, H, D = q.shape
    G, n = H // cache.Hkv, cache.block
    out, tol = np.zeros(q.shape), np.zeros((B, H))
    K, V = cache.values("k"), cache.values("v")
    for b in range(B):
        L = int(lens[b])
        nb = -(-L // n)
        for h in range(H):
            pos = [p for j in idx[b, h][:min(idx.shape[2], nb)] if 0 <= j < nb
                   for p in range(j * n, min((j + 1) * n, L))]
            out[b, h], tol[b, h] = attend(q[b, h].astype(np.float64), K[b, h // G, pos],
                                          V[b, h // G, pos], scale)
    return out, tol
