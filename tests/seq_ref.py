"""Plain implementations of the operators over packed sequences on the host (numpy, 64 bits).

Shares no code with the library."""

import math

import numpy as np

OK, DEVICE_INDEX, PAGES = 0, 6, 8


def pages(n, page):
    return -(-n // page)


def release(tables, free, n_free, lens, done, page):
    """(free, n_free, status) after the requests with done[b] gave their pages back."""
    free, n, status = free.copy(), int(n_free), OK
    N, room = len(free), True
    for b in range(len(lens)):
        if not done[b]:
            continue
        L = int(lens[b])
        if L < 0 or L > tables.shape[1] * page:
            status = DEVICE_INDEX
            continue
        own = tables[b, :pages(L, page)]
        if ((own < 0) | (own >= N)).any():
            status = DEVICE_INDEX
            continue
        room = room and n + len(own) <= N
        if len(own) and not room:
            status = DEVICE_INDEX
            continue
        free[n:n + len(own)] = own
        n += len(own)
    return free, n, status


def take(tables, free, n_free, lens, n_tok, page, T):
    """(tables, n_free, cu, pos, slots, statuses seen)."""
    tables, n, seen = tables.copy(), int(n_free), set()
    B, N = len(lens), len(free)
    cu, pos, slots = [0], np.full(T, -1, np.int32), np.full(T, -1, np.int32)
    asked = total = 0
    for b in range(B):
        L, t = int(lens[b]), int(n_tok[b])
        if L < 0 or t < 0 or L + t > tables.shape[1] * page:
            seen.add(DEVICE_INDEX)
            L = t = 0
        have, need = pages(L, page), pages(L + t, page) - pages(L, page)
        asked += need
        served = need == 0 or asked <= int(n_free)
        if served:
            for j in range(have, have + need):
                n -= 1
                tables[b, j] = free[n]
        else:
            seen.add(PAGES)
        if total + t > T:
            seen.add(DEVICE_INDEX if served else PAGES)
        for i in range(t):
            if total + i >= T:
                break
            p = L + i
            pos[total + i] = p
            if served:
                pg = tables[b, p // page]
                if 0 <= pg < N:
                    slots[total + i] = pg * page + p % page
                else:
                    seen.add(DEVICE_INDEX)
        total += t
        cu.append(min(total, T))
    return tables, n, np.array(cu, np.int32), pos, slots, seen


def freqs(rot, theta, scaling="none", factor=1.0, orig_len=0.0, low=1.0, high=32.0):
    """Angle of each pair per position."""
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "ramp":
        w = np.clip((orig_len * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * (w + (1 - w) / factor)
    if scaling == "ramp_index":
        def dim(r):
            return rot * math.log(orig_len / (2 * math.pi * r)) / (2 * math.log(theta))

        a, b = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        b = b + 0.001 if a == b else b
        w = 1 - np.clip((np.arange(rot // 2) - a) / (b - a), 0, 1)
        return f * (w + (1 - w) / factor)
    return f


def rope(x, pos, f, rot, interleaved=False, mscale=1.0, gain=None, layer=False, eps=1e-6):
    """Rows x [T, H, D] normalised (where there is a gain) and rotated, and a bound on the error of
    a binary32 evaluation.

    The bound: the norm's sum of D squares, root, quotient and two products give a value a
    relative error of at most (D + 8) 2^-24 (of a value less its mean, whose own error is D 2^-24
    of the row's mean magnitude); a sine is off by 2^-31 turns (2 pi 2^-31 = 2^-28.3), 2^-24 of
    the reduced angle and 2 units of its last place, under 2^-22 in all, and the turn adds two
    products and a sum: 2^-22 of both members of the pair."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    tol = np.zeros_like(x)
    if gain is not None:
        mag = np.abs(x).mean(-1, keepdims=True) if layer else 0
        x = x - x.mean(-1, keepdims=True) if layer else x
        r = 1 / np.sqrt(np.square(x).mean(-1, keepdims=True) + eps)
        # (a mean's error moves every value by it)
        tol = (np.abs(x) * (D + 8) + mag * 2 * D) * 2.0 ** -24 * r * np.abs(gain)
        x = x * r * gain
    out = x.copy()
    if rot:
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ang = np.asarray(pos, np.float64)[:, None, None] * f
        c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        both = np.abs(x[..., a]) + np.abs(x[..., b])
        t = abs(mscale) * (tol[..., a] + tol[..., b] + both * 3 * 2.0 ** -22)
        tol[..., a] = tol[..., b] = t
    return out, tol


def attend(q, K, V, pos, scale, half):
    """softmax(scale q K^T) V of rows q [n, D] at positions pos [n] over K, V [N, D], each row over
    positions p <= its own, and a bound on the error.

    A score's error is at most eps_s = (D + 16) 2^-23 sum_d |q_d k_d| scale (D products summed,
    the scale, the scaling by log2 e and its rounding; half: sums cut off instead of rounded),
    which moves a weight by a factor e^(+-2 eps_s) (numerator and denominator); weights and the
    n-term sums add (n + 32) 2^-23 of sum p |v|.  half (binary16 rows): a weight is rounded to
    binary16, 2^-11 of itself, and the result, 2^-11 of itself or 2^-25."""
    n, D = q.shape
    N = K.shape[0]
    s = q @ K.T * scale
    seen = np.arange(N)[None] <= np.asarray(pos)[:, None]
    big = (np.where(seen, np.abs(q) @ np.abs(K).T, 0)).max(1) * abs(scale)
    s = np.where(seen, s, -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out = p @ V
    mag = p @ np.abs(V)
    rel = 2 * (D + 16) * 2.0 ** -23 * big + (N + 32) * 2.0 ** -23
    tol = mag * (rel[:, None] + (2.0 ** -11 if half else 0)) + 1e-37
    if half:
        tol = tol + (np.abs(out) + tol) * 2.0 ** -11 + 2.0 ** -25
    return out, tol


def packed(q, K, V, cu, lens, scale, half, out=None):
    """Attention of all requests: q [T, H, D], K[b], V[b] [Hkv, len + n, D]."""
    T, H, D = q.shape
    out = np.zeros(q.shape) if out is None else out.astype(np.float64).copy()
    tol = np.zeros(q.shape)
    for b in range(len(cu) - 1):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if t1 <= t0:
            continue
        G = H // K[b].shape[0]
        pos = int(lens[b]) + np.arange(t1 - t0)
        for h in range(H):
            out[t0:t1, h], tol[t0:t1, h] = attend(q[t0:t1, h].astype(np.float64),
                                                  K[b][h // G].astype(np.float64),
                                                  V[b][h // G].astype(np.float64), pos, scale, half)
    return out, tol
