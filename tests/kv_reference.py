"""Plain 64-bit forms of the paged-cache operators, one sequence, head and token at a
time, for the tests. They share no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np
import torch

MIN_SCALE = 2.0 ** -60
E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()     # all codes' values


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Codes of 64-bit values: nearest, ties to the even code, saturating; NaN and
    infinities give 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    mag = E4M3[:0x7F]                                            # 0 .. 448, ascending, code = index
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.clip(np.searchsorted(mag, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mag[lo], mag[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code | (np.signbit(x) * 0x80)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def page_scale(amax: float) -> float:
    s = MIN_SCALE
    while amax > 448.0 * s:
        s *= 2.0
    return s


def rotate(x, cos, sin, rot, interleaved):
    """x [H, D] float64, cos/sin [rot/2] of one position."""
    y = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[:, a] = x[:, a] * cos[i] - x[:, b] * sin[i]
        y[:, b] = x[:, b] * cos[i] + x[:, a] * sin[i]
    return y


def append(state, k, v, q, table, lens, cu, cos, sin, rot, interleaved):
    """state: dict of float64 numpy arrays k, v (values' codes as uint8) and scales;
    changed in place. Returns the rotated queries."""
    P = state["k"].shape[2]
    qo = None if q is None else q.copy()
    for b, n in enumerate(lens):
        r0, r1 = cu[b], cu[b + 1]
        T = r1 - r0
        for t in range(T):
            pos = n - T + t
            if pos < 0:
                continue
            if q is not None and rot:
                qo[r0 + t] = rotate(q[r0 + t], cos[pos], sin[pos], rot, interleaved)
        first = max(n - T, 0)
        for page in range(first // P, (n - 1) // P + 1 if n > first else first // P):
            lo, hi = max(first, page * P), min(n, (page + 1) * P)
            phys = table[b][page]
            for name, x in (("k", k), ("v", v)):
                new = []
                for pos in range(lo, hi):
                    y = x[r0 + pos - (n - T)]
                    new.append(rotate(y, cos[pos], sin[pos], rot, interleaved) if name == "k" and rot else y)
                new = np.stack(new)                                        # [n, H, D]
                for h in range(new.shape[1]):
                    vals = np.abs(new[:, h])
                    vals = vals[np.isfinite(vals)]
                    s = page_scale(vals.max() if vals.size else 0.0)
                    codes, scales = state[name], state[name + "_scale"]
                    old = scales[phys, h]
                    if lo > page * P:
                        s = max(s, old)
                        if s != old:
                            held = E4M3[codes[phys, h, :lo - page * P]] * (old / s)
                            codes[phys, h, :lo - page * P] = e4m3_encode(held)
                    codes[phys, h, lo - page * P:hi - page * P] = e4m3_encode(new[:, h] / s)
                    scales[phys, h] = s
    return qo


def attention(state, q, table, lens, cu, scale):
    """[tokens, heads, D] float64 outputs; rows without a visible key are zero."""
    P, H = state["k"].shape[2], state["k"].shape[1]
    G = q.shape[1] // H
    out = np.zeros_like(q)
    for b, n in enumerate(lens):
        r0, r1 = cu[b], cu[b + 1]
        T = r1 - r0
        if n <= 0 or T == 0:
            continue
        pages = [table[b][i] for i in range((n - 1) // P + 1)]
        for h in range(H):
            kk = np.concatenate([E4M3[state["k"][p, h]] * state["k_scale"][p, h] for p in pages])
            vv = np.concatenate([E4M3[state["v"][p, h]] * state["v_scale"][p, h] for p in pages])
            for t in range(T):
                end = n - T + t + 1
                if end <= 0:
                    continue
                for g in range(G):
                    x = kk[:end] @ q[r0 + t, h * G + g] * scale
                    with np.errstate(invalid="ignore"):
                        p = np.exp(x - x.max())
                    out[r0 + t, h * G + g] = (p @ vv[:end]) / p.sum()
    return out


def rope_table(positions, rot, base=10000.0, stretch=1.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = (torch.arange(positions, dtype=torch.float64) / stretch)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def softmax_scale(D):
    return 1.0 / math.sqrt(D)
