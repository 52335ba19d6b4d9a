"""Plain float64 definitions of what surrounds a generation step's attention. TEST INFRASTRUCTURE.

The 4-bit cache's format, block tables and slots from lengths, and the RMS norm of queries and
keys with their rotation and its gradients.  Rotations are ``oracle.attn``'s.
"""
from __future__ import annotations

import numpy as np

from . import attn as OA

__all__ = ["E2M1", "fp4_scales", "quantise_fp4", "fp4_values", "page_tables", "qk_norm_rope",
           "qk_norm_rope_bwd"]

# magnitudes of e2m1: a subnormal, then 2^(e-1) * (1 + m/2)
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_TOP = 226  # the largest scale byte that is written, of 1.25 * 2^13


def fp4_scales():
    """The scales of bytes 0..226: 5 bits of exponent (bias 15), 3 of mantissa, as in an f16."""
    b = np.arange(_TOP + 1)
    e, m = b >> 3, (b & 7) / 8.0
    return np.where(e > 0, np.exp2(e - 15.0) * (1.0 + m), np.exp2(-14.0) * m)


def _nearest(values, y):
    """Indices of the nearest of ascending values; a tie goes to the even index, what lies past the
    last to the last."""
    hi = np.clip(np.searchsorted(values, y), 1, len(values) - 1)
    up, down = values[hi] - y, y - values[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise_fp4(x):
    """(bytes [..., d/2], scale bytes [..., d/16], values [..., d]) of rows x [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(b).all(-1)
    f = np.where(bad[..., None], 0.0, b)
    code = _nearest(fp4_scales(), np.abs(f).max(-1) / 6.0)
    s = fp4_scales()[code][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, np.abs(f) / s, 0.0)
    n = _nearest(E2M1, y)
    v = np.where(np.signbit(f), -E2M1[n], E2M1[n]) * s
    n = np.where(np.signbit(f) & ~bad[..., None], n + 8, n).reshape(x.shape)
    v = np.where(bad[..., None], np.nan, v).reshape(x.shape)
    return ((n[..., 0::2] | (n[..., 1::2] << 4)).astype(np.uint8),
            np.where(bad, 255, code).astype(np.uint8), v)


def fp4_values(data, scale):
    """What bytes [..., d/2] and scale bytes [..., d/16] stand for, [..., d]."""
    data, scale = np.asarray(data).astype(np.int64), np.asarray(scale).astype(np.int64)
    n = np.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1)
    s = np.append(fp4_scales(), np.full(255 - _TOP, np.nan))[scale]
    v = np.where(n >= 8, -E2M1[n & 7], E2M1[n & 7])
    return v * np.repeat(s, 16, axis=-1)


def page_tables(held, new, table, free, num_free, N, page_size, num_pages):
    """One sequence, one token after the other: (table, seq_lens, starts, slots, positions,
    free_left, whether an error is to be reported)."""
    table = [list(map(int, r)) for r in table]
    room = len(table[0]) * page_size
    wrong = not 0 <= num_free <= len(free)
    num_free = min(max(num_free, 0), len(free))
    slots, positions = [-1] * N, [0] * N
    lens, starts, tokens, asked, taken = [], [0], 0, 0, 0
    for b, (h, n) in enumerate(zip(map(int, held), map(int, new))):
        fits = h >= 0 and n >= 0 and h + n <= room
        have = -(-h // page_size) if fits else 0
        want = -(-(h + n) // page_size) - have if fits else 0
        n0 = max(n, 0)
        ok = fits and (n0 == 0 or tokens + n0 <= N) and (want == 0 or asked + want <= num_free)
        wrong |= not ok
        if ok:
            for i in range(n0):
                row = h + i
                p = row // page_size
                if p >= have:
                    page = int(free[num_free - 1 - (asked + p - have)])
                    if 0 <= page < num_pages and row % page_size == 0:
                        table[b][p] = page
                else:
                    page = table[b][p]
                positions[tokens + i] = row
                if 0 <= page < num_pages:
                    slots[tokens + i] = page * page_size + row % page_size
                else:
                    wrong = True
            if want:
                taken = asked + want
            lens.append(h + n0)
        else:
            lens.append(h if 0 <= h <= room else 0)
        tokens += n0
        asked += want
        starts.append(min(tokens, N))
    return table, lens, starts, slots, positions, num_free - taken, wrong


def _turn(x, pos, base, layout, back=False):
    """x [B, H, T, d] turned at positions pos [B, T] (back: by the opposite angles)."""
    if base <= 0:
        return np.asarray(x, dtype=np.float64)
    fn = OA.rope_rotate_transpose if back else OA.rope_rotate
    return np.stack([fn(x[b], pos[b], base, layout) for b in range(len(x))])


def qk_norm_rope(x, w, pos, eps, base, layout, norm=True):
    """R_pos (x / sqrt(mean(x^2) + eps) * w) of heads x [B, H, T, d] (w None: gains of 1)."""
    x = np.asarray(x, dtype=np.float64)
    if norm:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        x = x if w is None else x * np.asarray(w, dtype=np.float64)
    return _turn(x, pos, base, layout)


def qk_norm_rope_bwd(dy, x, w, pos, eps, base, layout, norm=True):
    """(dx, dw) of qk_norm_rope: with n = x r, the Jacobian of n is r (I - n n^T / d)."""
    g = _turn(np.asarray(dy, dtype=np.float64), pos, base, layout, back=True)
    if not norm:
        return g, None
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x * r
    gw = g if w is None else g * np.asarray(w, dtype=np.float64)
    return r * (gw - n * np.mean(gw * n, -1, keepdims=True)), (g * n).sum((0, 1, 2))
