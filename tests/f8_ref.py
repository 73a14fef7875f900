"""Plain 64-bit reference of the 8-bit cache and of rotary positions (numpy only)."""
from __future__ import annotations

import math

import numpy as np

REP_MAX, REP_MEAN, REP_QUEST, REP_FIX = 0, 1, 2, 3


def _decode_table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


TABLE = _decode_table()                       # value of each code
GRID = TABLE[:127].copy()                     # the 127 finite magnitudes, ascending


def decode(codes):
    return TABLE[np.asarray(codes, dtype=np.uint8)]


def encode(x):
    """Codes of 64-bit values: nearest, ties to the even code, saturating; NaN 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(GRID, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - GRID[lo], GRID[hi] - a       # exact: neighbours on one grid
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.signbit(x), c | 128, c).astype(np.uint8)
    return np.where(np.isnan(x), np.where(np.signbit(x), 0xFF, 0x7F), c).astype(np.uint8)


def block_scale(amax):
    for e in range(-15, 9):
        if amax <= 448.0 * 2.0 ** e or e == 8:
            return 2.0 ** e


def code_rows(x16, s):
    """Codes of binary16 rows under scale s."""
    y = x16.astype(np.float64) / s
    top = 240.0 if s == 256.0 else 448.0
    return encode(np.where(np.isnan(y), y, np.clip(y, -top, top)))


def same_codes(a, b):
    """Equal codes; NaN of either sign is one NaN."""
    na, nb = (a & 127) == 127, (b & 127) == 127
    return bool(((a == b) | (na & nb)).all())


class Cache:
    """Host copy of an 8-bit cache: code pools uint8 [P][H][128][128], scales [P][H]."""

    def __init__(self, k_code, k_scale, v_code, v_scale, table, lens):
        self.code = {"k": k_code.copy(), "v": v_code.copy()}
        self.scale = {"k": k_scale.astype(np.float64), "v": v_scale.astype(np.float64)}
        self.table, self.lens = table.copy(), lens.copy()

    def append(self, k16, v16, counts):
        """Rows of binary16 k16 / v16 ([tokens][H][128]), counts[b] of them to sequence b.
        Returns the (b, j) of the blocks completed."""
        done, at = [], 0
        for b, m in enumerate(counts):
            n = int(self.lens[b])
            pos = n
            while pos < n + m:
                j, r0 = divmod(pos, 128)
                r1 = min(128, n + m - j * 128)
                page = int(self.table[b, j])
                rows = slice(at + pos - n, at + pos - n + r1 - r0)
                for side, x in (("k", k16), ("v", v16)):
                    for h in range(x.shape[1]):
                        new = x[rows, h]
                        mag = np.abs(new.astype(np.float64))
                        mag = np.where(np.isnan(mag), 0.0, mag)
                        s = block_scale(min(mag.max(), 65504.0))
                        code = self.code[side][page, h]
                        if r0:
                            old = self.scale[side][page, h]
                            s = max(s, old)
                            if s > old:
                                code[:r0] = encode(decode(code[:r0]) * (old / s))
                        code[r0:r1] = code_rows(new, s)
                        self.scale[side][page, h] = s
                if r1 == 128:
                    done.append((b, j))
                pos += r1 - r0
            at += m
            self.lens[b] = n + m
        return done

    def values(self, side, page, h):
        return decode(self.code[side][page, h]) * self.scale[side][page, h]

    def reps(self, page, h, rep, stride=32):
        x = self.values("k", page, h)
        if rep == REP_MAX:
            return x.max(0, keepdims=True)
        if rep == REP_QUEST:
            return np.stack([x.min(0), x.max(0)])
        if rep == REP_MEAN:
            return x.sum(0, keepdims=True) / 128.0
        return x[::stride]

    def attend(self, q, b, h, blocks, scale):
        """softmax(scale q K^T) V over `blocks` of sequence b, sum p |v|, the largest
        scale sum |q k| of a score, and sum |v| / sum exp(s - max s); q [G][128]."""
        n = int(self.lens[b])
        k = np.concatenate([self.values("k", int(self.table[b, j]), h)[:max(0, n - j * 128)]
                            for j in blocks])
        v = np.concatenate([self.values("v", int(self.table[b, j]), h)[:max(0, n - j * 128)]
                            for j in blocks])
        s = q.astype(np.float64) @ k.T * scale
        p = np.exp(s - s.max(-1, keepdims=True))
        total = p.sum(-1, keepdims=True)
        p /= total
        return (p @ v, p @ np.abs(v), (np.abs(q.astype(np.float64)) @ np.abs(k).T).max() * scale,
                np.abs(v).sum(0)[None] / total)


def frequencies(rot, theta, scaling="plain", factor=1.0, original_len=0, fast=32.0, slow=1.0):
    """f_i in long double, and the amplitude."""
    L = np.longdouble
    theta = L(theta)
    if scaling == "ntk":
        theta = theta * L(factor) ** (L(rot) / L(rot - 2))
    f = []
    for i in range(rot // 2):
        w = theta ** (L(-2 * i) / L(rot))
        if scaling == "linear":
            w = w / L(factor)
        if scaling == "yarn":
            def edge(beta):
                return rot * math.log(original_len / (beta * 2 * math.pi)) / (2 * math.log(theta))
            lo = min(max(math.floor(edge(fast)), 0), rot - 1)
            hi = min(max(math.ceil(edge(slow)), 0), rot - 1)
            r = L(min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0))
            w = w / L(factor) * r + w * (1 - r)
        if scaling == "bands":
            t = L(original_len) * w / (2 * L(np.pi))
            r = min(max((t - slow) / (fast - slow), L(0)), L(1))
            w = w * r + w / L(factor) * (1 - r)
        f.append(w)
    return np.array(f, dtype=np.longdouble), \
        (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


PI2 = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))


def rotate(x, positions, f, amplitude, layout):
    """Rows [tokens][heads][128] rotated in 64 bits, and |x| + |y| of each channel's pair (0 where
    a channel passes through)."""
    x = x.astype(np.float64)
    n = len(f)
    ang = np.fmod(positions.astype(np.longdouble)[:, None] * f[None], PI2).astype(np.float64)
    cos, sin = (np.cos(ang) * amplitude)[:, None], (np.sin(ang) * amplitude)[:, None]
    out, mag = x.copy(), np.zeros_like(x)
    i = np.arange(n)
    a, b = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, mag


def rope_tolerance(want, mag, positions, f, amplitude):
    """Bound of |got - want|: the rounding to binary16 (2^-11 of the value, 2^-25 below its normal
    range), and in binary32 for |x| + |y|: two products, a sum, the amplitude (2^-24 each), sine
    and cosine to 2 ulp (2^-22), the angle's 32-bit fraction (2 pi 2^-33) and the frequency's
    binary64 roundings (2^-51 of the angle)."""
    far = np.abs(positions.astype(np.float64)).max() * float(max(f)) * 2.0 ** -51 if len(f) else 0
    work = mag * amplitude * (4 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -30 + far)
    return 2.0 ** -11 * (np.abs(want) + work) + 2.0 ** -25 + work
