"""Plain 64-bit restatements, for the tests, of a cache of 4 bits, of places for
new tokens and of norm and rotation: numpy on the host, sharing no code with the
package."""
import numpy as np

import paged_ref as ref

GROUP, TOP = 32, 215
NO_BLOCKS = 0x40
# Scale bytes: 2^(s // 8 - 14) * (1 + s % 8 / 8); bytes past TOP are NaN.
SCALE = np.array([2.0 ** (s // 8 - 14) * (1 + s % 8 / 8) if s <= TOP else np.nan for s in range(256)])


def unpack(codes):
    """Bytes [..., D / 2] -> codes [..., D], the low half first."""
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def values(codes, scale):
    c = unpack(codes).astype(np.float64) - 8
    with np.errstate(invalid="ignore"):
        return (c.reshape(*scale.shape, GROUP) * SCALE[scale][..., None]).reshape(c.shape)


def quantise(x):
    """x [..., D] float64 -> (bytes [..., D / 2], scale bytes [..., D / 32])."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0, g)
    s = np.minimum((np.abs(g).max(-1)[..., None] > 7 * SCALE[:TOP + 1]).sum(-1), TOP)
    q = np.clip(np.rint(g / SCALE[s][..., None]), -7, 7).astype(np.int64)     # rint: ties to even
    c = (q + 8).reshape(x.shape).astype(np.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4, np.where(bad, 255, s).astype(np.uint8)


class Cache(ref.Cache):
    """A cache of 4 bits for ref.attention: probabilities are of the query's type."""

    def __init__(self, k, v, tables, ks, vs):
        super().__init__(k, v, tables, ks, vs)
        self.e4m3 = False

    @staticmethod
    def _vals(t, s):
        return values(t.cpu().numpy(), s.cpu().numpy())


def reserve(L, n, tables, bs, free_list, count, mask, T):
    """(slots, positions, reserved, tables, count, status)"""
    tables = tables.copy()
    B, width = tables.shape
    slots, pos, res = np.full((B, T), -1), np.zeros((B, T), int), np.zeros(B, int)
    raw, count = count, min(max(count, 0), len(free_list))
    asked, given, status = 0, 0, 0
    for b in range(B):
        if L[b] < 0 or n[b] < 0 or n[b] > T or L[b] + n[b] >= 2 ** 31:
            status |= ref.LENGTH
            continue
        j0, j1 = -(-L[b] // bs), -(-(L[b] + n[b]) // bs)
        if n[b] and j1 > width:
            status |= ref.SHORT
            continue
        bad = 0
        if n[b] and L[b] % bs and tables[b, j0 - 1] < 0:
            bad |= ref.MISSING if tables[b, j0 - 1] == -1 else ref.BLOCK
        if (tables[b, j0:j1] < -1).any():
            bad |= ref.BLOCK
        if bad:
            status |= bad
            continue
        lack = [j for j in range(j0, j1) if tables[b, j] == -1]
        asked += len(lack)
        if lack and asked > count:
            status |= NO_BLOCKS
            continue
        for j in lack:
            tables[b, j] = free_list[count - 1 - given]
            given += 1
        res[b] = n[b]
        for i in range(n[b]):
            p = L[b] + i
            slots[b, i] = tables[b, p // bs] * bs + p % bs
            pos[b, i] = p if mask is None else L[b] + max(int(mask[b, i, :n[b]].sum()) - 1, 0)
    return slots, pos, res, tables, count - given if given else raw, status


def norm_rope(x, w, cos_sin, positions, eps, pairs):
    """(y, tol) of rows x [B, T, H, D]; tol bounds |fp32 result - y| before its last
    rounding: the sum of squares (D + 2 roundings), the root, the quotient and two
    products are off by (D / 2 + 8) 2^-24 relative at most, the rotation's products
    and sum by 3 * 2^-24 of |a cos| + |b sin|, the angles are given."""
    B, T, H, D = x.shape
    R = cos_sin.shape[1]
    y, rel = x.copy(), 0.0
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
        rel = (D / 2 + 8) * 2.0 ** -24
    big = np.abs(y)
    if R:
        c = cos_sin[positions][:, :, None, :R // 2]
        s = cos_sin[positions][:, :, None, R // 2:]
        j = np.arange(R // 2)
        ia, ib = (2 * j, 2 * j + 1) if pairs else (j, j + R // 2)
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        big[..., ia] = np.abs(a * c) + np.abs(b * s)
        big[..., ib] = np.abs(b * c) + np.abs(a * s)
    return y, (rel + 4 * 2.0 ** -24) * big
