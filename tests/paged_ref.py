"""Plain 64-bit restatement of the paged-cache operators for the tests: numpy
on the host, one position at a time, sharing no code with the package."""
import numpy as np
import torch

GROUP = 32
MISSING, LENGTH, SHORT, BLOCK, PATH = 0x2, 0x4, 0x8, 0x10, 0x20


def e4m3_values():
    """The 256 values of e4m3, from its definition: sign, 4 exponent bits with
    bias 7, 3 fraction bits, NaN at the two all-ones codes, no infinity."""
    v = np.empty(256)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if c & 127 == 127 else (-x if s else x)
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]  # magnitudes of codes 0 .. 126, increasing


def round_e4m3(x):
    """Nearest e4m3 code of |x| <= 448, ties to the even code; NaN otherwise."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == _POS[hi], hi, code)
    code = np.where(np.isfinite(x) & (a <= 448), code | (np.signbit(x).astype(int) << 7), 0x7F)
    return code.astype(np.uint8)


def quantise(x):
    """x [..., D] float64 -> (codes [..., D], scale bytes [..., D / 32])."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    amax = np.where(np.isfinite(g), np.abs(g), 0).max(-1)
    e = np.full(amax.shape, -120)
    for k in range(-120, 121):          # smallest e with amax <= 448 * 2^e
        e = np.where(amax > 448 * 2.0 ** k, k + 1, e)
    codes = round_e4m3(g / 2.0 ** e[..., None])
    return codes.reshape(x.shape), (e + 127).astype(np.uint8)


def values(codes, scale):
    """code * 2^(byte - 127); a scale byte of 255 is E8M0's NaN."""
    v = E4M3[codes].reshape(*codes.shape[:-1], -1, GROUP)
    w = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v * w[..., None]).reshape(codes.shape)


def to64(t):
    """A tensor's values in float64 (e4m3: of the codes)."""
    if t.dtype == torch.float8_e4m3fn:
        return E4M3[t.view(torch.uint8).cpu().numpy()]
    return t.detach().double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


class Cache:
    """A cache's values in float64 and its look-up."""

    def __init__(self, k, v, tables, ks=None, vs=None):
        self.e4m3 = ks is not None
        self.k, self.v = self._vals(k, ks), self._vals(v, vs)
        self.tables = tables.cpu().numpy()
        self.bs = k.shape[-2]
        self.nb = k.shape[-4]

    @staticmethod
    def _vals(t, s):
        if s is None:
            return to64(t)
        return values(t.view(torch.uint8).cpu().numpy(), s.cpu().numpy())

    def place(self, b, pos):
        """(block, row, status) of a position."""
        j = pos // self.bs
        if j >= self.tables.shape[1]:
            return None, None, SHORT
        blk = int(self.tables[b, j])
        if blk == -1:
            return None, None, MISSING
        if blk < 0 or blk >= self.nb:
            return None, None, BLOCK
        return blk, pos % self.bs, 0


def attention(q, cache, seq_lens, new_lens, mask, scale, unit):
    """(out, lse, tol, lse_tol, live, status) in float64.

    tol bounds |computed - exact| per element for a computation that forms the
    scores and sums in fp32, rounds each probability and the result to a type
    of half-step `unit` (fp16: 2^-11, bf16: 2^-8):
      scores      |ds| <= (D + 8) 2^-24 sum_d |q_d k_d| scale (products of two
                  16-bit values are exact in fp32; one rounding per addition,
                  doubled where an addition truncates), so exp(s) is off by a
                  factor of exp(ds); 2^-20 more for exp2 itself;
      rounding p  unit * sum_j p_j |v_j|; for fp16 also 2^-25 absolute per
                  probability below its normal range, relative to the largest
                  probability, which is at least 1 before normalising; over an
                  e4m3 cache probabilities are fp16 too, the largest at least
                  2^7 before normalising: half a subnormal step, 2^-25, is
                  2^-32 of it (bf16 has no such term, its range is fp32's);
      sums        (number of keys + 8) 2^-24 relative to sum_j p_j |v_j|, for
                  numerator and denominator;
      result      unit * |out|.
    """
    B, T, Hq, D = q.shape
    Hkv = cache.k.shape[1]
    G = Hq // Hkv
    out = np.zeros((B, T, Hq, D))
    lse = np.full((B, T, Hq), -np.inf)
    tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
    live = np.zeros((B, T), dtype=bool)
    status = 0
    for b in range(B):
        L, n = int(seq_lens[b]), int(new_lens[b])
        if L < 0 or n < 0 or n > T:
            status |= LENGTH
            continue
        live[b, :n] = True
        if n == 0:
            continue
        at, pos = [], []
        for j in range(L + n):
            blk, row, st = cache.place(b, j)
            status |= st
            if blk is not None:
                at.append((blk, row))
                pos.append(j)
        pos = np.array(pos, dtype=int)
        if not len(pos):
            continue
        blk = np.array([a[0] for a in at])
        row = np.array([a[1] for a in at])
        K, V = cache.k[blk, :, row], cache.v[blk, :, row]     # [S, Hkv, D]
        for i in range(n):
            see = pos < L
            new = pos >= L
            c = pos[new] - L
            see[new] = (c <= i) if mask is None else mask[b, i, c]
            if not see.any():
                continue
            for h in range(Hq):
                k, v = K[see, h // G], V[see, h // G]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = (k @ q[b, i, h]) * scale
                    ds = (D + 8) * 2.0 ** -23 * (np.abs(k) @ np.abs(q[b, i, h])) * abs(scale)
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p /= l
                    o = p @ v
                    a = p @ np.abs(v)
                out[b, i, h] = o
                lse[b, i, h] = m + np.log(l)
                S = len(s)
                rel = 2 * ds.max() + 2.0 ** -19 + 2 * (S + 8) * 2.0 ** -24
                t = (unit + rel) * a + unit * np.abs(o)
                if cache.e4m3:
                    t = t + S * 2.0 ** -32 * np.abs(v).max(0) / l
                if unit < 2.0 ** -10:
                    t = t + S * 2.0 ** -25 * np.abs(v).max(0) / l + 2.0 ** -25
                tol[b, i, h] = t * 1.01 + 1e-37
                lse_tol[b, i, h] = ds.max() + abs(m) * 2.0 ** -22 + (S + 8) * 2.0 ** -24 + 2.0 ** -19
    return out, lse, tol, lse_tol, live, status
