"""Plain reference of the paged 8-bit cache in numpy: its number format bit by bit, the
blocks' scales and how older rows follow them, and attention in fp64."""
from __future__ import annotations

import numpy as np

from kv4_ref import E4M3, f64

MIN_E, MAX_E = -32, 32
_POS = E4M3[:127]                       # the codes 0..126 ascend
_MIDS = (_POS[1:] + _POS[:-1]) / 2


def e4m3(y):
    """fp64 -> codes: to nearest, ties to the even code, past 448 to 448, NaN to 0x7F."""
    y = np.asarray(y, np.float64)
    a = np.where(np.isnan(y), 0, np.abs(y))
    low, high = np.searchsorted(_MIDS, a, "left"), np.searchsorted(_MIDS, a, "right")
    c = np.where((low != high) & (low % 2 == 1), high, low).astype(np.uint8)
    return np.where(np.isnan(y), np.uint8(0x7F), c | (np.signbit(y).astype(np.uint8) << 7))


def need(x):
    """The exponent of a block of values: the smallest e with max|x| <= 448 2^e."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    e = MIN_E
    while e < MAX_E and top > 448 * 2.0 ** e:
        e += 1
    return e


def exponent(byte):
    return np.clip(np.asarray(byte, np.int64) - 127, MIN_E, MAX_E)


class Cache:
    """A paged cache on the host, filled by append(); random bytes (NaN codes among them)
    stand wherever no row is written."""

    def __init__(self, rng, N, Hkv, d, page, block, lengths, spare=2):
        self.N, self.Hkv, self.d, self.page, self.block = N, Hkv, d, page, block
        wants = [max(0, -(-int(x) // page)) for x in lengths]
        self.max_pages = max(1, max(wants))
        self.n_pages = sum(wants) + spare
        perm = rng.permutation(self.n_pages)[: sum(wants)]
        self.table = np.full((N, self.max_pages), -1, np.int32)
        at = 0
        for n, m in enumerate(wants):
            self.table[n, :m] = perm[at: at + m]
            at += m
        self.codes = rng.integers(0, 256, (2, self.n_pages, Hkv, page, d), dtype=np.uint8)
        self.codes[rng.random(self.codes.shape) < 0.2] = 0x7F
        self.scales = rng.integers(0, 256, (2, self.n_pages, Hkv, page // block), dtype=np.uint8)

    def write(self, n, start, k, v):
        """Appends rows k, v [T, Hkv, d] (values that bf16 holds) of sequence n at `start`."""
        T = len(k)
        for b in range(start // self.block, -(-(start + T) // self.block) if T else 0):
            p0 = b * self.block
            ph = self.table[n, p0 // self.page]
            if ph < 0:
                continue
            r0, sb = p0 % self.page, p0 % self.page // self.block
            lo, hi = max(p0, start), min(p0 + self.block, start + T)
            for kv, x in enumerate((k, v)):
                for g in range(self.Hkv):
                    new = np.asarray(x[lo - start: hi - start, g], np.float64)
                    e = need(new)
                    rows = self.codes[kv, ph, g]
                    if p0 < start:
                        old = int(exponent(self.scales[kv, ph, g, sb]))
                        if e > old:
                            part = rows[r0: r0 + start - p0]
                            rows[r0: r0 + start - p0] = e4m3(E4M3[part] * 2.0 ** (old - e))
                        e = max(e, old)
                    with np.errstate(over="ignore", invalid="ignore"):
                        rows[r0 + lo - p0: r0 + hi - p0] = e4m3(new * 2.0 ** -e)
                    self.scales[kv, ph, g, sb] = e + 127

    def rows(self, i, n, pos):
        """fp64 values [Hkv, len(pos), d] of K (i = 0) or V; pages must exist."""
        pos = np.asarray(pos, np.int64)
        ph, r = self.table[n, pos // self.page], pos % self.page
        return (E4M3[self.codes[i].transpose(0, 2, 1, 3)[ph, r]]
                * 2.0 ** self.exps(i, n, pos)[..., None].transpose(1, 0, 2)).transpose(1, 0, 2)

    def exps(self, i, n, pos):
        """Scale exponents [Hkv, len(pos)]."""
        pos = np.asarray(pos, np.int64)
        ph, r = self.table[n, pos // self.page], pos % self.page
        return exponent(self.scales[i].transpose(0, 2, 1)[ph, r // self.block]).T


def attention(q, cache, lengths, bk=None, bv=None, scale=None):
    """fp64 attention of q [N][B][Hq][d] (bf16 bits) over the cache and the block's keys, and
    the bound of an implementation that holds queries as two e4m3 numbers and weights as
    four of them (few rows per KV head) or one fp16 (many), accumulates in fp32, handles
    the block's keys in fp32 and rounds the output to bf16.  A bf16 query has 8 bits: two
    numbers of 4 hold it but for e4m3's smallest step, 2^-9 (half of it lost), with the
    row's largest query at 2^7 or above; with few rows the second number stands for 2^-4.
      2^-8 |out|                       the output's rounding (half a bf16 step)
      2^-11 A_c                        a weight's rounding; A = sum_j p_j |v_j| over the
                                       cache (A_c) and over the block keys (A_b)
      2 delta (A_c + A_b)              relative error of each weight and of the row sum:
                                       delta = scale max_j sum_i ((d + 8) 2^-24 |q_i k_ji|
                                       + qs max|q| |k_ji|) + 2^-21: fp32 sums of d products,
                                       queries below a step (qs = 2^-21, many rows 2^-17),
                                       exp2
      2^-13 (A_c + A_b)                fp32 sums over up to 2^10 matrix steps
      2^-26 sum_c |v_j| 2^(top - e_j)  weights below a step: with few rows four numbers go
                                       down to 2^-21 (half of it lost) where a weight times
                                       its value's scale over the head's largest scale
                                       (exponents e_j, top) is held times 2^4 at least and
                                       the row's sum is 1 or more; with many rows fp16 holds
                                       more
    Returns (out, bound)."""
    N, B, Hq, d = q.shape
    G = Hq // cache.Hkv
    scale = 1 / np.sqrt(d) if scale is None else scale
    qs = 2.0 ** (-21 if B * G <= 16 else -17)
    qf = f64(q)
    out = np.zeros((N, B, Hq, d))
    tol = np.zeros_like(out)
    for n in range(N):
        L = int(lengths[n])
        pos = np.arange(L)
        pos = pos[cache.table[n, pos // cache.page] >= 0]
        k, v = cache.rows(0, n, pos), cache.rows(1, n, pos)
        ve = cache.exps(1, n, pos)
        m = k.shape[1]
        if bk is not None:
            k = np.concatenate((k, f64(bk[n]).transpose(1, 0, 2)), 1)
            v = np.concatenate((v, f64(bv[n]).transpose(1, 0, 2)), 1)
        if not k.shape[1]:
            continue
        for h in range(Hq):
            kk, vv, qq = k[h // G], v[h // G], qf[n, :, h]
            s = qq @ kk.T * scale
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[n, :, h] = p @ vv
            Ac, Ab = p[:, :m] @ np.abs(vv[:m]), p[:, m:] @ np.abs(vv[m:])
            ak = np.abs(kk)
            delta = scale * ((d + 8) * 2.0 ** -24 * (np.abs(qq) @ ak.T)
                             + qs * np.abs(qq).max(-1, keepdims=True) * ak.sum(-1)).max(-1) + 2.0 ** -21
            up = 2.0 ** (ve[h // G].max() - ve[h // G]) if m else np.zeros(0)
            tol[n, :, h] = 2.0 ** -8 * np.abs(out[n, :, h]) + 2.0 ** -11 * Ac \
                + (2 * delta[:, None] + 2.0 ** -13) * (Ac + Ab) \
                + 2.0 ** -26 * (up[:, None] * np.abs(vv[:m])).sum(0)
    return out, tol
