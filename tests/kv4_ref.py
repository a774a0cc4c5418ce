"""Plain reference of the paged 4-bit cache in numpy: its number formats bit by
bit, the quantisation in single fp32 operations (which numpy rounds as IEEE
asks, as the definition in include/herald.h does), and attention in fp64."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def _e4m3_table():
    t = np.empty(256, np.float64)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[b] = np.nan if b & 127 == 127 else v
        if b & 128:
            t[b] = -t[b]
    return t


E4M3 = _e4m3_table()


def bf16(x):
    """fp32/fp64 array -> the nearest bf16 bit patterns (ties to even)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(np.asarray(x, np.float32)), np.uint16(0x7FC0), r)


def f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x, scale0):
    """x [..., d] fp32 -> (codes [..., d/2], scales [..., d/16]) bytes."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 16)
    scale0 = np.float32(scale0)
    with np.errstate(all="ignore"):
        r = np.abs(g).max(-1) / (np.float32(6) * scale0)       # NaN stays
        r = r.astype(np.float64)
        # nearest e4m3, ties to the even code (the codes 0..126 ascend)
        pos = E4M3[:127]
        c = np.clip(np.where(np.isnan(r), 0, r), 0, 448)
        hi = np.clip(np.searchsorted(pos, c), 1, 126)
        lo = hi - 1
        dl, dh = c - pos[lo], pos[hi] - c
        s = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
        s = np.where(np.isnan(r), np.uint8(127), s)
        full = (E4M3[s].astype(np.float32) * scale0)[..., None]
        y = np.where(full > 0, g / np.where(full > 0, full, 1), np.float32(0)).astype(np.float64)
        a = np.abs(y)
        mids = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.])
        low, high = np.searchsorted(mids, a, "left"), np.searchsorted(mids, a, "right")
        code = np.where((low != high) & (low % 2 == 1), high, low)
        code = (code + 8 * np.signbit(y)).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def values(codes, scales, scale0):
    """Held bytes -> fp64 values [..., d] (scale0 as the fp32 it is)."""
    v = np.stack((E2M1[codes & 15], E2M1[codes >> 4]), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return v * np.repeat(E4M3[scales], 16, -1) * np.float64(np.float32(scale0))


def rotate32(x, cos_sin, pos, rot, interleaved):
    """x [..., T, H, d] fp32 at positions pos [..., T]: each product and sum rounded to fp32."""
    x = np.array(x, np.float32)
    if not rot:
        return x
    c, s = cos_sin[pos][..., None, :, 0], cos_sin[pos][..., None, :, 1]
    sl = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if interleaved else \
        (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
    a, b = x[sl[0]].copy(), x[sl[1]].copy()
    x[sl[0]] = a * c - b * s
    x[sl[1]] = b * c + a * s
    return x


def angles(n_pos, rot, theta=10000.0):
    a = np.arange(n_pos)[:, None] * theta ** (-np.arange(0, rot, 2) / rot)
    return np.ascontiguousarray(np.stack((np.cos(a), np.sin(a)), -1), np.float32)


class Cache:
    """A paged cache on the host, filled by append(); random bytes (NaN scales
    among them) stand wherever no row is written."""

    def __init__(self, rng, N, Hkv, d, page, lengths, k_scale=1.0, v_scale=1.0, spare=2):
        self.N, self.Hkv, self.d, self.page = N, Hkv, d, page
        self.k_scale, self.v_scale = k_scale, v_scale
        need = [max(0, -(-int(x) // page)) for x in lengths]
        self.max_pages = max(1, max(need))
        self.n_pages = sum(need) + spare
        perm = rng.permutation(self.n_pages)[: sum(need)]
        self.table = np.full((N, self.max_pages), -1, np.int32)
        at = 0
        for n, m in enumerate(need):
            self.table[n, :m] = perm[at: at + m]
            at += m
        self.codes = rng.integers(0, 256, (2, self.n_pages, Hkv, page, d // 2), dtype=np.uint8)
        self.scales = rng.integers(0, 256, (2, self.n_pages, Hkv, page, d // 16), dtype=np.uint8)
        self.scales[rng.random(self.scales.shape) < 0.2] = 0x7F

    def write(self, n, pos, k, v):
        """Rows k, v [len(pos), Hkv, d] fp32 of sequence n."""
        pos = np.asarray(pos)
        ph, r = self.table[n, pos // self.page], pos % self.page
        ok = ph >= 0
        for i, (x, s) in enumerate(((k, self.k_scale), (v, self.v_scale))):
            c, sc = quantise(x, s)
            self.codes[i].transpose(0, 2, 1, 3)[ph[ok], r[ok]] = c[ok]
            self.scales[i].transpose(0, 2, 1, 3)[ph[ok], r[ok]] = sc[ok]

    def rows(self, i, n, pos):
        """fp64 values [Hkv, len(pos), d] of K (i = 0) or V; pages must exist."""
        pos = np.asarray(pos, np.int64)
        ph, r = self.table[n, pos // self.page], pos % self.page
        c = self.codes[i].transpose(0, 2, 1, 3)[ph, r]
        s = self.scales[i].transpose(0, 2, 1, 3)[ph, r]
        return values(c, s, (self.k_scale, self.v_scale)[i]).transpose(1, 0, 2)


def attention(q, cache, lengths, bk=None, bv=None, scale=None):
    """fp64 attention of q [N][B][Hq][d] (bf16 bits) over the cache and the
    block's keys, and the bound of an implementation that rounds P to fp16
    (cache) or bf16 (block keys), accumulates in fp32 and rounds the output to
    bf16:
      2^-8 |out|                       the output's rounding (half a bf16 step)
      2^-11 A_c + 2^-8 A_b             P's rounding; A = sum_j p_j |v_j| over the
                                       cache and over the block keys
      2 delta (A_c + A_b)              relative error of each weight and of the
                                       row sum: delta = (d + 8) 2^-24 max_j
                                       sum_i |q_i k_ji| scale (fp32 sums of d
                                       products and a few fp32 roundings of the
                                       score) + 2^-21 (exp2)
      2^-13 (A_c + A_b)                fp32 sums over up to 2^10 matrix steps
      2^-30 sum_c |v_j|                P below fp16's 2^-14 is off by half a
                                       subnormal step, 2^-25, whatever its size;
                                       the row's largest P is at least 2^5 (its
                                       exponent base is set 11 below the largest
                                       score with few rows, 5 below it with many)
                                       and the row sum no less, so each cache key
                                       adds at most 2^-25 / 2^5 |v_j|
    Returns (out, bound)."""
    N, B, Hq, d = q.shape
    Hkv = cache.Hkv
    G = Hq // Hkv
    scale = 1 / np.sqrt(d) if scale is None else scale
    qf = f64(q)
    out = np.zeros((N, B, Hq, d))
    tol = np.zeros_like(out)
    for n in range(N):
        L = int(lengths[n])
        pos = np.arange(L)
        pos = pos[cache.table[n, pos // cache.page] >= 0]
        k, v = cache.rows(0, n, pos), cache.rows(1, n, pos)
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
            delta = (d + 8) * 2.0 ** -24 * (np.abs(qq) @ np.abs(kk).T).max(-1) * scale + 2.0 ** -21
            tol[n, :, h] = 2.0 ** -8 * np.abs(out[n, :, h]) + 2.0 ** -11 * Ac + 2.0 ** -8 * Ab \
                + (2 * delta[:, None] + 2.0 ** -13) * (Ac + Ab) + 2.0 ** -30 * np.abs(vv[:m]).sum(0)
    return out, tol
