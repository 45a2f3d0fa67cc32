"""Plain 64-bit reference of the 8-bit key / value cache and its attention
(csa2_kv8_*), restated from the rules in include/csa2.h with numpy alone: no
code, table or constant of the library."""
import math

import numpy as np


def e4m3_value(code):
    code = np.asarray(code, dtype=np.int64)
    e, m = (code >> 3) & 15, code & 7
    mag = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(code & 128, -mag, mag)


_POS = e4m3_value(np.arange(0x7F))              # 0 .. 448, ascending


def e4m3_encode(x):
    """Nearest code, ties to the even code, saturating; the sign kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_of(x):
    """The least power of two 2^e, -120 <= e <= 120, with max |finite x| <= 448 * 2^e."""
    a = np.abs(x)[np.isfinite(x)]
    top = a.max() if a.size else 0.0
    e = -120
    while e < 120 and top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    def __init__(self, batch, heads, dim, max_blocks, bs, n_blocks, table):
        self.B, self.heads, self.D, self.mb, self.bs = batch, heads, dim, max_blocks, bs
        self.table = table if table is not None else np.arange(batch * max_blocks).reshape(batch, max_blocks)
        self.k = np.zeros((n_blocks, heads, bs, dim), np.uint8)
        self.v = np.zeros_like(self.k)
        self.ks = np.zeros((n_blocks, heads))
        self.vs = np.zeros((n_blocks, heads))
        self.kb = np.zeros((n_blocks, heads, 2, dim), np.uint8)

    def append(self, b, start, k_new, v_new):
        """Rows [n, heads, dim] (float64) become positions start .. of sequence b."""
        n, bs = k_new.shape[0], self.bs
        at = start
        while at < start + n:
            end = min(start + n, (at // bs + 1) * bs)
            blk, r0, r1 = self.table[b, at // bs], at % bs, at % bs + end - at
            for h in range(self.heads):
                for codes, scales, src in ((self.k, self.ks, k_new), (self.v, self.vs, v_new)):
                    x = src[at - start:end - start, h]
                    s = scale_of(x)
                    was = scales[blk, h]
                    if r0:
                        s = max(s, was)
                        codes[blk, h, :r0] = np.where(s > was, e4m3_encode(e4m3_value(codes[blk, h, :r0]) * (was / s)),
                                                      codes[blk, h, :r0])
                    y = np.where(np.isnan(x), 0.0, x)
                    codes[blk, h, r0:r1] = e4m3_encode(y / s)
                    scales[blk, h] = s
                    if codes is self.k:
                        c = e4m3_value(codes[blk, h, r0:r1])
                        lo, hi = np.floor(c.min(0)), np.ceil(c.max(0))
                        if r0:
                            held = e4m3_value(self.kb[blk, h]) * (was / s)
                            lo, hi = np.minimum(lo, np.floor(held[0])), np.maximum(hi, np.ceil(held[1]))
                        self.kb[blk, h, 0], self.kb[blk, h, 1] = e4m3_encode(lo), e4m3_encode(hi)
            at = end

    def rows(self, b, h, t):
        """Keys and values (float64) of positions t of head h."""
        blk = self.table[b, t // self.bs]
        k = e4m3_value(self.k[blk, h, t % self.bs]) * self.ks[blk, h][:, None]
        v = e4m3_value(self.v[blk, h, t % self.bs]) * self.vs[blk, h][:, None]
        return k, v

    def attend(self, b, h, q, t, sm):
        """One query row over positions t: out, lse, and what error bounds need:
        sum of w |v| per channel, the greatest sum |q k| sm, max |v|."""
        D = self.D
        if len(t) == 0:
            return np.zeros(D), -math.inf, np.zeros(D), 0.0, 0.0
        k, v = self.rows(b, h, t)
        z = k @ q * sm
        m = z.max()
        w = np.exp(z - m)
        lse = m + math.log(w.sum())
        w = w / w.sum()
        return w @ v, lse, w @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * sm), float(np.abs(v).max())

    def select(self, b, h, q_group, p, n_sel, n_first, n_recent):
        """Chosen blocks of one row: q_group [G, D] float64."""
        vis = p // self.bs + 1 if p >= 0 else 0
        out = np.full(n_sel, -1, np.int32)
        if vis <= n_sel:
            out[:vis] = np.arange(vis)
            return out
        score = np.full(vis, -math.inf)
        q_group = np.where(np.isfinite(q_group), q_group, 0.0)
        blk = self.table[b, :vis]
        lo, hi, s = e4m3_value(self.kb[blk, h, 0]), e4m3_value(self.kb[blk, h, 1]), self.ks[blk, h]
        for q in q_group:
            e = -118
            while np.abs(q).max() > 127.0 * 2.0 ** e:
                e += 1
            qi = np.rint(q * 2.0 ** -e)
            score = np.maximum(score, (lo @ np.minimum(qi, 0) + hi @ np.maximum(qi, 0)) * s * 2.0 ** e)
        forced = [i for i in range(vis) if i < n_first or i >= vis - n_recent]
        rest = [i for i in range(vis) if n_first <= i < vis - n_recent]
        rest.sort(key=lambda i: (-score[i], i))
        out[:] = np.sort(np.array(forced + rest[:n_sel - len(forced)]))
        return out


def bounds(out, lse, wv, zmax, vmax, n, eps):
    """Error bounds of a row's output and lse.

    A weight is exp(z - max): z carries the fp32 accumulation of D <= 128
    products (each addition off by at most 2^-23 of the running magnitude,
    which sum |q k| bounds, 128 of them in chunks of 16: 2^-18 of it is ample),
    its scaling (2^-23 of |z|) and ex2 (2^-22): relative error dz = 2^-18 zmax +
    2^-20.  It is rounded to fp16 once (2^-11), or by at most 2^-25 2^-8 of the
    greatest weight once below fp16's normal range, at most n of those.  The
    sums add 2^-18.  Numerator and denominator both carry dz.  The output is
    rounded once (eps / 2).
    """
    dz = 2.0 ** -18 * zmax + 2.0 ** -20
    o = (2.0 ** -11 + 2 * dz + 2.0 ** -17) * wv + n * 2.0 ** -33 * vmax
    o = o + eps / 2 * (np.abs(out) + o) + 2.0 ** -25           # fp16's own subnormal step
    return o, dz + 2.0 ** -18 + 2.0 ** -22 * (abs(lse) if math.isfinite(lse) else 0.0)
