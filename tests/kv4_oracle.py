"""The 4-bit cache, rotary positions and their attention in fp64 numpy, from the
definitions (test infrastructure; shares no code with the package)."""
import math

import numpy as np


def bf16(x):
    """fp32 values rounded to the nearest bf16 (ties to even), as fp64."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, np.asarray(x, np.float32)).astype(np.float64)


def quantise(x):
    """Codes [..., d] (0..15) and scales [..., d/32] (fp64 of a bf16) of x [..., d]."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        m = np.abs(g).max(-1)
        bad = ~np.isfinite(g).all(-1)
        # m has 8 significant bits, so m / 7 in fp32 is never a tie of two bf16 that the quotient is not
        s = np.where(m < 2.0 ** -100, 0.0, bf16((m / 7).astype(np.float32)))
        s = np.where(bad, np.nan, s)
        use = (s > 0)[..., None]
        c = np.where(use, 8 + np.clip(np.floor(g / np.where(use, s[..., None], 1.0) + 0.5), -7, 7), 8.0)
    return c.astype(np.int64).reshape(np.shape(x)), s


def value(codes, scales):
    return ((codes - 8).reshape(*scales.shape, 32) * scales[..., None]).reshape(codes.shape)


def pack_tile(ck, sk, cv, sv):
    """The 18 d bytes of one tile from codes [16, d] and scales [16, d/32], entry by entry."""
    d = ck.shape[1]
    G = d // 32
    out = np.zeros(18 * d, np.uint8)
    for tok in range(16):
        for c in range(d):
            grp, r = divmod(c, 32)
            t, n = divmod(r, 8)
            out[((tok * 4 + t) * G + grp) * 4 + n // 2] |= int(ck[tok, c]) << (4 * (n % 2))
            g, i = divmod(r, 4)
            at = ((((tok // 8) * 8 + g) * 4 + tok % 8 // 2) * G + grp) * 2 + tok % 2
            out[8 * d + at * 2 + i // 2] |= int(cv[tok, c]) << (4 * (i % 2))
        for grp in range(G):
            for base, s in ((16 * d, sk), (17 * d, sv)):
                bits = np.float32(s[tok, grp]).view(np.uint32) >> 16
                if np.isnan(s[tok, grp]):
                    bits = 0x7fff
                at = base + 2 * (tok * G + grp)
                out[at], out[at + 1] = int(bits) & 255, int(bits) >> 8
    return out


def unpack_tile(b, d):
    """Codes and scales (ck, sk, cv, sv) of a tile's 18 d bytes."""
    G = d // 32
    ck, cv = np.zeros((16, d), np.int64), np.zeros((16, d), np.int64)
    for c in range(d):
        grp, r = divmod(c, 32)
        t, n = divmod(r, 8)
        g, i = divmod(r, 4)
        tok = np.arange(16)
        ck[:, c] = b[((tok * 4 + t) * G + grp) * 4 + n // 2] >> (4 * (n % 2)) & 15
        at = ((((tok // 8) * 8 + g) * 4 + tok % 8 // 2) * G + grp) * 2 + tok % 2
        cv[:, c] = b[8 * d + at * 2 + i // 2] >> (4 * (i % 2)) & 15
    s = b[16 * d:].copy().view(np.uint16).astype(np.uint32) << 16
    with np.errstate(invalid="ignore"):
        s = s.view(np.float32).astype(np.float64).reshape(2, 16, G)
    return ck, s[0], cv, s[1]


def rows(pool, pages, page, n, d):
    """K and V values [n, Hkv, d] of the first n tokens of a sequence with these pages."""
    H = pool.shape[1]
    k, v = np.zeros((n, H, d)), np.zeros((n, H, d))
    for t0 in range(0, n, 16):
        tile = pool[pages[t0 // page]].reshape(H, page // 16, 18 * d)[:, t0 % page // 16]
        m = min(16, n - t0)
        for h in range(H):
            ck, sk, cv, sv = unpack_tile(tile[h], d)
            k[t0:t0 + m, h], v[t0:t0 + m, h] = value(ck, sk)[:m], value(cv, sv)[:m]
    return k, v


def decode(q, ks, vs, scale):
    """O [B, Sq, Hq, d], LSE [B, Hq, Sq], and the sizes that bound the error of O and of
    LSE: sum_j p_j |v_j| and the largest sum of |q k| scale of a row.  q [B, Sq, Hq, d];
    ks, vs a list of [len, Hkv, d]."""
    B, Sq, Hq, d = q.shape
    o, w = np.zeros(q.shape), np.zeros(q.shape)
    lse, a = np.full((B, Hq, Sq), -np.inf), np.zeros((B, Hq, Sq))
    for b in range(B):
        n, H = ks[b].shape[:2]
        for h in range(Hq):
            kh, vh = ks[b][:, h // (Hq // H)], vs[b][:, h // (Hq // H)]
            for s in range(Sq):
                m = n - Sq + s + 1
                if m < 1:
                    continue
                x = kh[:m] @ q[b, s, h] * scale
                a[b, h, s] = (np.abs(kh[:m]) @ np.abs(q[b, s, h])).max() * scale
                lse[b, h, s] = x.max() + math.log(np.exp(x - x.max()).sum()) if np.isfinite(x.max()) else np.nan
                p = np.exp(x - lse[b, h, s])
                o[b, s, h], w[b, s, h] = p @ vh[:m], p @ np.abs(vh[:m])
    return o, lse, w, a


def rope(x, pos, axes, freq, interleaved, sign=1):
    """x [B, N, H, d] rotated, fp64; pos [B, N, A]."""
    y, half = np.array(x, np.float64), x.shape[-1] // 2
    x = y.copy()
    for p in range(len(freq)):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        t = (pos[:, :, axes[p]].astype(np.longdouble) * np.longdouble(freq[p]))[:, :, None]
        c, s = np.cos(t).astype(np.float64), sign * np.sin(t).astype(np.float64)
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    return y
