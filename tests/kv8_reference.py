"""The 8-bit KV cache's operators in float64 numpy, written from their definitions: a cache is a dict of
`k`, `v` [B][Hkv][capacity][hd] (the codes' values), `k_scale`, `v_scale`, `weight` [B][Hkv][capacity / block]
and `ids`; lengths are plain lists."""
import numpy as np

SCALE_EXP_MIN = -117


def e4m3(x):
    """Nearest e4m3 numbers, ties to even: 4 significant bits, least exponent -6, infinities to 448, NaN kept."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        m, e = np.frexp(np.where(np.isfinite(x), x, 0.0))  # x = m 2^e, |m| in [0.5, 1)
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        y = np.rint(np.where(np.isfinite(x), x, 0.0) / step) * step
        y = np.clip(np.where(np.isinf(x), np.sign(x) * 448.0, y), -448.0, 448.0)
    return np.where(np.isnan(x), np.nan, y)


def scale_of(a):
    """Least power of two 2^e, e >= -117, with a <= 448 2^e."""
    e = SCALE_EXP_MIN
    while not a <= 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(c, block, lens, k_new, v_new, counts):
    """k_new, v_new [B][n][Hkv][hd]; changes c in place."""
    B, H = c["k_scale"].shape[:2]
    for b in range(B):
        lo, hi = lens[b], lens[b] + counts[b]
        held = -(-lo // block)
        for j in range(lo // block, -(-hi // block)):
            r0, r1 = max(lo, j * block), min(hi, (j + 1) * block)
            if r0 >= r1:
                continue
            for h in range(H):
                for x, new in (("k", k_new), ("v", v_new)):
                    rows = np.asarray(new[b, r0 - lo:r1 - lo, h], dtype=np.float64)
                    fin = np.abs(rows[np.isfinite(rows)])
                    s = scale_of(fin.max() if fin.size else 0.0)
                    if lo > j * block:
                        was = c[x + "_scale"][b, h, j]
                        s = max(s, was)
                        c[x][b, h, j * block:lo] = e4m3(c[x][b, h, j * block:lo] * (was / s))
                    c[x][b, h, r0:r1] = e4m3(rows / s)
                    c[x + "_scale"][b, h, j] = s
                if j >= held:
                    c["weight"][b, h, j] = 0.0
                    c["ids"][b, h, j] = (c["ids"][b, h, held - 1] + 1 if held else 0) + j - held


def attend(c, block, lens, q):
    """q [B][Hq][hd] -> (out [B][Hq][hd], each block's weight [B][Hkv][blocks], the largest |logit|)."""
    B, H = c["k_scale"].shape[:2]
    gq = q.shape[1] // H
    out, weight, top = np.zeros(q.shape), np.zeros(c["k_scale"].shape), 0.0
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        at = np.arange(n) // block
        for h in range(H):
            k = c["k"][b, h, :n] * c["k_scale"][b, h, at][:, None]
            v = c["v"][b, h, :n] * c["v_scale"][b, h, at][:, None]
            s = np.asarray(q[b, h * gq:(h + 1) * gq], dtype=np.float64) @ k.T / np.sqrt(q.shape[2])
            top = max(top, float(np.abs(s[np.isfinite(s)]).max(initial=0.0)))
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[b, h * gq:(h + 1) * gq] = p @ v
            np.add.at(weight[b, h], at, p.sum(0))
    return out, weight, top


def evict(c, block, lens, budget, sink, recent):
    """Changes c in place; returns the new lengths."""
    B, H = c["k_scale"].shape[:2]
    after = list(lens)
    for b in range(B):
        n = -(-lens[b] // block)
        if n <= budget:
            continue
        after[b] = lens[b] - (n - budget) * block
        for h in range(H):
            ids, w = c["ids"][b, h], c["weight"][b, h]

            def order(i):
                safe = ids[i] < sink or ids[i] > ids[n - 1] - recent or i == n - 1
                return (0, 0.0, i) if safe else (1, np.inf if np.isnan(w[i]) else -w[i], i)

            def by(i):  # NaN behind every number, -inf included
                safe, v, j = order(i)
                return (safe, bool(np.isnan(w[i])) and safe == 1, v, j)

            keep = sorted(sorted(range(n), key=by)[:budget])
            stay = {i for i in keep if i < budget - 1}
            src = [i for i in keep if i >= budget - 1]
            dst = [i for i in range(budget) if i not in stay]
            for x in ("k", "v"):
                rows = c[x][b, h].reshape(-1, block, c[x].shape[3])
                rows[dst] = rows[src].copy()
            for x in ("k_scale", "v_scale", "weight", "ids"):
                c[x][b, h, dst] = c[x][b, h, src].copy()
    return after
