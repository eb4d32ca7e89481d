"""Float64 references of the decode-step operators (numpy, from their
definitions) and the bounds their fp32 sums are held to."""
import math

import numpy as np

U = 2.0 ** -24          # half a step of fp32 arithmetic, relative


def unpack(qw):
    """uint32 words -> codes, low nibble first"""
    sh = (4 * np.arange(8)).astype(np.uint32)
    return ((qw[..., None] >> sh) & 15).reshape(*qw.shape[:-1], -1).astype(np.float64)


def packed_layer(rng, m, d, g, act=False, exact=False, lead=()):
    """A random packed layer (or a stack): dict of host arrays"""
    ng = 1 if g == -1 else d // g
    qw = rng.integers(0, 2 ** 32, (*lead, m, d // 8), dtype=np.uint32)
    z = rng.integers(0, 16, (*lead, m, ng))
    zp = np.concatenate([z, np.zeros((*lead, m, ng % 2), z.dtype)], -1)
    qz = (zp[..., 0::2] | (zp[..., 1::2] << 4)).astype(np.uint8)
    sc = (2.0 ** -rng.integers(4, 9, z.shape) if exact else rng.uniform(1e-3, 3e-2, z.shape))
    perm = None
    if act:
        perm = np.argsort(rng.random((*lead, d)), -1).astype(np.int32)
    return dict(qw=qw, z=z, qz=qz, sc=sc.astype(np.float16), perm=perm, g=g)


def dense(lay, e=None, magnitude=False):
    """Q (or s (c + z), the size of what the kernels sum) in original column order"""
    pick = (lambda a: a) if e is None else (lambda a: a[e])
    c, z, s = unpack(pick(lay["qw"])), pick(lay["z"]), pick(lay["sc"]).astype(np.float64)
    g = c.shape[1] // s.shape[1]
    z, s = np.repeat(z, g, 1), np.repeat(s, g, 1)
    q = s * (c + z if magnitude else c - z)
    if lay["perm"] is None:
        return q
    out = np.empty_like(q)
    out[:, pick(lay["perm"])] = q
    return out


def sum_units(d):
    """Roundings, in half steps of the summed magnitudes, that a product over d
    columns goes through: the longest chain of the kernels is one lane's d / 32
    terms, the joins of lanes, warps and slices add fewer than 24."""
    return (d / 32 + 24) * U


def lora(x, lay, a, b, scaling, ids):
    """(y, bound)"""
    x = x.astype(np.float64)
    a, b = a.astype(np.float64), b.astype(np.float64)
    d, r = x.shape[1], a.shape[1]
    y = x @ dense(lay).T
    bound = sum_units(d) * (np.abs(x) @ dense(lay, magnitude=True).T)
    for t, i in enumerate(ids):
        if 0 <= i < len(a):
            s = float(scaling[i])
            y[t] += s * (b[i] @ (a[i] @ x[t]))
            bound[t] += (sum_units(d) + sum_units(r) + 2 * U) * abs(s) * (
                np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[t])))
    return y, bound + 2 * U * np.abs(y)


def routes(logits, k, renorm):
    """Per token: [(expert, weight)], heaviest first"""
    out = []
    for row in logits.astype(np.float64):
        row = np.minimum(row, np.finfo(np.float32).max)
        live = [e for e in range(len(row)) if row[e] > -math.inf]
        best = sorted(live, key=lambda e: (-row[e], e))[:k]
        if not best:
            out.append([])
            continue
        p = {e: math.exp(row[e] - row[best[0]]) for e in live}
        total = math.fsum(p[e] for e in (best if renorm else live))
        out.append([(e, p[e] / total) for e in best])
    return out


def moe(x, logits, k, renorm, inn, out):
    """(y, bound).  The bound carries the sums' errors of gate and up through h
    = silu(gate) up (|silu'| <= 1.1) and through the second product; h enters it
    as two fp16 parts (22 bits: 2^-21 with the scaling); a route's weight has
    four roundings of expf, sum and quotient: 2^-20."""
    x = x.astype(np.float64)
    T, d = x.shape
    f = out["qw"].shape[-1] * 8
    y, bound = np.zeros((T, d)), np.zeros((T, d))
    cache = {}
    for t, row in enumerate(routes(logits, k, renorm)):
        for e, w in row:
            if e not in cache:
                cache[e] = [dense(lay, e, mag) for lay in (inn, out) for mag in (False, True)]
            qi, mi, qo, mo = cache[e]
            v, dv = qi @ x[t], sum_units(d) * (mi @ np.abs(x[t]))
            g, u = v[:f], v[f:]
            sg = g / (1 + np.exp(-g))
            h = sg * u
            dh = 1.1 * np.abs(u) * dv[:f] + np.abs(sg) * dv[f:] + dv[:f] * dv[f:] + 2.0 ** -20 * np.abs(h)
            o = qo @ h
            do = mo @ dh + (sum_units(f) + 2.0 ** -21) * (mo @ np.abs(h))
            y[t] += w * o
            bound[t] += w * (do + 2.0 ** -20 * np.abs(o))
    return y, bound + 8 * U * np.abs(y)


# ---- the 4-bit cache ------------------------------------------------------

def key_nibbles(D):
    """place[d]: the nibble of a key's words that holds element d"""
    d, nb = np.arange(D), D // 32
    return ((d % 32 // 8) * nb + d // 32) * 8 + d % 8


def value_nibbles(D):
    d, nb = np.arange(D), D // 32
    return ((d % 32 // 4) * nb + d // 32) * 4 + d % 4


def rotate(x, pos, table, inter, dtype):
    """The rotation in the given arithmetic (fp32 rounds every operation)"""
    x = x.astype(dtype).copy()
    if table is None:
        return x
    n = table.shape[1] // 2
    c, s = table[pos, :n].astype(dtype)[:, None], table[pos, n:].astype(dtype)[:, None]
    i = np.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + n)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def quantize(x, g):
    """codes, fp16 scales, zero points of rows x (fp32 arithmetic, each operation
    rounded): the definition of gptq_kv4_append"""
    f = np.float32
    big = np.finfo(f).max
    x = np.where(np.isnan(x), -big, np.clip(x, -big, big)).astype(f)
    v = x.reshape(*x.shape[:-1], -1, g)
    with np.errstate(over="ignore"):
        mn, mx = np.minimum(v.min(-1), f(0)), np.maximum(v.max(-1), f(0))
        flat = mn == mx
        mn, mx = np.where(flat, f(-1), mn), np.where(flat, f(1), mx)
        s = ((mx - mn) * f(1 / 15)).astype(np.float16)
        s = np.where(s == 0, np.float16(2.0 ** -24), np.where(np.isinf(s), np.float16(65504), s))
        sf = s.astype(f)
        z = np.clip(np.rint(-mn / sf), 0, 15).astype(f)
        c = np.clip(np.rint(v / sf[..., None]) + z[..., None], 0, 15)
    return c.astype(f).reshape(x.shape), s, z


def words(codes, place):
    """codes in element order -> the row's words with element d at nibble place[d]"""
    n = np.zeros(codes.shape, np.uint32)
    n[..., place] = codes.astype(np.uint32)
    n = n.reshape(*n.shape[:-1], -1, 8)
    return (n << (4 * np.arange(8)).astype(np.uint32)).sum(-1).astype(np.uint32)


def attention(q, K, V, Km, Vm, scale, lens, start, window, out):
    """K, V (seqs lists of L x hkv x D) the held values, Km, Vm the magnitudes
    s (c + z).  Fills out, returns the bound: fp16 rounding of the result, and,
    relative to sum p |V|'s magnitude, the scores' fp32 error (chains of D / 8 +
    8 terms and the 2 steps of the scaling), 2^-20 for exp2 and the two-part
    probabilities, and the sums' chains of L / 32 + 64 terms."""
    bound = np.zeros(out.shape)
    T, hq, D = q.shape
    q = q.astype(np.float64)
    for b, L in enumerate(lens):
        n = start[b + 1] - start[b]
        grp = hq // (K[b].shape[1] if L else 1)
        for i in range(n):
            t = start[b] + i
            hi = L - n + i + 1
            lo = max(0, hi - window) if window else 0
            out[t] = 0
            if hi <= lo:
                continue
            for h in range(hq):
                hk = h // grp
                s = scale * (K[b][lo:hi, hk] @ q[t, h])
                es = scale * np.max(Km[b][lo:hi, hk] @ np.abs(q[t, h])) * (D / 8 + 10) * 2 * U
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ V[b][lo:hi, hk]
                out[t, h] = o
                rel = 2 * es + 2.0 ** -20 + ((hi - lo) / 32 + 64) * U
                bound[t, h] = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + rel * (p @ Vm[b][lo:hi, hk]) * 1.01
    return bound
