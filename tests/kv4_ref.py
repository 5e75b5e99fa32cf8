"""Plain 64-bit restatement of the paged 4-bit cache (include/fa_kv4.h) for the
tests: numpy, one request and one head at a time, no code of the library."""
import numpy as np

NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of a word that holds channel c


def bf16_bits(x):
    """fp64 -> bf16 bits, nearest, ties to even (x representable in fp32's range)."""
    x = np.asarray(x, np.float64)
    bits = x.view(np.int64)
    # 7 fraction bits of fp64's 52 stay; subnormal results are rounded at bf16's quantum
    r = ((bits + ((1 << 44) - 1) + ((bits >> 45) & 1)) >> 45) << 45
    big = r.view(np.float64)
    q = 2.0 ** -133
    small = np.rint(x / q) * q
    v = np.where(np.abs(x) < 2.0 ** -126, small, big)
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x, group):
    """fp64 [..., d] (bf16 values) -> codes [..., d], scale bits and minimum bits [..., d/group]."""
    g = x.reshape(*x.shape[:-1], -1, group)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        odd = ~np.isfinite(g).all(-1)
        lo, hi = np.where(odd, 0.0, lo), np.where(odd, 0.0, hi)
        sb = bf16_bits((hi - lo) / 15.0)
        s = bf16_value(sb)
        safe = np.where(s > 0, s, 1.0)[..., None]
        y, m = np.where(odd[..., None], 0.0, g), lo[..., None]
        D = y - m
        bb = D - y
        lost = (y - (D - bb)) + (-m - bb)  # y - m - D, exactly: bf16 values may be far apart
        f = np.clip(np.floor(D / safe), 0, 14)
        over = D - (f + 0.5) * safe        # exact near 0, so its sign is right
        over = np.where(over == 0, lost, over)
        c = f + ((over > 0) | ((over == 0) & (f % 2 == 1)))
        c = np.where(s[..., None] > 0, np.clip(c, 0, 15), 0).astype(np.int64)
    sb = np.where(odd, 0x7fc0, sb).astype(np.uint16)
    mb = np.where(odd, 0x7fc0, bf16_bits(lo)).astype(np.uint16)
    return c.reshape(x.shape), sb, mb


def values(codes, scale_bits, min_bits, group):
    c = codes.reshape(*codes.shape[:-1], -1, group).astype(np.float64)
    with np.errstate(all="ignore"):
        v = bf16_value(min_bits)[..., None] + bf16_value(scale_bits)[..., None] * c
    return v.reshape(codes.shape)


def pack(codes):
    w = codes.reshape(*codes.shape[:-1], -1, 8)
    nib = np.zeros_like(w)
    nib[..., NIBBLE] = w
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).astype(np.uint8).reshape(*codes.shape[:-1], -1)


def unpack(b):
    w = b.reshape(*b.shape[:-1], -1, 4).astype(np.int64)
    nib = np.stack([w & 15, w >> 4], -1).reshape(*w.shape[:-1], 8)
    return nib[..., NIBBLE].reshape(*b.shape[:-1], -1)


def sections(page, d, group):
    """Byte ranges of a record: K codes, K params, V codes, V params."""
    n, p = page * d // 2, page * 4 * (d // group)
    at, out = 0, []
    for size in (n, p, n, p):
        out.append((at, at + size))
        at += size
    return out


def token_rows(cache, slots, page, d, group):
    """numpy cache [pages, heads, record], slots >= 0 -> (K, V), each a tuple
    (codes [T, heads, d], scale bits, minimum bits)."""
    slots = np.asarray(slots, np.int64)
    rec = cache[slots // page]
    off = slots % page
    out = []
    sec = sections(page, d, group)
    for c, p in (sec[0:2], sec[2:4]):
        codes = rec[..., c[0]:c[1]].reshape(len(slots), cache.shape[1], page, d // 2)
        par = rec[..., p[0]:p[1]].reshape(len(slots), cache.shape[1], page, 4 * (d // group))
        codes = codes[np.arange(len(slots)), :, off]
        par = np.ascontiguousarray(par[np.arange(len(slots)), :, off]).view(np.uint16)
        out.append((unpack(codes), par[..., 0::2], par[..., 1::2]))
    return out


def random_cache(rng, pages, heads, page, d, group, spread=1.0):
    """A cache whose every row is quantised from drawn keys and values (numpy uint8)."""
    cache = np.zeros((pages, heads, sections(page, d, group)[-1][1]), np.uint8)
    sec = sections(page, d, group)
    for c, p in (sec[0:2], sec[2:4]):
        x = bf16_value(bf16_bits(spread * rng.standard_normal((pages, heads, page, d))
                                 + rng.standard_normal((1, heads, 1, d))))
        codes, sb, mb = quantise(x, group)
        cache[..., c[0]:c[1]] = pack(codes).reshape(pages, heads, -1)
        par = np.stack([sb, mb], -1).reshape(pages, heads, page, -1)
        cache[..., p[0]:p[1]] = np.ascontiguousarray(par).view(np.uint8).reshape(pages, heads, -1)
    return cache


def attention(q, cache, table, cu, kv_len, page, group, scale, causal, window):
    """fp64 O [total, Hq, d], L [total, Hq], and bounds of what the kernels' arithmetic may
    change: tol_o, tol_l of the same shapes.

    Scores: products of bf16 queries and codes are exact and summed in fp32 as
    sum q (128 + c), scaled and offset by (m - 128 s) sum q; each of at most d / 16 + 8 partial
    sums loses at most 2^-22 of the sum of the magnitudes (a truncating accumulator), which
    bounds the score's error e.  The weights p = exp(score) are then off by a factor
    exp(2 e) (numerator and denominator), the weights and the values are rounded to bf16 (half
    a step, 2^-8), the sum of the rounded weights divides, and O is rounded to bf16 once more:
      |dO| <= (2 (e^{2e} - 1) + 3 * 2^-8 * 1.02) sum p |v| + 2^-8 |O|
      |dL| <= e + 2^-21 (|L| + 8).
    """
    total, Hq, d = q.shape
    heads = cache.shape[1]
    per = Hq // heads
    O, tol_o = np.zeros((total, Hq, d)), np.zeros((total, Hq, d))
    L, tol_l = np.full((total, Hq), -np.inf), np.zeros((total, Hq))
    for b in range(len(kv_len)):
        lo, hi = int(cu[b]), int(cu[b + 1])
        n = hi - lo
        length = int(min(max(kv_len[b], 0), table.shape[1] * page))
        if n == 0:
            continue
        j = np.arange(length)
        if length:
            slots = table[b, j // page].astype(np.int64) * page + j % page
            (kc, ks, km), (vc, vs, vm) = token_rows(cache, slots, page, d, group)
        pos = length - n + np.arange(n)
        see = np.ones((n, length), bool)
        if causal or window >= 0:
            see &= j[None] <= pos[:, None]
        if window >= 0:
            see &= j[None] >= pos[:, None] - window
        for h in range(Hq):
            if not length:
                continue
            g = h // per
            K = values(kc[:, g], ks[:, g], km[:, g], group)
            V = values(vc[:, g], vs[:, g], vm[:, g], group)
            s_abs = np.repeat(np.abs(bf16_value(ks[:, g])), group, -1)
            m_abs = np.repeat(np.abs(bf16_value(km[:, g])), group, -1)
            Q = q[lo:hi, h]
            with np.errstate(all="ignore"):
                S = scale * (Q @ K.T)
                mag = scale * (np.abs(Q) @ (271.0 * s_abs + m_abs).T)
                err = (d / 16 + 8) * 2.0 ** -22 * mag
                S = np.where(see, S, -np.inf)
                err = np.where(see, err, 0.0)
                top = S.max(-1, keepdims=True)
                empty = ~see.any(-1)
                P = np.exp(S - np.where(empty[:, None], 0.0, top))
                P = np.where(see, P, 0.0)
                l = P.sum(-1, keepdims=True)
                P = P / np.where(l > 0, l, 1.0) if np.isfinite(l).all() else P / l
                Vs = V
                bad = ~np.isfinite(V).all(-1)
                o = np.zeros((n, d))
                ab = np.zeros((n, d))
                for i in range(n) if bad.any() else ():
                    o[i] = P[i, see[i]] @ Vs[see[i]]
                    ab[i] = P[i, see[i]] @ np.abs(Vs[see[i]])
                if not bad.any():
                    o, ab = P @ Vs, P @ np.abs(Vs)
                e = err.max(-1)
                O[lo:hi, h] = o
                L[lo:hi, h] = np.where(empty, -np.inf, (top + np.log(l))[:, 0])
                grow = 2.0 * np.expm1(2.0 * e)
                tol_o[lo:hi, h] = (grow[:, None] + 3.06 * 2.0 ** -8) * ab + 2.0 ** -8 * np.abs(o)
                tol_l[lo:hi, h] = e + 2.0 ** -21 * (np.abs(np.where(empty, 0.0, L[lo:hi, h])) + 8)
    return O, L, tol_o, tol_l


def plan(past, new, table, ring, head, count, page, max_tokens):
    """The step's bookkeeping, request by request.  Returns kv_len, cu, slots, state, table, ring."""
    B, width = table.shape
    F = len(ring)
    table, ring0, ring = table.copy(), ring, ring.copy()
    cu, slots, kv = [0], [], []
    used = back = served = 0
    open_ = True
    tail = head + count
    for b in range(B):
        p, n = int(past[b]), int(new[b])
        valid = p >= 0 and n >= -1 and p + max(n, 0) <= width * page
        held = -(-p // page) if valid else 0
        if valid and n == -1:
            for j in range(held):
                ring[(tail + back) % F] = table[b, j]
                back += 1
        take = -(-(p + max(n, 0)) // page) - held if valid and n >= 0 else 0
        add = max(n, 0) if valid else 0
        if open_ and valid and used + take <= count and cu[-1] + add <= max_tokens:
            for j in range(take):
                table[b, held + j] = ring0[(head + used + j) % F]
            for t in range(p, p + add):
                slots.append(int(table[b, t // page]) * page + t % page)
            used += take
            served += 1
        else:
            open_ = False
            add = 0
        cu.append(cu[-1] + add)
        kv.append(0 if n == -1 else p + add)
    slots = slots + [-1] * (max_tokens - len(slots))
    state = [(head + used) % F, count - used + back, cu[-1], served]
    return [np.asarray(x, np.int32) for x in (kv, cu, slots, state)] + [table, ring]
