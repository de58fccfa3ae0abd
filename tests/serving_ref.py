"""Plain float64 (and, for the encoder, float32) forms of the serving operators, and the error
bounds that their tests use.

Bounds.  Sums of n fp32 terms are taken to err by at most 8 sqrt(n) 2^-24 times the sum of the
terms' magnitudes (independent roundings).  A result stored in f16 adds 2^-11 of its size (2^-25
below the normal range); what an operator holds in fewer bits on the way adds the term named at
each bound."""
import numpy as np

EPS = 2.0 ** -24


def _half_ulp(y, out):
    return np.maximum(2.0 ** -11 * np.abs(y), 2.0 ** -25) if out == "f16" else 2.0 ** -24 * np.abs(y)


# ------------------------------------------------------------------------------- adapters

def adapter(X, A, B, rank, scale, ids, base, out):
    """(Y, bound).  X (T, d_in), A (n, r, d_in), B (n, d_out, r); base None: zeros."""
    X, A, B = (np.asarray(t, np.float64) for t in (X, A, B))
    T, n, r_max = X.shape[0], A.shape[0], B.shape[2]
    y = np.zeros((T, B.shape[1])) if base is None else np.asarray(base, np.float64).copy()
    mag = np.abs(y)
    for t in range(T):
        a = int(ids[t])
        if not 0 <= a < n:
            continue
        r = min(max(int(rank[a]), 0), r_max)
        u, um = A[a, :r] @ X[t], np.abs(A[a, :r]) @ np.abs(X[t])
        y[t] += float(scale[a]) * (B[a, :, :r] @ u)
        mag[t] += abs(float(scale[a])) * (np.abs(B[a, :, :r]) @ um)
    # the second product takes u in 22 bits
    return y, (8 * np.sqrt(X.shape[1] + r_max) * EPS + 2.0 ** -22) * mag + _half_ulp(y, out)


# ------------------------------------------------------------------------------- 8-bit codes

def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -mag if c & 0x80 else mag
        if c & 0x7F == 0x7F:
            v[c] = np.nan
    return v


E4M3 = _e4m3_values()


def decode(codes, kind):
    codes = np.asarray(codes, np.uint8)
    return E4M3[codes] if kind == "fp8" else codes.view(np.int8).astype(np.float64)


def encode(x, scale, kind):
    """Codes of fp32 x / fp32 scale (0 where scale is 0)."""
    x, scale = np.asarray(x, np.float32), np.asarray(scale, np.float32)
    q = np.where(scale > 0, x / np.where(scale > 0, scale, np.float32(1)), np.float32(0))
    q = q.astype(np.float32)
    if kind == "int8":
        return np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    pos = E4M3[:127]                                   # 0 .. 448
    mid = (pos[1:] + pos[:-1]) / 2
    a = np.abs(q.astype(np.float64))
    code = np.searchsorted(mid, a, side="left")        # a tie stays below
    tie = np.isin(a, mid)
    code = np.where(tie & (code % 2 == 1), code + 1, code)  # ... unless that code is odd
    return (code | np.where(np.signbit(x) & (scale > 0), 0x80, 0)).astype(np.uint8)


def tame(x):
    x = np.asarray(x, np.float32)
    return np.clip(np.where(np.isnan(x), np.float32(0), x), np.float32(-65504), np.float32(65504))


def append(k, v, kscale, vscale, kind, K, V, tok_start, cached, table, page):
    """In place on the arrays k (pages, heads, page, dim), v (pages, heads, dim, page)."""
    n_pages, heads, P, dim = k.shape
    top = np.float32(448 if kind == "fp8" else 127)
    n_tok = K.shape[0]
    for r in range(len(cached)):
        t0 = min(max(int(tok_start[r]), 0), n_tok)
        n = min(max(int(tok_start[r + 1]), t0), n_tok) - t0
        pos, row = max(int(cached[r]), 0), t0
        while n > 0:
            lo = pos % P
            m = min(n, P - lo)
            lp = pos // P
            pg = int(table[r, lp]) if lp < table.shape[1] else -1
            if 0 <= pg < n_pages:
                for h in range(heads):
                    for codes, scales, src, tr in ((k, kscale, K, False), (v, vscale, V, True)):
                        x = tame(src[row:row + m, h * dim:(h + 1) * dim])
                        need = np.float32(np.abs(x).max()) / top
                        old = np.float32(scales[pg, h]) if lo else np.float32(0)
                        s = max(need, old)
                        block = codes[pg, h].T if tr else codes[pg, h]     # (page, dim) views
                        if need > old and lo:
                            was = (decode(block[:lo], kind).astype(np.float32) * old)
                            block[:lo] = encode(was.astype(np.float32), s, kind)
                        block[lo:lo + m] = encode(x, s, kind)
                        scales[pg, h] = s
            pos, row, n = pos + m, row + m, n - m


# ------------------------------------------------------------------------------- attention

def attention(k, v, kscale, vscale, kind, Q, tok_start, length, table, q_heads, sm_scale, window,
              sinks, out):
    """(O, bound, written): O (n_tok, q_heads, dim); rows of no request are not written."""
    n_pages, heads, P, dim = k.shape
    n_tok, g = Q.shape[0], q_heads // heads
    Q = np.asarray(Q, np.float64).reshape(n_tok, q_heads, dim)
    o, bound = np.zeros((n_tok, q_heads, dim)), np.zeros((n_tok, q_heads, dim))
    written = np.zeros(n_tok, bool)
    # softmax weights: 11 bits for f16 output, 22 for f32, down to 2^-38 of the largest
    wbits = 2.0 ** -11 if out == "f16" else 2.0 ** -21
    for r in range(len(length)):
        t0 = min(max(int(tok_start[r]), 0), n_tok)
        n = min(max(int(tok_start[r + 1]), t0), n_tok) - t0
        have = max(int(length[r]), 0)
        j = np.arange(min(have, table.shape[1] * P))
        pg = table[r, j // P].astype(np.int64)
        there = (pg >= 0) & (pg < n_pages)
        j, pg = j[there], pg[there]
        written[t0:t0 + n] = True
        for h in range(heads if n else 0):
            ks = decode(k[pg, h, j % P], kind) * kscale[pg, h, None].astype(np.float64)
            vc = decode(v[pg, h, :, j % P], kind)
            vs = vscale[pg, h].astype(np.float64)
            for i in range(n):
                p = have - n + i
                seen = j <= p
                if window > 0:
                    seen &= (p - j < window) | (j < sinks)
                if not seen.any():
                    continue
                kk, cc, ss = ks[seen], vc[seen], vs[seen]
                for x in range(h * g, (h + 1) * g):
                    q = Q[t0 + i, x]
                    s = (kk @ q) * sm_scale
                    es = (8 * np.sqrt(dim) + 8) * EPS * (np.abs(kk) @ np.abs(q)) * sm_scale
                    top = s.max()
                    w = np.exp(s - top)
                    # weight error: scores of this key and of the largest, exp's argument and
                    # value, then its stored bits
                    ew = w * (es + es.max() + 2.0 ** -22 * (2 + np.abs(s) + abs(top)))
                    ew += np.maximum(wbits * w, 2.0 ** -38)
                    l = w.sum()
                    vv = np.abs(cc) * ss[:, None]
                    o[t0 + i, x] = (w @ (cc * ss[:, None])) / l
                    bound[t0 + i, x] = (
                        ew @ vv + np.full(len(w), 2.0 ** -38) @ np.abs(cc) * ss.max()
                        + 16 * np.sqrt(len(w)) * EPS * (w @ vv)) / l + np.abs(
                            o[t0 + i, x]) * (ew.sum() / l + 16 * np.sqrt(len(w)) * EPS)
    return o, bound + _half_ulp(o, out), written
