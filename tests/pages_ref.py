"""Plain forms of the calls that keep the pages of the 8-bit cache, and of the selection of beams in
float64.  Whole numbers have to be equal."""
import numpy as np


def is_page(p, n):
    return 0 <= p < n


def lowest_free(refs):
    return iter([p for p, c in enumerate(refs) if c == 0])


def tables(refs, page, cached, n_new, n_tok, table):
    """In place on refs and table; the batch as a dict."""
    n_pages, width = len(refs), table.shape[1]
    start, length = [0], []
    req, pos = np.full(n_tok, -1), np.full(n_tok, -1)
    slot, missing = np.full(n_tok, -1, np.int64), 0
    free = lowest_free(refs.tolist())
    for r, (c, n) in enumerate(zip(cached, n_new)):
        c, n = max(int(c), 0), max(int(n), 0)
        n = min(n, n_tok - start[-1])
        start.append(start[-1] + n)
        length.append(c + n)
        for i in range(-(-c // page), min(-(-(c + n) // page), width)):
            if not is_page(table[r, i], n_pages):
                table[r, i] = next(free, -1)
                if table[r, i] < 0:
                    missing += 1
                else:
                    refs[table[r, i]] = 1
        for x in range(n):
            t, p = start[r] + x, c + x
            req[t], pos[t] = r, p
            if p // page < width and is_page(table[r, p // page], n_pages):
                slot[t] = int(table[r, p // page]) * page + p % page
    return {"tok_start": np.array(start), "length": np.array(length, np.int64), "tok_req": req,
            "tok_pos": pos, "slot": slot, "missing": np.array([missing])}


def release(refs, table, first=None, last=None):
    for r in range(table.shape[0]):
        lo = 0 if first is None else max(int(first[r]), 0)
        hi = table.shape[1] if last is None else min(int(last[r]), table.shape[1])
        for i in range(lo, hi):
            if is_page(table[r, i], len(refs)):
                refs[table[r, i]] -= 1
            table[r, i] = -1


def reorder(refs, page, table, length, parent, keep=False):
    """In place on refs; (table_out, length_out, src, dst, missing)."""
    n_pages, width = len(refs), table.shape[1]
    n_in, n_out = len(length), len(parent)
    out = np.full((n_out, width), -1, np.int64)
    length_out = np.zeros(n_out, np.int64)
    used = [min(-(-max(int(t), 0) // page), width) for t in length]
    for b, p in enumerate(parent):
        if 0 <= p < n_in:
            length_out[b] = max(int(length[p]), 0)
            for i in range(used[p]):
                if is_page(table[p, i], n_pages):
                    out[b, i] = table[p, i]
                    refs[table[p, i]] += 1
    if not keep:
        for row in table:
            for p in row:
                if is_page(p, n_pages):
                    refs[p] -= 1
    src, dst = np.full(n_out, -1), np.full(n_out, -1)
    missing, free, left = 0, lowest_free(refs.tolist()), []
    before = refs.copy()
    for b, p in enumerate(parent):
        t = int(length_out[b])
        if t % page == 0 or t // page >= width or out[b, t // page] < 0:
            continue
        old = out[b, t // page]
        children = [x for x in range(n_out) if parent[x] == p]
        if children[0] == b and before[old] == len(children):
            continue
        new = next(free, -1)
        out[b, t // page] = new
        left.append(old)
        if new < 0:
            missing += 1
        else:
            refs[new] = 1
            src[b], dst[b] = old, new
    for p in left:
        refs[p] -= 1
    return out, length_out, src, dst, np.array([missing])


def copy_pages(k, v, kscale, vscale, src, dst, length=None):
    """In place on k (pages, heads, page, dim), v (pages, heads, dim, page) and the scales."""
    n_pages, _, page, _ = k.shape
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (is_page(s, n_pages) and is_page(d, n_pages)):
            continue
        n = 0 if length is None else max(int(length[i]), 0) % page
        n = page if n == 0 else -(-n // 16) * 16
        k[d, :, :n] = k[s, :, :n]
        v[d, :, :, :n] = v[s, :, :, :n]
        kscale[d], vscale[d] = kscale[s], vscale[s]


def counts(n_pages, *tables_):
    """What refs has to be: how many entries of the tables name each page."""
    c = np.zeros(n_pages, np.int64)
    for t in tables_:
        for p in np.asarray(t).reshape(-1):
            if is_page(p, n_pages):
                c[p] += 1
    return c


# ------------------------------------------------------------------------------- beams

F32_MAX = float(np.finfo(np.float32).max)


def beam_totals(logits, score, eos, done=None):
    """total (rows, vocab) in float64, -inf where there is no continuation."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, F32_MAX))
    total = np.full(x.shape, -np.inf)
    for r in range(x.shape[0]):
        if not np.isfinite(score[r]):
            continue
        if done is not None and done[r]:
            total[r, eos] = float(score[r])
            continue
        top = x[r].max()
        if top > -np.inf:
            total[r] = float(score[r]) + (x[r] - (top + np.log(np.exp(x[r] - top).sum())))
    return total


def beam_select(logits, score, width, eos=-1, done=None, norm=None):
    """(parent, token, score, done, key): key in float64, for looking at near ties."""
    total = beam_totals(logits, score, eos, done)
    rows, vocab = total.shape
    norm = np.ones(rows) if norm is None else np.asarray(norm, np.float64)
    fine = (norm > 0) & np.isfinite(norm)
    with np.errstate(invalid="ignore"):
        key = np.where(fine[:, None], total * np.where(fine, norm, 1)[:, None], -np.inf)
    x = np.asarray(logits, np.float64)
    out = []
    for r0 in range(0, rows, width):
        found = []
        for r in range(r0, r0 + width):
            live = np.flatnonzero(key[r] > -np.inf)
            order = live[np.lexsort((live, -np.nan_to_num(x[r, live], neginf=-1e300)))][:width]
            found += [(-key[r, v], r, i, v) for i, v in enumerate(order)]
        found = sorted(found)[:width]
        for k, r, _, v in found:
            out.append((r, v, total[r, v], bool((done is not None and done[r]) or v == eos), -k))
        out += [(r0, -1, -np.inf, False, -np.inf)] * (width - len(found))
    return tuple(np.array(c) for c in zip(*out))
